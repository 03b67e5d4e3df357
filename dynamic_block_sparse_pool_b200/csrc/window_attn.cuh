// Arguments of the window attention's kernels and their launchers.
#pragma once

#include "window.cuh"

namespace dsa {

struct WindowAttn {
  int B, H, Hk, D;
  Window w;
  float scale;
  const void *q, *k, *v;      // [B, H or Hk, Nq or Nk, D]
  void* out;                  // [B, H, Nq, D]
  float* lse;                 // [B, H, Nq]; forward: NULL if not wanted
  // backward
  const void *o, *dout;       // the forward's output and its gradient
  void *dq, *dk, *dv;
  float* delta;               // workspace, [B, H, Nq]
  int num_sms;
  unsigned* err;
};

struct DecodeAttn {
  int B, H, Hk, group, Nq, cap;
  float scale;
  int left, sink;             // left: at most Window::kNoBound
  const void *q, *k, *v;      // q [B, H, Nq, D]; k, v [B, Hk, cap, D] through strides
  long long ks[3], vs[3];     // strides of stream, head, key, in elements
  const int32_t* lens;        // [B]: keys in the cache, the new tokens' among them
  void* out;                  // [B, H, Nq, D]
  float* lse;                 // [B, H, Nq], NULL if not wanted
  int num_sms;
  unsigned* err;
};

cudaError_t launch_window_decode(const DecodeAttn& a, bool bf16, int D, cudaStream_t s);

// bf16 on tcgen05
cudaError_t launch_window_fwd_sm100(const WindowAttn& a, cudaStream_t s, const char** why);
cudaError_t launch_window_bwd_sm100(const WindowAttn& a, cudaStream_t s, const char** why);
// fp32 on CUDA cores
cudaError_t launch_window_fwd_simt(const WindowAttn& a, cudaStream_t s);
cudaError_t launch_window_bwd_simt(const WindowAttn& a, cudaStream_t s);

}  // namespace dsa
