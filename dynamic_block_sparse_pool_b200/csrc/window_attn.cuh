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
  float* shares;              // workspace, simt_share_floats (fp32)
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
  int groups;                 // CTAs per head that join through the workspace
  float* ws;                  // [groups][B H Nq][D], then [groups][B H Nq] (maximum, sum)
  unsigned* err;
};

// How the keys of one head are shared: `cluster` CTAs that join on the SMs, or
// `groups` that join through the workspace (one of the two is 1).
struct DecodePlan {
  int tiles, cluster, groups;  // tiles: of a group's rows
};
DecodePlan decode_plan(bool bf16, int B, int H, int Hk, int Nq, int cap, int D, int left, int sink);

cudaError_t launch_window_decode(const DecodeAttn& a, const DecodePlan& plan, bool bf16, int D, cudaStream_t s,
                                 const char** why);

// bf16 on tcgen05
cudaError_t launch_window_fwd_sm100(const WindowAttn& a, cudaStream_t s, const char** why);
cudaError_t launch_window_bwd_sm100(const WindowAttn& a, cudaStream_t s, const char** why);
// fp32 on CUDA cores
// Chunks of a gradient tile's pairs, and the floats their shares take.
struct SimtChunks {
  int chunk_q, chunks_q, chunk_k, chunks_k;
};
SimtChunks simt_chunks(int B, int H, int Hk, const Window& w);
size_t simt_share_floats(int B, int H, int Hk, const Window& w, int D);
cudaError_t launch_window_fwd_simt(const WindowAttn& a, cudaStream_t s);
cudaError_t launch_window_bwd_simt(const WindowAttn& a, cudaStream_t s);

}  // namespace dsa
