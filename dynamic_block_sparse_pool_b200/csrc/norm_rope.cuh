// Arguments of the per-head norm with rotation (launchers in
// qk_norm_rope.cu).  Strides are in elements; x and dx rows are contiguous.
#pragma once

#include "common.cuh"

namespace dsa {

// Most CTAs the backward uses (three on each of 148 SMs); each leaves its
// share of one weight gradient in the workspace.
constexpr int kNormRopeBwdCtas = 444;

struct RopeArgs {
  const float2* table;      // per axis a: [len[a]][pairs[a]] (cos, sin), axes one after another
  const int32_t* pos;       // [B or 1][N][3]
  long long pos_bstride;    // 3 N, or 0 where every batch entry has the same positions
  int pairs[3], len[3];
};

struct NormRopeFwd {
  const void *xq, *xk;
  const float *xq_scale, *xk_scale;  // set: x is int8 codes
  long long qb, qn, qh, kb, kn, kh;
  bool bf16;
  int B, N, Hq, Hk, D;
  const float *wq, *wk;              // NULL: ones
  float eps;
  RopeArgs rope;
  bool halves;
  void *q, *k;
  int8_t *xq8, *xk8;                 // set: the codes of x are written too
  float *xq8_scale, *xk8_scale;
  unsigned* err;
};

struct NormRopeBwd {
  const void *gq, *gk;
  const void *xq, *xk;
  const float *xq_scale, *xk_scale;
  long long qb, qn, qh, kb, kn, kh;
  bool bf16;
  int B, N, Hq, Hk, D;
  const float *wq, *wk;
  float eps;
  RopeArgs rope;
  bool halves;
  void *dxq, *dxk;
  long long dqb, dqn, dqh, dkb, dkn, dkh;
  float *dwq, *dwk;                  // NULL: not wanted
  float* part;                       // kNormRopeBwdCtas * D floats
  unsigned* err;
};

cudaError_t launch_rope_table(int positions, int pairs, double theta, float2* table, cudaStream_t s);
cudaError_t launch_qk_norm_rope(const NormRopeFwd& f, cudaStream_t s);
cudaError_t launch_qk_norm_rope_bwd(const NormRopeBwd& f, cudaStream_t s);

}  // namespace dsa
