// Norms of queries and keys for each head with the position rotation in the
// same pass, and its gradient.
//
// Per (token, head) row x of D values, with r = 1 / sqrt(mean(x^2) + eps):
//   forward   n = x r w;  every pair (a, b) of n turns by its angle:
//             (a cos - b sin, a sin + b cos).
//   backward  g = the gradient turned back;  dw = sum over rows of g x r;
//             with h = x r and m = mean(g w h):  dx = r (g w - h m).
// All in fp32 from the loaded values, rounded once at the store.
//
// Bound by memory (about 3 to 4 operations per byte): every row is read once
// and written once, so nothing but the layout is left to choose.  x is
// token-major (strided: the fused projection's output is read in place), y
// is head-major, and the rotation depends on the token alone, so a warp
// keeps one token: it fetches the token's cosines and sines once (from small
// per-axis tables that stay in L1) and runs over the token's heads, D / 8
// threads of eight values per row.  Reads are whole token rows; writes are
// one row per head, next to those of the seven tokens of the CTA's other
// warps.  kUnroll rows per thread are in flight to cover the latency of HBM.
//
// x may be 8-bit rows (codes and scales, rows8.cuh) in place of bf16 or fp32,
// and the forward can write those of x beside y, so a training step keeps a
// byte per value where it kept two and reads less in the backward.
#include <algorithm>

#include "norm_rope.cuh"
#include "rows8.cuh"

namespace dsa {
namespace {

using namespace rows8;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Cosine and sine of the pairs a thread's eight values belong to: four
// neighbouring pairs, or (halves) eight, the partner values being in the
// thread D / 16 further on.
template <int D, bool HALVES>
struct Turn {
  static constexpr int kPairs = HALVES ? 8 : 4;
  float c[kPairs], s[kPairs];

  // The token's angles from the tables.  A position below 0 does not turn;
  // one past its axis' table is reported and does not turn either.
  __device__ __forceinline__ void load(const RopeArgs& a, int b, int n, int sub, unsigned* err) {
    const int32_t* p = a.pos + b * a.pos_bstride + (long long)n * 3;
    const int first = HALVES ? (8 * sub) % (D / 2) : 4 * sub;
    int at[3];
    bool bad = false;
#pragma unroll
    for (int x = 0; x < 3; ++x) {
      const int v = a.pairs[x] > 0 ? p[x] : -1;
      bad |= v >= a.len[x] && a.pairs[x] > 0;
      at[x] = v >= a.len[x] ? -1 : v;
    }
    if (bad && sub == 0) flag_error(err, kErrPosition);
#pragma unroll
    for (int m = 0; m < kPairs; ++m) {
      int i = first + m, base = 0, x = 0;
      if (i >= a.pairs[0]) {
        i -= a.pairs[0];
        base = a.len[0] * a.pairs[0];
        x = 1;
        if (i >= a.pairs[1]) {
          i -= a.pairs[1];
          base += a.len[1] * a.pairs[1];
          x = 2;
        }
      }
      const int pa = x == 0 ? a.pairs[0] : x == 1 ? a.pairs[1] : a.pairs[2];
      const int v = x == 0 ? at[0] : x == 1 ? at[1] : at[2];
      float2 t = make_float2(1.f, 0.f);
      if (v >= 0 && i < pa) t = __ldg(a.table + base + (long long)v * pa + i);
      c[m] = t.x;
      s[m] = t.y;
    }
  }

  // Turns the thread's eight values (back: by the opposite angle).
  template <bool BACK>
  __device__ __forceinline__ void apply(float (&v)[8], int sub) const {
    if (HALVES) {
      // first half: a cos - b sin; second half: b cos + a sin
      const bool lower = sub < D / 16;
      const float sign = (lower != BACK) ? -1.f : 1.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float o = __shfl_xor_sync(0xffffffffu, v[e], D / 16);
        v[e] = fmaf(v[e], c[e % kPairs], sign * o * s[e % kPairs]);
      }
    } else {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float a = v[2 * m], b = v[2 * m + 1], t = BACK ? -s[m % kPairs] : s[m % kPairs];
        v[2 * m] = fmaf(a, c[m % kPairs], -b * t);
        v[2 * m + 1] = fmaf(a, t, b * c[m % kPairs]);
      }
    }
  }
};

// One side (q or k) of a pass.
template <typename TIn>
struct Side {
  const TIn* x;
  const float* xs;   // scales of 8-bit x
  long long b, n, h; // strides of x, in elements
  int heads;
  const float* w;
};

__device__ __forceinline__ void load_weight(const float* w, int sub, float (&v)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 1.f;
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = __ldg(w + 8 * sub + e);
}

template <typename TIn>
__device__ __forceinline__ void fetch(const Side<TIn>& s, int b, int n, int h, int N, int sub, Raw<TIn>& r) {
  load8(s.x + b * s.b + n * s.n + h * s.h + 8 * sub, r);
}
__device__ __forceinline__ void fetch(const Side<int8_t>& s, int b, int n, int h, int N, int sub,
                                      Raw<int8_t>& r) {
  load8(s.x + b * s.b + n * s.n + h * s.h + 8 * sub, r);
  r.scale = __ldg(s.xs + ((long long)b * N + n) * s.heads + h);
}

template <typename TIn, typename TOut>
struct FwdArgs {
  Side<TIn> q, k;
  TOut *yq, *yk;
  int8_t *cq, *ck;   // codes of x (SAVE8)
  float *sq, *sk;
  int N;
  long long tokens;  // B * N
  float eps;
  RopeArgs rope;
  unsigned* err;
};

// Grid: x = tokens / 8 (one warp per token), y = parts of the token's heads.
// A step is kUnroll * (32 / TPR) heads of q or of k.
template <typename TIn, typename TOut, int D, bool HALVES, bool SAVE8, int UNROLL>
__global__ void __launch_bounds__(kThreads)
qk_norm_rope_kernel(const FwdArgs<TIn, TOut> a) {
  constexpr int TPR = D / 8, RPW = 32 / TPR, kStep = UNROLL * RPW;
  const int lane = threadIdx.x & 31, sub = lane % TPR, slot = lane / TPR;
  const long long token = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (token >= a.tokens) return;
  const int b = (int)(token / a.N), n = (int)(token - (long long)b * a.N);
  const int steps_q = ceil_div(a.q.heads, kStep), steps = steps_q + ceil_div(a.k.heads, kStep);
  const int per = ceil_div(steps, (int)gridDim.y);
  const int s0 = blockIdx.y * per, s1 = min(steps, s0 + per);
  Turn<D, HALVES> turn;
  float w[8];
  for (int st = s0; st < s1; ++st) {
    const bool is_k = st >= steps_q;
    const Side<TIn>& side = is_k ? a.k : a.q;
    const int heads = side.heads, h0 = (is_k ? st - steps_q : st) * kStep + slot;
    Raw<TIn> raw[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      fetch(side, b, n, min(h0 + u * RPW, heads - 1), a.N, sub, raw[u]);
    if (st == s0) turn.load(a.rope, b, n, sub, a.err);
    if (st == s0 || st == steps_q) load_weight(side.w, sub, w);
    TOut* y = is_k ? a.yk : a.yq;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int h = h0 + u * RPW;
      float v[8];
      values8(raw[u], v);
      if (SAVE8) {
        float scale;
        const uint2 c = encode8<TPR>(v, scale);
        if (h < heads) {
          const long long row = token * heads + h;
          *reinterpret_cast<uint2*>((is_k ? a.ck : a.cq) + row * D + 8 * sub) = c;
          if (sub == 0) (is_k ? a.sk : a.sq)[row] = scale;
        }
      }
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
      const float r = rsqrtf(row_sum<TPR>(ss) * (1.0f / D) + a.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] * r * w[e];
      turn.template apply<false>(v, sub);
      if (h < heads) store8(y + (((long long)b * heads + h) * a.N + n) * D + 8 * sub, v);
    }
  }
}

template <typename TX, typename TG>
struct BwdArgs {
  Side<TX> q, k;
  const TG *gq, *gk;        // gradients of y, [B, heads, N, D]
  TG *dq, *dk;              // gradients of x
  long long dqb, dqn, dqh, dkb, dkn, dkh;  // their strides, in elements
  float* part;              // [CTAs][2][D]: the CTA's share of dwq | dwk
  int N;
  long long tokens;
  float eps;
  RopeArgs rope;
  unsigned* err;
};

// Persistent: warp g of all the warps takes tokens g, g + warps, ... (the grid
// does not depend on the data, so each thread sums dw over the same rows in
// the same order every time), then the CTA's threads are added in order.
template <typename TX, typename TG, int D, bool HALVES, int UNROLL>
__global__ void __launch_bounds__(kThreads)
qk_norm_rope_bwd_kernel(const BwdArgs<TX, TG> a) {
  constexpr int TPR = D / 8, RPW = 32 / TPR, kStep = UNROLL * RPW;
  __shared__ float red[kWarps * RPW][D];
  const int lane = threadIdx.x & 31, sub = lane % TPR, slot = lane / TPR, warp = threadIdx.x >> 5;
  const int steps_q = ceil_div(a.q.heads, kStep), steps = steps_q + ceil_div(a.k.heads, kStep);
  const int per = ceil_div(steps, (int)gridDim.y);
  const int s0 = blockIdx.y * per, s1 = min(steps, s0 + per);
  float dwq[8], dwk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dwq[e] = dwk[e] = 0.f;
  for (long long token = (long long)blockIdx.x * kWarps + warp; token < a.tokens;
       token += (long long)gridDim.x * kWarps) {
    const int b = (int)(token / a.N), n = (int)(token - (long long)b * a.N);
    Turn<D, HALVES> turn;
    float w[8];
    for (int st = s0; st < s1; ++st) {
      const bool is_k = st >= steps_q;
      const Side<TX>& side = is_k ? a.k : a.q;
      const TG* gy = is_k ? a.gk : a.gq;
      const int heads = side.heads, h0 = (is_k ? st - steps_q : st) * kStep + slot;
      Raw<TX> raw[UNROLL];
      Raw<TG> grad[UNROLL];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int h = min(h0 + u * RPW, heads - 1);
        fetch(side, b, n, h, a.N, sub, raw[u]);
        load8(gy + (((long long)b * heads + h) * a.N + n) * D + 8 * sub, grad[u]);
      }
      if (st == s0) turn.load(a.rope, b, n, sub, a.err);
      if (st == s0 || st == steps_q) load_weight(side.w, sub, w);
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int h = h0 + u * RPW;
        float x[8], g[8];
        values8(raw[u], x);
        values8(grad[u], g);
        turn.template apply<true>(g, sub);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
        const float r = rsqrtf(row_sum<TPR>(ss) * (1.0f / D) + a.eps);
        float m = 0.f;
        const bool in = h < heads;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] *= r;
          const float gh = in ? g[e] * x[e] : 0.f;
          if (is_k) dwk[e] += gh; else dwq[e] += gh;
          g[e] *= w[e];
          m = fmaf(g[e], x[e], m);
        }
        m = row_sum<TPR>(m) * (1.0f / D);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = r * fmaf(-x[e], m, g[e]);
        if (in) {
          TG* d = is_k ? a.dk + b * a.dkb + n * a.dkn + h * a.dkh : a.dq + b * a.dqb + n * a.dqn + h * a.dqh;
          store8(d + 8 * sub, x);
        }
      }
    }
  }
#pragma unroll
  for (int side = 0; side < 2; ++side) {
#pragma unroll
    for (int e = 0; e < 8; ++e) red[warp * RPW + slot][8 * sub + e] = side ? dwk[e] : dwq[e];
    __syncthreads();
    if (threadIdx.x < D) {
      float sum = 0.f;
#pragma unroll 4
      for (int i = 0; i < kWarps * RPW; ++i) sum += red[i][threadIdx.x];
      a.part[((long long)(blockIdx.y * gridDim.x + blockIdx.x) * 2 + side) * D + threadIdx.x] = sum;
    }
    __syncthreads();
  }
}

// dw [2][D] from the CTAs' shares: thread (column, part) adds every
// (blockDim / (2 D))-th share in order, then the parts are added in order.
__global__ void __launch_bounds__(1024)
weight_grad_kernel(const float* __restrict__ part, int ctas, int D, float* __restrict__ dwq,
                   float* __restrict__ dwk) {
  __shared__ float red[1024];
  const int cols = 2 * D, col = threadIdx.x % cols, p = threadIdx.x / cols, parts = blockDim.x / cols;
  float sum = 0.f;
#pragma unroll 4
  for (int i = p; i < ctas; i += parts) sum += part[(long long)i * cols + col];
  red[threadIdx.x] = sum;
  __syncthreads();
  if (p == 0) {
    for (int i = 1; i < parts; ++i) sum += red[i * cols + col];
    float* dw = col < D ? dwq : dwk;
    if (dw) dw[col % D] = sum;
  }
}

template <typename TIn, typename TOut, int D, bool HALVES, bool SAVE8>
cudaError_t fwd_t(const NormRopeFwd& f, cudaStream_t s) {
  constexpr int RPW = 32 / (D / 8);
  FwdArgs<TIn, TOut> a;
  a.q = {static_cast<const TIn*>(f.xq), f.xq_scale, f.qb, f.qn, f.qh, f.Hq, f.wq};
  a.k = {static_cast<const TIn*>(f.xk), f.xk_scale, f.kb, f.kn, f.kh, f.Hk, f.wk};
  a.yq = static_cast<TOut*>(f.q);
  a.yk = static_cast<TOut*>(f.k);
  a.cq = f.xq8; a.ck = f.xk8; a.sq = f.xq8_scale; a.sk = f.xk8_scale;
  a.N = f.N;
  a.tokens = (long long)f.B * f.N;
  a.eps = f.eps;
  a.rope = f.rope;
  a.err = f.err;
  const unsigned gx = (unsigned)((a.tokens + kWarps - 1) / kWarps);
  // Few tokens (single-token steps): one row per thread and step, and the
  // heads spread over CTAs, for latency; otherwise a warp takes its token's
  // heads four rows per thread at a time.
  if (a.tokens < 2048) {
    const int steps = ceil_div(f.Hq, RPW) + ceil_div(f.Hk, RPW);
    const int gy = std::max(1, std::min(steps, (int)(16384 / a.tokens)));
    qk_norm_rope_kernel<TIn, TOut, D, HALVES, SAVE8, 1><<<dim3(gx, gy), kThreads, 0, s>>>(a);
  } else {
    qk_norm_rope_kernel<TIn, TOut, D, HALVES, SAVE8, 4><<<dim3(gx, 1), kThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

template <typename TIn, typename TOut>
cudaError_t fwd_dispatch(const NormRopeFwd& f, cudaStream_t s) {
#define DSA_FWD(DD, HALVES)                                                   \
  return f.xq8 ? fwd_t<TIn, TOut, DD, HALVES, true>(f, s) : fwd_t<TIn, TOut, DD, HALVES, false>(f, s)
  if (f.D == 64) {
    if (f.halves) DSA_FWD(64, true);
    DSA_FWD(64, false);
  }
  if (f.halves) DSA_FWD(128, true);
  DSA_FWD(128, false);
#undef DSA_FWD
}

// From codes: nothing to save again.
template <typename TOut>
cudaError_t fwd_from8(const NormRopeFwd& f, cudaStream_t s) {
  if (f.D == 64)
    return f.halves ? fwd_t<int8_t, TOut, 64, true, false>(f, s) : fwd_t<int8_t, TOut, 64, false, false>(f, s);
  return f.halves ? fwd_t<int8_t, TOut, 128, true, false>(f, s) : fwd_t<int8_t, TOut, 128, false, false>(f, s);
}

struct BwdGrid { int x, y; };

// The persistent grid: at most kNormRopeBwdCtas CTAs, no more than the
// tokens (times the parts of the heads, where the tokens are few) can use.
BwdGrid bwd_grid(long long tokens, int Hq, int Hk) {
  const int gx = (int)std::min<long long>((tokens + kWarps - 1) / kWarps, kNormRopeBwdCtas);
  const int gy = std::max(1, std::min((Hq + 7) / 8 + (Hk + 7) / 8, kNormRopeBwdCtas / gx));
  return {gx, gy};
}

template <typename TX, typename TG, int D, bool HALVES>
cudaError_t bwd_t(const NormRopeBwd& f, cudaStream_t s) {
  BwdArgs<TX, TG> a;
  a.q = {static_cast<const TX*>(f.xq), f.xq_scale, f.qb, f.qn, f.qh, f.Hq, f.wq};
  a.k = {static_cast<const TX*>(f.xk), f.xk_scale, f.kb, f.kn, f.kh, f.Hk, f.wk};
  a.gq = static_cast<const TG*>(f.gq);
  a.gk = static_cast<const TG*>(f.gk);
  a.dq = static_cast<TG*>(f.dxq);
  a.dk = static_cast<TG*>(f.dxk);
  a.dqb = f.dqb; a.dqn = f.dqn; a.dqh = f.dqh;
  a.dkb = f.dkb; a.dkn = f.dkn; a.dkh = f.dkh;
  a.part = f.part;
  a.N = f.N;
  a.tokens = (long long)f.B * f.N;
  a.eps = f.eps;
  a.rope = f.rope;
  a.err = f.err;
  const BwdGrid g = bwd_grid(a.tokens, f.Hq, f.Hk);
  qk_norm_rope_bwd_kernel<TX, TG, D, HALVES, 2><<<dim3(g.x, g.y), kThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  weight_grad_kernel<<<1, 1024, 0, s>>>(f.part, g.x * g.y, D, f.dwq, f.dwk);
  return cudaGetLastError();
}

template <typename TX, typename TG>
cudaError_t bwd_dispatch(const NormRopeBwd& f, cudaStream_t s) {
  if (f.D == 64) return f.halves ? bwd_t<TX, TG, 64, true>(f, s) : bwd_t<TX, TG, 64, false>(f, s);
  return f.halves ? bwd_t<TX, TG, 128, true>(f, s) : bwd_t<TX, TG, 128, false>(f, s);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeFwd& f, cudaStream_t s) {
  if (f.xq_scale)
    return f.bf16 ? fwd_from8<__nv_bfloat16>(f, s) : fwd_from8<float>(f, s);
  return f.bf16 ? fwd_dispatch<__nv_bfloat16, __nv_bfloat16>(f, s) : fwd_dispatch<float, float>(f, s);
}

cudaError_t launch_qk_norm_rope_bwd(const NormRopeBwd& f, cudaStream_t s) {
  if (f.xq_scale)
    return f.bf16 ? bwd_dispatch<int8_t, __nv_bfloat16>(f, s) : bwd_dispatch<int8_t, float>(f, s);
  return f.bf16 ? bwd_dispatch<__nv_bfloat16, __nv_bfloat16>(f, s) : bwd_dispatch<float, float>(f, s);
}

}  // namespace dsa
