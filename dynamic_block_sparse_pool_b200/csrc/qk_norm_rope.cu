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
// Bound by memory (about 3 to 4 operations per byte), and where rows are held
// in 8 bits by instruction issue as well: every row is read once and written
// once, so the layout and the instruction count are left to choose.  x is
// token-major (strided: the fused projection's output is read in place), y
// is head-major, and the rotation depends on the token alone, so a warp
// keeps one token: it fetches the token's cosines and sines once (from small
// per-axis tables that stay in L1) and runs over the token's heads, D / 8
// threads of eight values per row.  Reads are whole token rows; writes are
// one row per head, next to those of the seven tokens of the CTA's other
// warps.  The loads that cover the latency of HBM: four rows per thread in
// registers (forward), asynchronous copies three steps ahead (backward, where
// the sums of dw need the registers).
//
// x may be 8-bit rows (codes and scales, rows8.cuh) in place of bf16 or fp32,
// and the forward can write those of x beside y, so a training step keeps a
// byte per value where it kept two and reads less in the backward.
//
// Measured, D = 128, bf16, counted bytes (each value once), L2 flushed between
// calls: 118,800 tokens, 24 + 24 heads: forward 469 us (6.2 TB/s), saving codes 646
// (5.6), from codes 424 (5.2), backward 697 (6.3), from codes 740 (4.9; 65 to 80 %
// of the issue slots are taken); back to back the forward that saves codes and the
// backward from them take 1,512 us together.  75,600 tokens, 40 + 40 heads: forward
// 506 us (6.1).  D = 64, 17,776 tokens, 48 + 48 heads: backward 120 us (5.5).
#include <algorithm>

#include "norm_rope.cuh"
#include "rows8.cuh"

namespace dsa {
namespace {

using namespace rows8;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// The turn of a thread's eight values, as y = x c + partner(x) s.  Neighbouring
// pairs: the partner is the other value of the pair (single operations: the
// packed ones would need a swapped copy of every pair, which costs what they
// save).  Halves: it is the same value of the thread D / 16 further on, and the
// signs are in s.
template <int D, bool HALVES>
struct Turn {
  Pair c[4], s[4];      // halves
  float c1[4], s1[4];   // neighbours

  // The token's angles from the tables.  A position below 0 does not turn;
  // one past its axis' table is reported and does not turn either.
  __device__ __forceinline__ void load(const RopeArgs& a, int b, int n, int sub, unsigned* err) {
    constexpr int kPairs = HALVES ? 8 : 4;
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
    float2 t[kPairs];
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
      t[m] = make_float2(1.f, 0.f);
      if (v >= 0 && i < pa) t[m] = __ldg(a.table + base + (long long)v * pa + i);
    }
    if (HALVES) {
      const float sign = sub < D / 16 ? -1.f : 1.f;  // first half: a cos - b sin
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        c[m] = pair(t[(2 * m) % kPairs].x, t[(2 * m + 1) % kPairs].x);
        s[m] = pair(sign * t[(2 * m) % kPairs].y, sign * t[(2 * m + 1) % kPairs].y);
      }
    } else {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        c1[m] = t[m].x;
        s1[m] = t[m].y;
      }
    }
  }
  // The opposite turn.
  __device__ __forceinline__ void reverse() {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      if (HALVES) s[m] = mul_f32x2(s[m], both(-1.f));
      else s1[m] = -s1[m];
    }
  }
  __device__ __forceinline__ void apply(Pair (&v)[4]) const {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      float x, y;
      unpack_f32x2(v[m], x, y);
      if (HALVES) {
        const Pair o = pair(__shfl_xor_sync(0xffffffffu, x, D / 16), __shfl_xor_sync(0xffffffffu, y, D / 16));
        v[m] = fma_f32x2(v[m], c[m], mul_f32x2(o, s[m]));
      } else {
        v[m] = pair(fmaf(x, c1[m], -(y * s1[m])), fmaf(y, c1[m], x * s1[m]));
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

__device__ __forceinline__ void load_weight(const float* w, int sub, Pair (&v)[4]) {
#pragma unroll
  for (int m = 0; m < 4; ++m)
    v[m] = w ? pair(__ldg(w + 8 * sub + 2 * m), __ldg(w + 8 * sub + 2 * m + 1)) : both(1.f);
}

template <typename TIn>
__device__ __forceinline__ void fetch(const TIn* p, const float*, long long, Raw<TIn>& r) {
  load8(p, r);
}
__device__ __forceinline__ void fetch(const int8_t* p, const float* scales, long long row, Raw<int8_t>& r) {
  load8(p, r);
  r.scale = __ldg(scales + row);
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
// A step is UNROLL * (32 / TPR) heads of q or of k.
template <typename TIn, typename TOut, int D, bool HALVES, bool SAVE8, int UNROLL>
__global__ void __launch_bounds__(kThreads, sizeof(TIn) == 4 ? 3 : 4)
qk_norm_rope_kernel(const FwdArgs<TIn, TOut> a) {
  constexpr int TPR = D / 8, RPW = 32 / TPR, kStep = UNROLL * RPW;
  const int lane = threadIdx.x & 31, sub = lane % TPR, slot = lane / TPR;
  const int token = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (token >= (int)a.tokens) return;
  const int b = token / a.N, n = token - b * a.N;
  const long long ystep = (long long)a.N * D;  // from head to head in y
  const int steps_q = ceil_div(a.q.heads, kStep), steps = steps_q + ceil_div(a.k.heads, kStep);
  const int per = ceil_div(steps, (int)gridDim.y);
  const int s0 = blockIdx.y * per, s1 = min(steps, s0 + per);
  Turn<D, HALVES> turn;
  Pair w[4];
  const TIn* px = nullptr;    // running pointers over the side's heads
  TOut* py = nullptr;
  for (int st = s0; st < s1; ++st) {
    const bool is_k = st >= steps_q;
    const Side<TIn>& side = is_k ? a.k : a.q;
    const int heads = side.heads, h0 = (is_k ? st - steps_q : st) * kStep + slot;
    if (st == s0 || st == steps_q) {
      px = side.x + b * side.b + n * side.n + h0 * side.h + 8 * sub;
      py = (is_k ? a.yk : a.yq) + ((long long)b * heads + h0) * ystep + (long long)n * D + 8 * sub;
    }
    Raw<TIn> raw[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      // (a lane past the heads reads its first row again)
      const int h = h0 + u * RPW < heads ? u * RPW : 0;
      fetch(px + (h0 < heads ? h : 0) * side.h - (h0 < heads ? 0 : (h0 - heads + 1) * side.h), side.xs,
            (long long)token * heads + min(h0 + h, heads - 1), raw[u]);
    }
    if (st == s0) turn.load(a.rope, b, n, sub, a.err);
    if (st == s0 || st == steps_q) load_weight(side.w, sub, w);
    float inv[UNROLL], save = 0.f;
    if constexpr (SAVE8) {
      uint32_t top[UNROLL];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) top[u] = row_top<TPR>(top_bits(raw[u]));
      save = scales8<TPR>(top, sub, inv);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int h = h0 + u * RPW;
      Pair v[4];
      values(raw[u], v);
      Pair ss = 0ull;
#pragma unroll
      for (int m = 0; m < 4; ++m) ss = fma_f32x2(v[m], v[m], ss);
      if constexpr (SAVE8) {
        if (h < heads) {
          const long long row = (long long)token * heads + h;
          *reinterpret_cast<uint2*>((is_k ? a.ck : a.cq) + row * D + 8 * sub) = encode8(v, inv[u]);
          if (sub == 2 * u) (is_k ? a.sk : a.sq)[row] = save;
        }
      }
      // (8-bit rows: v holds the codes, the row is scale * v)
      const float scale = scale_of(raw[u]);
      const Pair r = both(scale * rsqrtf(scale * scale * row_sum<TPR>(added(ss)) * (1.0f / D) + a.eps));
#pragma unroll
      for (int m = 0; m < 4; ++m) v[m] = mul_f32x2(mul_f32x2(v[m], r), w[m]);
      turn.apply(v);
      if (h < heads) store(py + u * RPW * ystep, v);
    }
    px += kStep * side.h;
    py += kStep * ystep;
  }
}

// One side of the backward.
template <typename TX, typename TG>
struct BwdSide {
  Side<TX> x;
  const TG* g;         // gradient of y, [B, heads, N, D]
  TG* d;               // gradient of x
  long long b, n, h;   // its strides, in elements
};

template <typename TX, typename TG>
struct BwdArgs {
  BwdSide<TX, TG> q, k;
  int parts_q;         // parts of q's heads; the other parts are k's
  int heads_per_part;
  float* part;         // [parts][gridDim.x][D]: the CTAs' shares of dwq, then of dwk
  int N;
  long long tokens;    // < 2^31 - 2^16, so a place past the last one fits too
  float eps;
  RopeArgs rope;
  unsigned* err;
};

// A thread's eight values into its slots, and back.
__device__ __forceinline__ void fetch_async(uint32_t slot, const __nv_bfloat16* p, const float*, int) {
  copy_async<16>(slot, p);
}
__device__ __forceinline__ void fetch_async(uint32_t slot, const float* p, const float*, int) {
  copy_async<16>(slot, p);
  copy_async<16>(slot + 16 * kThreads, p + 4);
}
// (the row's first thread brings in the scale for all of them)
__device__ __forceinline__ void fetch_async(uint32_t slot, const int8_t* p, const float* scale, int sub) {
  copy_async<8>(slot, p);
  if (sub == 0) copy_async<4>(slot + 8, scale);
}
__device__ __forceinline__ void read_slot(const uint4* slot, Raw<__nv_bfloat16>& r, int) { r.v = slot[0]; }
__device__ __forceinline__ void read_slot(const uint4* slot, Raw<float>& r, int) {
  r.v = slot[0];
  r.w = slot[kThreads];
}
// (the scale lies in the first thread's slot: it reads it and hands it on.  Read by
// all from that slot it takes a fence on either side, before and after, since the
// next copy into the slot is the first thread's: 2 % slower in bf16.)
__device__ __forceinline__ void read_slot(const uint4* slot, Raw<int8_t>& r, int sub) {
  r.v = *reinterpret_cast<const uint2*>(slot);
  r.scale = __shfl_sync(0xffffffffu, *reinterpret_cast<const float*>(reinterpret_cast<const uint32_t*>(slot) + 2),
                        (threadIdx.x & 31) - sub);
}

// Steps of the backward whose loads are in flight: enough bytes for HBM's
// latency with three CTAs on an SM (32 or 64 KB of shared memory each).
constexpr uint32_t kDepth = 4;
template <typename TX, typename TG>
constexpr int bwd_slots() { return Slots<TX>::kCount + Slots<TG>::kCount; }

// Grid: x = CTAs over the tokens, y = parts of q's, then of k's heads.  Warp g
// of a part takes tokens g, g + warps, ... (the grid does not depend on the
// data, so each thread sums dw over the same rows in the same order every
// time), then the CTA's threads are added in order.  A step is one row per
// thread; its loads go out kDepth - 1 steps ahead.
template <typename TX, typename TG, int D, bool HALVES>
__global__ void __launch_bounds__(kThreads, 3)
qk_norm_rope_bwd_kernel(const BwdArgs<TX, TG> a) {
  constexpr int TPR = D / 8, RPW = 32 / TPR, SX = Slots<TX>::kCount, SLOTS = bwd_slots<TX, TG>();
  extern __shared__ __align__(16) uint4 ring[];  // [kDepth][SLOTS][kThreads]
  __shared__ float red[kWarps * RPW][D];
  let_next_start();
  const int lane = threadIdx.x & 31, sub = lane % TPR, slot = lane / TPR, warp = threadIdx.x >> 5;
  const bool is_k = blockIdx.y >= a.parts_q;
  const BwdSide<TX, TG>& side = is_k ? a.k : a.q;
  const int heads = side.x.heads;
  const int ha = (is_k ? blockIdx.y - a.parts_q : blockIdx.y) * a.heads_per_part, hz = min(heads, ha + a.heads_per_part);
  const int stride = gridDim.x * kWarps, tokens = (int)a.tokens;
  const long long gstep = (long long)a.N * D;  // from head to head in g
  Pair w[4], dw[4];
  load_weight(side.x.w, sub, w);
#pragma unroll
  for (int m = 0; m < 4; ++m) dw[m] = 0ull;

  // Where the next loads come from: a token and running pointers over its
  // heads (64-bit products and divisions only where the token changes).
  int ft = blockIdx.x * kWarps + warp, fh = 0;
  const TX* px = nullptr;
  const TG* pg = nullptr;
  const float* ps = nullptr;
  auto aim = [&]() {
    const int b = ft / a.N, n = ft - b * a.N;
    fh = ha + slot;
    px = side.x.x + b * side.x.b + n * side.x.n + fh * side.x.h + 8 * sub;
    pg = side.g + ((long long)b * heads + fh) * gstep + (long long)n * D + 8 * sub;
    if (sizeof(TX) == 1) ps = side.x.xs + (long long)ft * heads + fh;
  };
  const uint32_t ring0 = shared_at(ring + threadIdx.x);
  uint32_t fs = 0, rs = 0;  // steps fetched and taken so far
  if (ft < tokens) aim();
  auto fetch_step = [&]() {
    if (ft < tokens) {
      if (fh < hz) {  // (a lane past the heads leaves its slots as they are)
        const uint32_t to = ring0 + (fs % kDepth) * (SLOTS * kThreads * 16);
        fetch_async(to, px, ps, sub);
        fetch_async(to + SX * kThreads * 16, pg, nullptr, sub);
      }
      ++fs;
      fh += RPW;
      px += RPW * side.x.h;
      pg += RPW * gstep;
      ps += RPW;
      if (fh - slot >= hz) {
        ft += stride;
        if (ft < tokens) aim();
      }
    }
    copy_commit();
  };
#pragma unroll
  for (uint32_t i = 0; i < kDepth - 1; ++i) fetch_step();

  for (int token = blockIdx.x * kWarps + warp; token < tokens; token += stride) {
    const int b = token / a.N, n = token - b * a.N;
    TG* dx = side.d + b * side.b + n * side.n + (ha + slot) * side.h + 8 * sub;
    Turn<D, HALVES> turn;
    turn.load(a.rope, b, n, sub, a.err);
    turn.reverse();
    for (int h = ha + slot; h - slot < hz; h += RPW) {
      fetch_step();
      copy_wait<kDepth - 1>();
      const uint4* from = ring + (rs % kDepth) * (SLOTS * kThreads) + threadIdx.x;
      ++rs;
      Raw<TX> raw;
      Raw<TG> grad;
      read_slot(from, raw, sub);
      read_slot(from + SX * kThreads, grad, sub);
      const bool in = h < hz;
      Pair x[4], g[4], ss = 0ull, dot = 0ull;
      values(raw, x);
      values(grad, g);
      turn.apply(g);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        ss = fma_f32x2(x[m], x[m], ss);
        dot = fma_f32x2(mul_f32x2(g[m], w[m]), x[m], dot);
      }
      // both sums in one round of shuffles; mean(g w h) = r mean(g w x)
      float s1 = added(ss), s2 = added(dot);
#pragma unroll
      for (int o = 1; o < TPR; o <<= 1) {
        s1 += __shfl_xor_sync(0xffffffffu, s1, o);
        s2 += __shfl_xor_sync(0xffffffffu, s2, o);
      }
      // (8-bit rows: x holds the codes, the row is scale * x)
      const float scale = scale_of(raw);
      const float r = rsqrtf(scale * scale * s1 * (1.0f / D) + a.eps);
      const Pair r2 = both(r), h1 = both(scale * r), m2 = both(-r * r * (scale * s2 * (1.0f / D)));
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const Pair h2 = mul_f32x2(x[m], h1);
        const Pair gh = fma_f32x2(g[m], h2, dw[m]);
        if (in) dw[m] = gh;  // a lane past the heads adds nothing
        x[m] = fma_f32x2(mul_f32x2(g[m], w[m]), r2, mul_f32x2(h2, m2));
      }
      if (in) store(dx, x);
      dx += RPW * side.h;
    }
  }
  copy_wait<0>();
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    float lo, hi;
    unpack_f32x2(dw[m], lo, hi);
    red[warp * RPW + slot][8 * sub + 2 * m] = lo;
    red[warp * RPW + slot][8 * sub + 2 * m + 1] = hi;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float sum = 0.f;
#pragma unroll 4
    for (int i = 0; i < kWarps * RPW; ++i) sum += red[i][threadIdx.x];
    a.part[((long long)blockIdx.y * gridDim.x + blockIdx.x) * D + threadIdx.x] = sum;
  }
}

// dwq (block 0) or dwk (block 1) from the CTAs' shares: thread (column, p)
// adds every (1024 / D)-th share in order, then the p sums are added in order.
__global__ void __launch_bounds__(1024)
weight_grad_kernel(const float* __restrict__ part, int ctas_q, int ctas_k, int D, float* __restrict__ dwq,
                   float* __restrict__ dwk) {
  __shared__ float red[1024];
  wait_for_previous();
  const float* p0 = blockIdx.x ? part + (long long)ctas_q * D : part;
  const int ctas = blockIdx.x ? ctas_k : ctas_q, col = threadIdx.x % D, p = threadIdx.x / D, parts = 1024 / D;
  float sum = 0.f;
#pragma unroll 4
  for (int i = p; i < ctas; i += parts) sum += p0[(long long)i * D + col];
  red[threadIdx.x] = sum;
  __syncthreads();
  if (p == 0) {
    for (int i = 1; i < parts; ++i) sum += red[i * D + col];
    float* dw = blockIdx.x ? dwk : dwq;
    if (dw) dw[col] = sum;
  }
}

// One axis' table in 64 bits: grid x over positions, one thread per pair.
__global__ void rope_table_kernel(int positions, int pairs, double theta, float2* __restrict__ table) {
  const int i = threadIdx.x;
  const double f = pow(theta, -(double)i / pairs);
  for (int p = blockIdx.x * blockDim.y + threadIdx.y; p < positions; p += gridDim.x * blockDim.y) {
    double s, c;
    sincos(p * f, &s, &c);
    table[(long long)p * pairs + i] = make_float2((float)c, (float)s);
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

// Heads per part and CTAs over the tokens: parts as long as the smaller side,
// shorter ones while the tokens leave SMs idle, and at most kNormRopeBwdCtas
// CTAs in all: as many as run at once (four a step apart cost a quarter of the
// rate: registers spilled and a second wave).
struct BwdGrid {
  int heads, parts_q, parts_k, x;
  BwdGrid(long long tokens, int Hq, int Hk, int step) {
    const long long rows = (tokens + kWarps - 1) / kWarps;
    heads = std::max(step, std::min(Hq, Hk));
    while (heads > step && rows * (ceil_div(Hq, heads) + ceil_div(Hk, heads)) < kNormRopeBwdCtas)
      heads = std::max(step, heads / 2);
    // (no more parts than CTAs)
    while (ceil_div(Hq, heads) + ceil_div(Hk, heads) > kNormRopeBwdCtas) heads *= 2;
    parts_q = ceil_div(Hq, heads);
    parts_k = ceil_div(Hk, heads);
    x = (int)std::min<long long>(rows, std::max(1, kNormRopeBwdCtas / (parts_q + parts_k)));
  }
};

template <typename TX, typename TG, int D, bool HALVES>
cudaError_t bwd_t(const NormRopeBwd& f, cudaStream_t s) {
  BwdArgs<TX, TG> a;
  a.q = {{static_cast<const TX*>(f.xq), f.xq_scale, f.qb, f.qn, f.qh, f.Hq, f.wq},
         static_cast<const TG*>(f.gq), static_cast<TG*>(f.dxq), f.dqb, f.dqn, f.dqh};
  a.k = {{static_cast<const TX*>(f.xk), f.xk_scale, f.kb, f.kn, f.kh, f.Hk, f.wk},
         static_cast<const TG*>(f.gk), static_cast<TG*>(f.dxk), f.dkb, f.dkn, f.dkh};
  a.part = f.part;
  a.N = f.N;
  a.tokens = (long long)f.B * f.N;
  a.eps = f.eps;
  a.rope = f.rope;
  a.err = f.err;
  const BwdGrid g(a.tokens, f.Hq, f.Hk, 32 / (D / 8));
  a.parts_q = g.parts_q;
  a.heads_per_part = g.heads;
  const int smem = (int)kDepth * bwd_slots<TX, TG>() * kThreads * 16;
  cudaError_t e = cudaFuncSetAttribute(qk_norm_rope_bwd_kernel<TX, TG, D, HALVES>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  qk_norm_rope_bwd_kernel<TX, TG, D, HALVES><<<dim3(g.x, g.parts_q + g.parts_k), kThreads, smem, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_next(weight_grad_kernel, 2, 1024, 0, s, f.part, g.x * g.parts_q, g.x * g.parts_k, D, f.dwq, f.dwk);
}

template <typename TX, typename TG>
cudaError_t bwd_dispatch(const NormRopeBwd& f, cudaStream_t s) {
  if (f.D == 64) return f.halves ? bwd_t<TX, TG, 64, true>(f, s) : bwd_t<TX, TG, 64, false>(f, s);
  return f.halves ? bwd_t<TX, TG, 128, true>(f, s) : bwd_t<TX, TG, 128, false>(f, s);
}

}  // namespace

cudaError_t launch_rope_table(int positions, int pairs, double theta, float2* table, cudaStream_t s) {
  const dim3 block((unsigned)pairs, (unsigned)std::max(1, 128 / pairs));
  rope_table_kernel<<<(unsigned)std::min(ceil_div(positions, (int)block.y), 2048), block, 0, s>>>(positions, pairs, theta,
                                                                                              table);
  return cudaGetLastError();
}

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
