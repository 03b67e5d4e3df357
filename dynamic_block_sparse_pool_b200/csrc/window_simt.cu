// Window attention in exact fp32 on CUDA cores: forward and backward.
//
// Serves fp32 inputs, where a tf32 or bf16 product would miss fp32 results.
// One CTA (256 threads) per tile of 64 queries (forward, dQ) or 64 keys (dK,
// dV); the tiles of the other side stream through shared memory.  Bound by
// the FMA pipe: thread (ty, tx) of 16 x 16 owns rows ty + 16 a and columns tx
// + 16 b (a, b < 4) of every 64 x 64 product, read from shared memory as
// float4 along the summed dimension, 8 loads for 64 FMAs.  Rows are padded to
// D + 4 (64 + 4) floats, so the 16 columns of a load fall in different banks.
//
// Formulas as in window_fwd_sm100.cu and window_bwd_sm100.cu.  dK and dV of a
// key head are summed over its query heads and queries in a fixed order, no
// atomics: equal bits from run to run.  A tile pair takes about 5 us, so where
// the tiles of one side are few, or one of them (a sink's) sees far more than
// the others, a gradient tile's pairs are cut into chunks (SimtChunks), one CTA
// each, whose partial sums a last kernel adds in order.  All gradients come out
// of one launch, so dQ's CTAs fill in where dK's and dV's run out (1,003 tokens,
// 4 heads on 2, D = 64: 101 -> 81 us with the row terms and the join; 2 x 4,000
// tokens, 8 heads on 4, D = 128, causal over 1,000: 3.56 -> 3.28 ms, 22 TFLOP/s).
// Forward of the latter 0.98 ms, 29 TFLOP/s.  Shared-memory reads are at 62 % of
// their peak rate and FMA at 50 %, with 8 warps on an SM (D = 128).
#include <algorithm>

#include "window_attn.cuh"

namespace dsa {
namespace {

constexpr int T = 64;        // queries and keys of a tile
constexpr int SP = T + 4;    // padded row of a 64 x 64 tile
constexpr int kThreads = 256;

template <int D>
constexpr int padded() { return D + 4; }

// Rows r0 .. r0 + 63 of a [rows, D] head into shared memory; rows past `end`
// read as zeros.
template <int D>
__device__ __forceinline__ void stage(float* dst, const float* __restrict__ src, int r0, int end) {
  constexpr int V = D / 4;
  for (int i = threadIdx.x; i < T * V; i += kThreads) {
    const int r = i / V, c = 4 * (i - r * V);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < end) v = *reinterpret_cast<const float4*>(src + (size_t)(r0 + r) * D + c);
    *reinterpret_cast<float4*>(dst + r * padded<D>() + c) = v;
  }
}

// acc[a][b] += A[ty + 16 a] . B[tx + 16 b] over D columns
template <int D>
__device__ __forceinline__ void product_nt(float (&acc)[4][4], const float* A, const float* B, int ty, int tx) {
  constexpr int P = padded<D>();
#pragma unroll 4
  for (int d = 0; d < D; d += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) x[a] = *reinterpret_cast<const float4*>(A + (ty + 16 * a) * P + d);
#pragma unroll
    for (int b = 0; b < 4; ++b) y[b] = *reinterpret_cast<const float4*>(B + (tx + 16 * b) * P + d);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        acc[a][b] = fmaf(x[a].x, y[b].x, acc[a][b]);
        acc[a][b] = fmaf(x[a].y, y[b].y, acc[a][b]);
        acc[a][b] = fmaf(x[a].z, y[b].z, acc[a][b]);
        acc[a][b] = fmaf(x[a].w, y[b].w, acc[a][b]);
      }
  }
}

// acc[a][4 g + u] += sum over k of W[ty + 16 a][k] B[k][64 g + 4 tx + u]
template <int D>
__device__ __forceinline__ void product_nn(float (&acc)[4][D / 16], const float* W, const float* B, int ty, int tx) {
  constexpr int P = padded<D>();
#pragma unroll 2
  for (int k = 0; k < T; k += 4) {
    float w[4][4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const float4 v = *reinterpret_cast<const float4*>(W + (ty + 16 * a) * SP + k);
      w[a][0] = v.x; w[a][1] = v.y; w[a][2] = v.z; w[a][3] = v.w;
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int g = 0; g < D / 64; ++g) {
        const float4 y = *reinterpret_cast<const float4*>(B + (k + kk) * P + 64 * g + 4 * tx);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          acc[a][4 * g] = fmaf(w[a][kk], y.x, acc[a][4 * g]);
          acc[a][4 * g + 1] = fmaf(w[a][kk], y.y, acc[a][4 * g + 1]);
          acc[a][4 * g + 2] = fmaf(w[a][kk], y.z, acc[a][4 * g + 2]);
          acc[a][4 * g + 3] = fmaf(w[a][kk], y.w, acc[a][4 * g + 3]);
        }
      }
  }
}

template <int D>
__device__ __forceinline__ void store_rows(float* dst, const float (&acc)[4][D / 16], int r0, int end, float (&mul)[4],
                                           int ty, int tx) {
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int r = r0 + ty + 16 * a;
    if (r < end)
#pragma unroll
      for (int g = 0; g < D / 64; ++g)
        *reinterpret_cast<float4*>(dst + (size_t)r * D + 64 * g + 4 * tx) =
            make_float4(acc[a][4 * g] * mul[a], acc[a][4 * g + 1] * mul[a], acc[a][4 * g + 2] * mul[a],
                        acc[a][4 * g + 3] * mul[a]);
  }
}

// Is key u visible to the query at position t?
__device__ __forceinline__ bool sees(const Window& w, int t, int u) {
  return u < w.Nk && u <= t + w.right && (u < w.sink || u >= t - w.left);
}

// sum / max over the 16 threads (tx) of a row
__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float max16(float v) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
window_fwd_simt_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                       const Window w, int group, float scale, float* __restrict__ out, float* __restrict__ lse) {
  constexpr int P = padded<D>();
  extern __shared__ __align__(16) float sm[];
  float* Q = sm;
  float* KV = Q + T * P;   // K, then V of the same tile
  float* W = KV + T * P;   // weights
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int tiles = ceil_div(w.Nq, T), bh = blockIdx.x / tiles, q0 = (blockIdx.x - bh * tiles) * T;
  const int q1 = min(q0 + T, w.Nq);
  const size_t qh = (size_t)bh * w.Nq * D, kh = (size_t)(bh / group) * w.Nk * D;
  stage<D>(Q, q + qh, q0, w.Nq);
  float o[4][D / 16], m[4], l[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    m[a] = -INFINITY;
    l[a] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) o[a][c] = 0.f;
  }
  const KeyTiles<T> kt = KeyTiles<T>::of(w, q0, q1);
  for (int e = 0; e < kt.count(); ++e) {
    const int k0 = kt.tile(e) * T;
    __syncthreads();  // the previous tile's V and weights are consumed
    stage<D>(KV, k + kh, k0, w.Nk);
    __syncthreads();
    float s[4][4] = {};
    product_nt<D>(s, Q, KV, ty, tx);
    const bool whole = all_visible(w, q0, q1, k0, k0 + T);
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int t = w.off + q0 + ty + 16 * a;
      float top = -INFINITY;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        s[a][b] = whole || sees(w, t, k0 + tx + 16 * b) ? s[a][b] * scale : -INFINITY;
        top = fmaxf(top, s[a][b]);
      }
      const float mn = fmaxf(m[a], max16(top));
      // a row with no visible key so far keeps m = -inf; 0 in its place makes its weights 0
      const float mu = mn == -INFINITY ? 0.f : mn;
      const float alpha = expf(m[a] - mu);
      float sum = 0.f;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float x = expf(s[a][b] - mu);
        W[(ty + 16 * a) * SP + tx + 16 * b] = x;
        sum += x;
      }
      l[a] = l[a] * alpha + sum16(sum);
      m[a] = mn;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[a][c] *= alpha;
    }
    __syncthreads();  // K is consumed, the weights are written
    stage<D>(KV, v + kh, k0, w.Nk);
    __syncthreads();
    product_nn<D>(o, W, KV, ty, tx);
  }
  float inv[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) inv[a] = l[a] == 0.f ? 0.f : 1.f / l[a];
  store_rows<D>(out + qh, o, q0, q1, inv, ty, tx);
  if (lse && tx == 0)
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int r = q0 + ty + 16 * a;
      if (r < q1) lse[(size_t)bh * w.Nq + r] = l[a] == 0.f ? -INFINITY : m[a] + logf(l[a]);
    }
}

// P and dS of a 64 x 64 tile; hidden pairs, and rows without keys (lse =
// -inf), have both 0.  (A row that met a NaN has lse = NaN, which is not
// without keys: its P and dS are NaN.)
__device__ __forceinline__ void weights(const float (&s)[4][4], const float (&dp)[4][4], float (&p)[4][4],
                                        float (&ds)[4][4], const Window& w, int q0, int k0, bool whole, float scale,
                                        const float* lse, const float* delta, int ty, int tx) {
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int r = ty + 16 * a;
    const float ls = lse[r], de = delta[r];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const bool in = whole || sees(w, w.off + q0 + r, k0 + tx + 16 * b);
      p[a][b] = in && ls != -INFINITY ? expf(fmaf(scale, s[a][b], -ls)) : 0.f;
      ds[a][b] = in && ls != -INFINITY ? p[a][b] * (dp[a][b] - de) : 0.f;
    }
  }
}

__device__ __forceinline__ void stage_vec(float* dst, const float* src, int r0, int end, float pad) {
  if (threadIdx.x < T) dst[threadIdx.x] = r0 + threadIdx.x < end ? src[r0 + threadIdx.x] : pad;
}

struct BwdSimt {
  const float *q, *k, *v, *dout, *lse, *delta;
  Window w;
  int heads_q, heads_k, group;  // B H, B Hk, H / Hk
  float scale;
  SimtChunks cut;
  float *dq, *dk, *dv;
  // shares [slot][T][D]: dQ's, and dK's and dV's of the tiles with sinks and of the others
  float *share_q, *share_k[2], *share_v[2];
  unsigned ctas_k;              // CTAs of dK and dV; the others are dQ's
};

// A chunk of a tile of a gradient: the first chunks of all tiles come first, then
// layer by layer the further ones of the tiles that have them.
struct Place {
  int head, tile, y;
  template <int N>
  __device__ __forceinline__ Place(unsigned i, int heads, int tiles, const SimtCut (&cut)[N]) : y(0) {
    unsigned per = (unsigned)heads * tiles, run = tiles;
    int first = 0;
    if (i >= per) {
      i -= per;
      for (int c = 0; c < N; ++c) {
        run = cut[c].tiles();
        per = (unsigned)heads * run;
        first = cut[c].from;
        const unsigned n = per * (cut[c].parts - 1);
        if (i < n) break;
        i -= n;
      }
      y = 1 + (int)(i / per);
      i %= per;
    }
    head = (int)(i / run);
    tile = first + (int)(i - head * run);
  }
  template <int N>
  static unsigned count(int heads, int tiles, const SimtCut (&cut)[N]) {
    unsigned n = (unsigned)heads * tiles;
    for (int c = 0; c < N; ++c) n += (unsigned)heads * cut[c].tiles() * (cut[c].parts - 1);
    return n;
  }
};

// dQ of a query tile
template <int D>
__device__ __forceinline__ void dq_tile(const BwdSimt& a, unsigned i) {
  const float* __restrict__ q = a.q;
  const float* __restrict__ k = a.k;
  const float* __restrict__ v = a.v;
  const float* __restrict__ dout = a.dout;
  const Window w = a.w;
  const float scale = a.scale;
  constexpr int P = padded<D>();
  extern __shared__ __align__(16) float sm[];
  float *Q = sm, *O = Q + T * P, *K = O + T * P, *V = K + T * P, *W = V + T * P, *ls = W + T * SP, *de = ls + T;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const SimtCut cuts[1] = {a.cut.q};
  const Place at(i, a.heads_q, ceil_div(w.Nq, T), cuts);
  const int bh = at.head, q0 = at.tile * T, q1 = min(q0 + T, w.Nq);
  const size_t qh = (size_t)bh * w.Nq * D, kh = (size_t)(bh / a.group) * w.Nk * D;
  const KeyTiles<T> kt = KeyTiles<T>::of(w, q0, q1);
  const int e0 = at.y * cuts[0].chunk, e1 = min(kt.count(), e0 + cuts[0].chunk);
  if (at.y > 0 && e0 >= e1) return;  // (chunk 0 writes its zeros)
  stage<D>(Q, q + qh, q0, w.Nq);
  stage<D>(O, dout + qh, q0, w.Nq);
  stage_vec(ls, a.lse + (size_t)bh * w.Nq, q0, w.Nq, -INFINITY);
  stage_vec(de, a.delta + (size_t)bh * w.Nq, q0, w.Nq, 0.f);
  float acc[4][D / 16] = {};
  for (int e = e0; e < e1; ++e) {
    const int k0 = kt.tile(e) * T;
    __syncthreads();
    stage<D>(K, k + kh, k0, w.Nk);
    stage<D>(V, v + kh, k0, w.Nk);
    __syncthreads();
    float s[4][4] = {}, dp[4][4] = {}, p[4][4], ds[4][4];
    product_nt<D>(s, Q, K, ty, tx);
    product_nt<D>(dp, O, V, ty, tx);
    weights(s, dp, p, ds, w, q0, k0, all_visible(w, q0, q1, k0, k0 + T), scale, ls, de, ty, tx);
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int b = 0; b < 4; ++b) W[(ty + 16 * c) * SP + tx + 16 * b] = ds[c][b];
    __syncthreads();
    product_nn<D>(acc, W, K, ty, tx);
  }
  float mul[4] = {scale, scale, scale, scale};
  if (cuts[0].shared(at.tile))
    store_rows<D>(a.share_q + cuts[0].slot(bh, at.tile, at.y) * (T * D), acc, 0, q1 - q0, mul, ty, tx);
  else
    store_rows<D>(a.dq + qh, acc, q0, q1, mul, ty, tx);
}

// dK and dV of a key tile, over the query heads of its key head
template <int D>
__device__ __forceinline__ void dkdv_tile(const BwdSimt& a, unsigned i) {
  const float* __restrict__ q = a.q;
  const float* __restrict__ dout = a.dout;
  const Window w = a.w;
  const int group = a.group;
  const float scale = a.scale;
  constexpr int P = padded<D>();
  extern __shared__ __align__(16) float sm[];
  float *K = sm, *V = K + T * P, *Q = V + T * P, *O = Q + T * P, *W = O + T * P, *ls = W + T * SP, *de = ls + T;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const Place at(i, a.heads_k, ceil_div(w.Nk, T), a.cut.k);
  const int kind = at.tile >= a.cut.sink_tiles;
  const SimtCut cut = a.cut.k[kind];
  const int kv = at.head, k0 = at.tile * T, k1 = min(k0 + T, w.Nk);
  const size_t kh = (size_t)kv * w.Nk * D;
  const QueryRun run = QueryRun::of(w, k0, k1);
  const int i0 = run.q0 / T, per = run.tiles<T>(), n = per * group;  // query tiles per head, head after head
  const int e0 = at.y * cut.chunk, e1 = min(n, e0 + cut.chunk);
  if (at.y > 0 && e0 >= e1) return;  // (chunk 0 writes its zeros)
  stage<D>(K, a.k + kh, k0, w.Nk);
  stage<D>(V, a.v + kh, k0, w.Nk);
  float ak[4][D / 16] = {}, av[4][D / 16] = {};
  for (int e = e0; e < e1; ++e) {
    const int h = e / per, q0 = (i0 + e - h * per) * T;
    const size_t bh = (size_t)kv * group + h, qh = bh * w.Nq * D;
    __syncthreads();
    stage<D>(Q, q + qh, q0, w.Nq);
    stage<D>(O, dout + qh, q0, w.Nq);
    stage_vec(ls, a.lse + bh * w.Nq, q0, w.Nq, -INFINITY);
    stage_vec(de, a.delta + bh * w.Nq, q0, w.Nq, 0.f);
    __syncthreads();
    float s[4][4] = {}, dp[4][4] = {}, p[4][4], ds[4][4];
    product_nt<D>(s, Q, K, ty, tx);
    product_nt<D>(dp, O, V, ty, tx);
    weights(s, dp, p, ds, w, q0, k0, all_visible(w, q0, min(q0 + T, w.Nq), k0, k0 + T), scale, ls, de, ty, tx);
    // transposed into shared memory: row = key
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int b = 0; b < 4; ++b) W[(tx + 16 * b) * SP + ty + 16 * c] = p[c][b];
    __syncthreads();
    product_nn<D>(av, W, O, ty, tx);
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int b = 0; b < 4; ++b) W[(tx + 16 * b) * SP + ty + 16 * c] = ds[c][b];
    __syncthreads();
    product_nn<D>(ak, W, Q, ty, tx);
  }
  float one[4] = {1.f, 1.f, 1.f, 1.f}, mul[4] = {scale, scale, scale, scale};
  if (cut.shared(at.tile)) {
    const size_t share = cut.slot(kv, at.tile, at.y) * (T * D);
    store_rows<D>(a.share_v[kind] + share, av, 0, k1 - k0, one, ty, tx);
    store_rows<D>(a.share_k[kind] + share, ak, 0, k1 - k0, mul, ty, tx);
  } else {
    store_rows<D>(a.dv + kh, av, k0, k1, one, ty, tx);
    store_rows<D>(a.dk + kh, ak, k0, k1, mul, ty, tx);
  }
}

// All gradients: dK's and dV's CTAs, then dQ's, which fill in behind them.
template <int D>
__global__ void __launch_bounds__(kThreads, D == 64 ? 2 : 1)
window_bwd_simt_kernel(const BwdSimt a) {
  let_next_start();
  wait_for_previous();
  if (blockIdx.x < a.ctas_k)
    dkdv_tile<D>(a, blockIdx.x);
  else
    dq_tile<D>(a, blockIdx.x - a.ctas_k);
}

// Sums the shares of four columns of a row, i-th of all rows of a gradient's tiles
// that have shares (a tile as many as it has chunks, at least one).
template <int D, bool KEYS>
__device__ __forceinline__ void join(const BwdSimt& a, const SimtCut& cut, const float* __restrict__ shares,
                                     long long i, float* __restrict__ out) {
  constexpr int V = D / 4;
  const Window w = a.w;
  const long long row = i / V, t = row / T;
  const int head = (int)(t / cut.tiles()), tile = cut.from + (int)(t - (long long)head * cut.tiles());
  const int r = (int)(row - t * T), N = KEYS ? w.Nk : w.Nq, x0 = tile * T, x1 = min(x0 + T, N);
  if (x0 + r >= x1) return;
  const int n = KEYS ? QueryRun::of(w, x0, x1).tiles<T>() * a.group : KeyTiles<T>::of(w, x0, x1).count();
  const int chunks = max(1, ceil_div(n, cut.chunk));
  const float4* p = reinterpret_cast<const float4*>(shares + (cut.slot(head, tile, 0) * T + r) * D) + i % V;
  float4 s = *p;
#pragma unroll 4
  for (int c = 1; c < chunks; ++c) {
    p += T * V;
    const float4 x = *p;
    s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
  }
  reinterpret_cast<float4*>(out + ((size_t)head * N + x0 + r) * D)[i % V] = s;
}

// All gradients that have shares, one after another.
template <int D>
__global__ void __launch_bounds__(kThreads)
window_join_simt_kernel(const BwdSimt a) {
  wait_for_previous();
  constexpr int V = D / 4;
  long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    const SimtCut& cut = a.cut.k[kind];
    const long long n = (long long)a.heads_k * cut.tiles() * (T * V);
    if (i < n) return join<D, true>(a, cut, a.share_k[kind], i, a.dk);
    if ((i -= n) < n) return join<D, true>(a, cut, a.share_v[kind], i, a.dv);
    i -= n;
  }
  if (i < (long long)a.heads_q * a.cut.q.tiles() * (T * V)) join<D, false>(a, a.cut.q, a.share_q, i, a.dq);
}

template <int D>
cudaError_t fwd_d(const WindowAttn& a, cudaStream_t s) {
  const size_t smem = (2 * T * padded<D>() + T * SP) * sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(window_fwd_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  window_fwd_simt_kernel<D><<<a.B * a.H * ceil_div(a.w.Nq, T), kThreads, smem, s>>>(
      static_cast<const float*>(a.q), static_cast<const float*>(a.k), static_cast<const float*>(a.v), a.w, a.H / a.Hk,
      a.scale, static_cast<float*>(a.out), a.lse);
  return cudaGetLastError();
}

template <int D>
cudaError_t bwd_d(const WindowAttn& a, cudaStream_t s) {
  const size_t smem = (4 * T * padded<D>() + T * SP + 2 * T) * sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(window_bwd_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  BwdSimt p;
  p.q = static_cast<const float*>(a.q);
  p.k = static_cast<const float*>(a.k);
  p.v = static_cast<const float*>(a.v);
  p.dout = static_cast<const float*>(a.dout);
  p.lse = a.lse;
  p.delta = a.delta;
  p.w = a.w;
  p.heads_q = a.B * a.H;
  p.heads_k = a.B * a.Hk;
  p.group = a.H / a.Hk;
  p.scale = a.scale;
  p.cut = simt_chunks(a.B, a.H, a.Hk, a.w);
  p.dq = static_cast<float*>(a.dq);
  p.dk = static_cast<float*>(a.dk);
  p.dv = static_cast<float*>(a.dv);
  long long rows = 0;  // to be joined
  float* at = a.shares;
  auto room = [&](const SimtCut& c, int heads) {
    float* here = at;
    at += c.slots(heads) * (T * D);
    rows += (long long)heads * c.tiles() * T;
    return here;
  };
  p.share_q = room(p.cut.q, p.heads_q);
  for (int kind = 0; kind < 2; ++kind) {
    p.share_k[kind] = room(p.cut.k[kind], p.heads_k);
    p.share_v[kind] = room(p.cut.k[kind], p.heads_k);
  }
  const SimtCut cut_q[1] = {p.cut.q};
  p.ctas_k = Place::count(p.heads_k, ceil_div(a.w.Nk, T), p.cut.k);
  const unsigned ctas_q = Place::count(p.heads_q, ceil_div(a.w.Nq, T), cut_q);
  e = launch_next(window_bwd_simt_kernel<D>, p.ctas_k + ctas_q, kThreads, smem, s, p);
  if (e != cudaSuccess || rows == 0) return e;
  return launch_next(window_join_simt_kernel<D>, (unsigned)((rows * (D / 4) + kThreads - 1) / kThreads), kThreads, 0, s,
                     p);
}

}  // namespace

// The chunks of tile pairs: as long as a third of an SM's share of all pairs
// (half: 3 % slower, a quarter: the same where pairs are many, 6 % slower where they are
// few); one chunk where the longest tile is at most half as long again.  Key tiles
// with sinks, which far more queries see, are judged apart from the others, and
// only tiles with more than one chunk have shares: with shares for every tile of a
// gradient, 100,000 tokens, one head, D = 128, causal over 1,000 with four sinks took
// 2.56 GB of workspace for 0.10 GB of gradients (now 2 MB).
SimtChunks simt_chunks(int B, int H, int Hk, const Window& w) {
  auto cut = [](long long share, int t0, int t1, auto count) {
    int longest = 1;
    for (int t = t0; t < t1; ++t) longest = std::max(longest, count(t));
    SimtCut c = {longest, 1, t0, t0};
    if (2ll * longest > 3 * share) {
      c.chunk = (int)share;
      c.parts = ceil_div(longest, c.chunk);
      while (count(c.from) <= c.chunk) ++c.from;  // (the longest tile stops both)
      for (c.to = t1; count(c.to - 1) <= c.chunk;) --c.to;
    }
    return c;
  };
  auto share = [](long long heads, int tiles, auto count) {
    long long all = 0;
    for (int t = 0; t < tiles; ++t) all += count(t);
    return std::max(1ll, (all * heads + 443) / 444);
  };
  const int group = H / Hk, tq = ceil_div(w.Nq, T), tk = ceil_div(w.Nk, T);
  auto keys = [&](int t) { return KeyTiles<T>::of(w, t * T, std::min((t + 1) * T, w.Nq)).count(); };
  auto queries = [&](int t) { return QueryRun::of(w, t * T, std::min((t + 1) * T, w.Nk)).tiles<T>() * group; };
  SimtChunks c;
  c.sink_tiles = ceil_div(w.sink, T);
  c.q = cut(share((long long)B * H, tq, keys), 0, tq, keys);
  const long long sk = share((long long)B * Hk, tk, queries);
  c.k[0] = cut(sk, 0, c.sink_tiles, queries);
  c.k[1] = cut(sk, c.sink_tiles, tk, queries);
  return c;
}

size_t simt_share_floats(int B, int H, int Hk, const Window& w, int D) {
  const SimtChunks c = simt_chunks(B, H, Hk, w);
  return (c.q.slots(B * H) + 2 * (c.k[0].slots(B * Hk) + c.k[1].slots(B * Hk))) * (T * D);
}

cudaError_t launch_window_fwd_simt(const WindowAttn& a, cudaStream_t s) {
  return a.D == 64 ? fwd_d<64>(a, s) : fwd_d<128>(a, s);
}

cudaError_t launch_window_bwd_simt(const WindowAttn& a, cudaStream_t s) {
  return a.D == 64 ? bwd_d<64>(a, s) : bwd_d<128>(a, s);
}

}  // namespace dsa
