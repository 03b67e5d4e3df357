// Window attention of a few new tokens over a cache of keys and values.
//
// Query i of Nq stands at position t = len - Nq + i of its stream and sees
// the keys u <= t with u < sink or u >= t - left (window.cuh with right = 0);
// len is read from device memory, so one captured launch serves a growing
// cache.
//
// Bound by memory: the visible keys and values are read once (2 D values per
// key for 4 D Nq H / Hk operations).  A CTA takes one key head and up to 16
// (fp32: 4 or 2) of its rows -- the query heads of the group times the new
// tokens -- so the group shares every key that is read.  Every warp takes steps
// of 16 or 32 (fp32: 8) keys in turn and keeps its own running maximum, sum and
// output in registers; the warps' results are joined in shared memory.  Where
// heads alone do not fill the SMs, several CTAs share one head's keys
// (decode_plan): small work as a cluster that joins through distributed shared
// memory, in the one launch; large work as single CTAs that leave their results
// in a workspace for a second small kernel (clusters do not pack the SMs as
// densely).  Either way in a fixed order.
//
// bf16: products on mma.sync (16 rows; at these sizes its rate is far above
// what memory feeds).  Each of eight warps has a ring of steps in shared memory,
// filled by TMA copies of 16 or 32 rows x 64 columns (192 KB on their way per SM, with
// nothing for the load-store units to do: per-lane cp.async held the kernel to
// 4.2 TB/s and register loads to 4.9; a bulk copy of one row takes 17 cycles to
// issue, as long as one of 2 KB).  The order of the summed dimension is free, so
// lane (g, c) takes elements 16 c .. 16 c + 15 of every 64 of key g's row for
// four k-steps, and Q is held in the same order; for P V the order of the output
// columns is free, so lane group g takes eight neighbouring columns of every 64
// of a value row, and two rows' elements are paired by byte permutes.  In the
// 128-byte swizzle both kinds of 16-byte reads fall in different banks.
// fp32: dot products on CUDA cores, four lanes per key; each lane group of
// four keeps the softmax of its own keys.
//
// Measured, D = 128, bf16, calls back to back: one stream, 40 heads of 32,400 keys
// 116 us (5.7 TB/s), 32 streams of 4,100 keys, 32 heads on 8, 89 us (6.0); with L2
// flushed between calls 130 and 106.
//
// Rows of the cache that no query sees may hold anything: a step may bring some
// in behind the end of a run (bf16), but their scores become -inf and their
// values 0 before use.
#include <cooperative_groups.h>

#include <algorithm>

#include "sm100.cuh"
#include "tile_map.cuh"
#include "window_attn.cuh"

namespace dsa {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarpsF32 = 4, kWarpsMma = 8;
constexpr float kLn2 = 0.69314718055994530942f, kLog2e = 1.4426950408889634f;

// One stream's visible keys: [0, first) and [lo, hi), as steps of K keys.
template <int K>
struct Steps {
  int first, lo, hi, nf, n;
  __device__ __forceinline__ Steps(int len, int nq, int left, int sink) {
    hi = max(len, 0);
    first = min(sink, hi);
    lo = max(first, len - nq - left);
    lo = min(lo, hi);
    nf = (first + K - 1) / K;
    n = nf + (hi - lo + K - 1) / K;
  }
  // keys base .. end-1 of the run that step s belongs to
  __device__ __forceinline__ void at(int s, int& base, int& end) const {
    base = s < nf ? s * K : lo + (s - nf) * K;
    end = s < nf ? first : hi;
  }
};

__device__ __forceinline__ bool sees(int t, int u, int left, int sink) {
  return u <= t && (u < sink || u >= t - left);
}

// A share's maximum as it is handed on: one whose every score was NaN has none,
// but its sum shows that it is not a share without keys (a maximum ignores NaN).
__device__ __forceinline__ float share_max(float m, float l) { return l == l ? m : l; }

// The warps' rows, their maxima and sums in shared memory -> the outputs.
// part: [kWarps][ROWS][D] outputs relative to m, m and l: [kWarps][ROWS]; m is
// -inf where there were no keys and NaN where l is (share_max).
// Warp 0's place then holds the CTA's, and each CTA of the cluster finishes
// its share of the rows from all of them.
template <typename T, int D, int ROWS, int kWarps>
__device__ __forceinline__ void join(float* part, float* pm, float* pl, int rows, size_t row0, const DecodeAttn& a) {
  constexpr int kThreads = 32 * kWarps;
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = cluster.num_blocks(), rank = cluster.block_rank();
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
    const int r = i / (D / 4), d = 4 * (i - r * (D / 4));
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, pm[w * ROWS + r]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      // a warp without a visible key has m = -inf and adds nothing
      const float a = pm[w * ROWS + r] == -INFINITY ? 0.f : exp2f(pm[w * ROWS + r] - m);
      const float4 v = *reinterpret_cast<const float4*>(part + (w * ROWS + r) * D + d);
      acc.x += a * v.x; acc.y += a * v.y; acc.z += a * v.z; acc.w += a * v.w;
    }
    *reinterpret_cast<float4*>(part + r * D + d) = acc;  // only this thread reads place 0's (r, d)
  }
  __syncthreads();
  if (threadIdx.x < rows) {
    const int r = threadIdx.x;
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, pm[w * ROWS + r]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      l += pm[w * ROWS + r] == -INFINITY ? 0.f : pl[w * ROWS + r] * exp2f(pm[w * ROWS + r] - m);
    pm[r] = share_max(m, l);
    pl[r] = l;
  }
  cluster.sync();
  for (int i = rank * kThreads + threadIdx.x; i < rows * (D / 4); i += cs * kThreads) {
    const int r = i / (D / 4), d = 4 * (i - r * (D / 4));
    float m = -INFINITY;
    for (int k = 0; k < cs; ++k) m = fmaxf(m, cluster.map_shared_rank(pm, k)[r]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    for (int k = 0; k < cs; ++k) {
      const float mk = cluster.map_shared_rank(pm, k)[r];
      const float a = mk == -INFINITY ? 0.f : exp2f(mk - m);
      const float4 v = *reinterpret_cast<const float4*>(cluster.map_shared_rank(part, k) + r * D + d);
      acc.x += a * v.x; acc.y += a * v.y; acc.z += a * v.z; acc.w += a * v.w;
      l += a * cluster.map_shared_rank(pl, k)[r];
    }
    const size_t row = row0 + r;
    if (a.groups > 1) {  // this CTA's share, for decode_join_kernel
      const size_t at = (size_t)blockIdx.y * a.B * a.H * a.Nq + row;
      *reinterpret_cast<float4*>(a.ws + at * D + d) = acc;
      if (d == 0)
        reinterpret_cast<float2*>(a.ws + (size_t)a.groups * a.B * a.H * a.Nq * D)[at] = make_float2(share_max(m, l), l);
      continue;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T* o = static_cast<T*>(a.out) + row * D + d;
    o[0] = Elem<T>::from_f(acc.x * inv);
    o[1] = Elem<T>::from_f(acc.y * inv);
    o[2] = Elem<T>::from_f(acc.z * inv);
    o[3] = Elem<T>::from_f(acc.w * inv);
    if (a.lse && d == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

// One row per CTA from the groups' shares; thread = column.
template <typename T, int D>
__global__ void __launch_bounds__(D)
decode_join_kernel(const DecodeAttn a) {
  wait_for_previous();
  const size_t rows = (size_t)a.B * a.H * a.Nq, row = blockIdx.x;
  const float2* ml = reinterpret_cast<const float2*>(a.ws + a.groups * rows * D);
  float m = -INFINITY;
  for (int g = 0; g < a.groups; ++g) m = fmaxf(m, ml[g * rows + row].x);
  float acc = 0.f, l = 0.f;
#pragma unroll 4
  for (int g = 0; g < a.groups; ++g) {
    const float2 v = ml[g * rows + row];
    const float f = v.x == -INFINITY ? 0.f : exp2f(v.x - m);
    acc = fmaf(f, a.ws[(g * rows + row) * D + threadIdx.x], acc);
    l = fmaf(f, v.y, l);
  }
  static_cast<T*>(a.out)[row * D + threadIdx.x] = Elem<T>::from_f(l == 0.f ? 0.f : acc / l);
  if (a.lse && threadIdx.x == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 2^x on the multi-function unit (the PTX approximate base-2 exponential).
__device__ __forceinline__ float exp2_mufu(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The stream's length, 0 (and reported) where it is outside [0, cap].
__device__ __forceinline__ int stream_len(const DecodeAttn& a, int b) {
  const int len = a.lens[b];
  if (len >= 0 && len <= a.cap) return len;
  if (threadIdx.x == 0) flag_error(a.err, kErrLength);
  return 0;
}

// Shared memory of the bf16 kernel: per warp a ring of three steps, each
// D / 64 swizzled parts of K of 64 columns, then of V (192 KB for the CTA, one
// on each SM).  At D = 64 a step is 32 keys: with 16 its softmax takes longer
// than its loads (122 against 105 us for 393 MB).
template <int D>
struct Ring {
  static constexpr int kKeys = D == 128 ? 16 : 32;
  static constexpr int kPart = kKeys * 128;       // bytes
  static constexpr int kStep = 2 * (D / 64) * kPart;
  static constexpr int kStages = 3;
  static constexpr int kBytes = kWarpsMma * kStages * kStep;
};

// Which key head and tile of its rows a CTA (or a cluster) has.  Grid: x = cluster
// size * key heads of all streams * row tiles (more tiles than the other dimensions
// have places where many heads share a key head), y = groups.  The heads run first:
// with the tiles of a head side by side, all at the same keys, 4 streams, 32 heads
// on 8, 8 new tokens, 4,000 keys in fp32 take 296 us, so 236.
struct RowTile {
  int kvh, tile;
  __device__ __forceinline__ RowTile(const DecodeAttn& a, int cluster_size) {
    const int at = blockIdx.x / cluster_size, heads = a.B * a.Hk;
    tile = at / heads;
    kvh = at - tile * heads;
  }
};

// One CTA has up to 16 rows.
template <int D>
__global__ void __launch_bounds__(32 * kWarpsMma, 1)
window_decode_mma_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const DecodeAttn a) {
  let_next_start();
  using R = Ring<D>;
  constexpr int ROWS = 16, K = R::kKeys, KT = K / 8, kWarps = kWarpsMma, ST = R::kStages;
  constexpr int KS = D / 32;      // 16-byte reads of a key row per lane
  constexpr int NT = D / 8;       // column tiles of 8 of the output
  constexpr int VW = D / 64;      // 16-byte reads of a value row per lane
  extern __shared__ __align__(1024) uint8_t ring[];
  float* part = reinterpret_cast<float*>(ring);  // [kWarps][ROWS][D], once the ring is done with
  __shared__ __align__(8) uint64_t full[kWarps * ST];
  __shared__ float pm[kWarps * ROWS], pl[kWarps * ROWS];
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = cluster.num_blocks(), rank = cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const RowTile at(a, cs);
  const int kvh = at.kvh, b = kvh / a.Hk, kh = kvh - b * a.Hk;
  const int all = a.group * a.Nq, row0 = at.tile * ROWS, rows = min(ROWS, all - row0);
  const int len = stream_len(a, b);
  const Steps<K> st(len, a.Nq, a.left, a.sink);
  // rows of the group are contiguous in q: (head, token)
  const size_t q_rows = ((size_t)b * a.H + (size_t)kh * a.group) * a.Nq;

  const uint8_t* mine = ring + warp * ST * R::kStep;
  const uint32_t to = sm100::smem_u32(mine), bar0 = sm100::smem_u32(full + warp * ST);
  if (sm100::smem_u32(ring) & 1023u) {  // the swizzle needs 1024-byte alignment
    if (threadIdx.x == 0) flag_error(a.err, kErrAlign);
    return;  // (every CTA alike)
  }
  if (lane < ST) sm100::mbar_init(bar0 + 8 * lane, 1);
  sm100::fence_mbar_init();
  __syncwarp();
  auto load = [&](int s, int stage) {
    __syncwarp();  // every lane is done with the stage
    if (s >= st.n || lane != 0) return;
    int base, end;
    st.at(s, base, end);
    const uint32_t bar = bar0 + 8 * stage, dst = to + stage * R::kStep;
    sm100::mbar_expect_tx(bar, R::kStep);
#pragma unroll
    for (int x = 0; x < D / 64; ++x) {
      sm100::tma_load_4d(dst + x * R::kPart, &tmK, 64 * x, base, kh, b, bar);
      sm100::tma_load_4d(dst + (D / 64 + x) * R::kPart, &tmV, 64 * x, base, kh, b, bar);
    }
  };
  const int stride = a.groups * cs * kWarps;
  int s = ((int)blockIdx.y * cs + rank) * kWarps + warp;
  int ahead = s;  // the next step to load
#pragma unroll
  for (int i = 0; i < ST; ++i, ahead += stride) load(ahead, i);

  uint4 qa[KS], qb[KS];  // rows g and g + 8
#pragma unroll
  for (int i = 0; i < KS; ++i) {
    const __nv_bfloat16* q =
        static_cast<const __nv_bfloat16*>(a.q) + (q_rows + row0) * D + 64 * (i >> 1) + 16 * c + 8 * (i & 1);
    qa[i] = g < rows ? *reinterpret_cast<const uint4*>(q + g * D) : make_uint4(0, 0, 0, 0);
    qb[i] = g + 8 < rows ? *reinterpret_cast<const uint4*>(q + (g + 8) * D) : make_uint4(0, 0, 0, 0);
  }
  const int ta = len - a.Nq + (row0 + g) % a.Nq, tb = len - a.Nq + (row0 + g + 8) % a.Nq;
  const int t_first = len - a.Nq, t_last = len - 1;
  const float sc = a.scale * kLog2e;

  float o[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  float ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;
  int stage = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (; s < st.n; s += stride) {
    if (!(ok = __all_sync(0xffffffffu, sm100::mbar_wait(bar0 + 8 * stage, phase)))) break;
    const uint8_t* kr = mine + stage * R::kStep;
    const uint8_t* vr = kr + (D / 64) * R::kPart;
    float x[KT][4] = {}, y[KT][4] = {};  // two sums each: shorter chains of products
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        const uint4 k = *reinterpret_cast<const uint4*>(kr + (i >> 1) * R::kPart + 128 * (8 * t + g) +
                                                        16 * ((2 * c + (i & 1)) ^ g));
        mma16816(x[t], qa[i].x, qb[i].x, qa[i].y, qb[i].y, k.x, k.y);
        mma16816(y[t], qa[i].z, qb[i].z, qa[i].w, qb[i].w, k.z, k.w);
      }
    int base, end;
    st.at(s, base, end);
    const bool whole = base + K <= end && base + K - 1 <= t_first && (s < st.nf || base >= t_last - a.left);
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[t][e] = (x[t][e] + y[t][e]) * sc;
    if (!whole) {
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int u = base + 8 * t + 2 * c + e;
          if (u >= end || !sees(ta, u, a.left, a.sink)) x[t][e] = -INFINITY;
          if (u >= end || !sees(tb, u, a.left, a.sink)) x[t][2 + e] = -INFINITY;
        }
    }
    float na = ma, nb = mb;
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      na = max3f(na, x[t][0], x[t][1]);
      nb = max3f(nb, x[t][2], x[t][3]);
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      na = fmaxf(na, __shfl_xor_sync(0xffffffffu, na, d));
      nb = fmaxf(nb, __shfl_xor_sync(0xffffffffu, nb, d));
    }
    if (__any_sync(0xffffffffu, na > ma || nb > mb)) {
      const float fa = na > ma ? exp2f(ma - na) : 1.f, fb = nb > mb ? exp2f(mb - nb) : 1.f;
      ma = na;
      mb = nb;
      la *= fa;
      lb *= fb;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        o[j][0] *= fa; o[j][1] *= fa;
        o[j][2] *= fb; o[j][3] *= fb;
      }
    }
    // a row that saw no key yet keeps m = -inf; 0 in its place makes its weights 0
    const float ra = ma == -INFINITY ? 0.f : ma, rb = mb == -INFINITY ? 0.f : mb;
    uint32_t pa[KT], pb[KT];
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const float p0 = exp2_mufu(x[t][0] - ra), p1 = exp2_mufu(x[t][1] - ra);
      const float p2 = exp2_mufu(x[t][2] - rb), p3 = exp2_mufu(x[t][3] - rb);
      la += p0 + p1;
      lb += p2 + p3;
      pa[t] = pack2(p0, p1);
      pb[t] = pack2(p2, p3);
    }
#pragma unroll
    for (int k16 = 0; k16 < KT / 2; ++k16) {
      const uint32_t a0 = pa[2 * k16], a1 = pb[2 * k16], a2 = pa[2 * k16 + 1], a3 = pb[2 * k16 + 1];
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        uint4 v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * k16 + 2 * c + (r & 1) + 8 * (r >> 1);
          v[r] = *reinterpret_cast<const uint4*>(vr + w * R::kPart + 128 * row + 16 * (g ^ (row & 7)));
          if (!whole && base + row >= end) v[r] = make_uint4(0u, 0u, 0u, 0u);
        }
        const uint32_t* v0 = reinterpret_cast<const uint32_t*>(&v[0]);
        const uint32_t* v1 = reinterpret_cast<const uint32_t*>(&v[1]);
        const uint32_t* v2 = reinterpret_cast<const uint32_t*>(&v[2]);
        const uint32_t* v3 = reinterpret_cast<const uint32_t*>(&v[3]);
#pragma unroll
        for (int y4 = 0; y4 < 4; ++y4) {
          const int j = 8 * w + 2 * y4;
          mma16816(o[j], a0, a1, a2, a3, __byte_perm(v0[y4], v1[y4], 0x5410), __byte_perm(v2[y4], v3[y4], 0x5410));
          mma16816(o[j + 1], a0, a1, a2, a3, __byte_perm(v0[y4], v1[y4], 0x7632),
                   __byte_perm(v2[y4], v3[y4], 0x7632));
        }
      }
    }
    load(ahead, stage);
    ahead += stride;
    if (++stage == ST) {
      stage = 0;
      phase ^= 1u;
    }
  }
  if (!ok) {
    if (lane == 0) flag_error(a.err, kErrTimeout);
    // copies may still be in flight: wait (bounded) for all of them
    for (int i = 0; i < ST && s < st.n; ++i, s += stride) {
      sm100::mbar_wait(bar0 + 8 * stage, phase);
      if (++stage == ST) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    la += __shfl_xor_sync(0xffffffffu, la, d);
    lb += __shfl_xor_sync(0xffffffffu, lb, d);
  }
  __syncthreads();  // every warp is done with the ring
  // column tile 8 x + y, column 2c + e of it is column 64 x + 8 (2c + e) + y of the row
  float* pw = part + warp * ROWS * D;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int d = 64 * (j >> 3) + 8 * (2 * c + e) + (j & 7);
      pw[g * D + d] = o[j][e];
      pw[(g + 8) * D + d] = o[j][2 + e];
    }
  }
  if (c == 0) {
    pm[warp * ROWS + g] = share_max(ma, la);
    pm[warp * ROWS + g + 8] = share_max(mb, lb);
    pl[warp * ROWS + g] = la;
    pl[warp * ROWS + g + 8] = lb;
  }
  join<__nv_bfloat16, D, ROWS, kWarps>(part, pm, pl, rows, q_rows + row0, a);
}

// Grid as above with tiles of 4 or 2 rows; lane (g, c): key g of a step of 8,
// elements 16 x + 4 c .. + 3 of its row.
template <int D>
__global__ void __launch_bounds__(32 * kWarpsF32, 2)
window_decode_f32_kernel(const DecodeAttn a) {
  let_next_start();
  constexpr int kWarps = kWarpsF32, kThreads = 32 * kWarps;
  constexpr int ROWS = 256 / D, K = 8, X = D / 16;  // as many rows as registers hold
  __shared__ __align__(16) float part[kWarps * ROWS * D];
  __shared__ __align__(16) float qs[ROWS * D];
  __shared__ float pm[kWarps * ROWS], pl[kWarps * ROWS];
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = cluster.num_blocks(), rank = cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const RowTile at(a, cs);
  const int kvh = at.kvh, b = kvh / a.Hk, kh = kvh - b * a.Hk;
  const int all = a.group * a.Nq, row0 = at.tile * ROWS, rows = min(ROWS, all - row0);
  const int len = stream_len(a, b);
  const Steps<K> st(len, a.Nq, a.left, a.sink);
  const size_t q_rows = ((size_t)b * a.H + (size_t)kh * a.group) * a.Nq;
  const float* kp = static_cast<const float*>(a.k) + b * a.ks[0] + kh * a.ks[1];
  const float* vp = static_cast<const float*>(a.v) + b * a.vs[0] + kh * a.vs[1];
  for (int i = threadIdx.x; i < ROWS * D; i += kThreads)
    qs[i] = i < rows * D ? static_cast<const float*>(a.q)[(q_rows + row0) * D + i] : 0.f;
  __syncthreads();
  const float sc = a.scale * kLog2e;
  float o[ROWS][4 * X], m[ROWS], l[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int d = 0; d < 4 * X; ++d) o[r][d] = 0.f;
  }
  for (int s = ((int)blockIdx.y * cs + rank) * kWarps + warp; s < st.n; s += a.groups * cs * kWarps) {
    int base, end;
    st.at(s, base, end);
    const int u = base + g, key = min(u, end - 1);
    float dot[ROWS] = {};
    const float* k = kp + (long long)key * a.ks[2] + 4 * c;
#pragma unroll
    for (int x = 0; x < X; ++x) {
      const float4 y = *reinterpret_cast<const float4*>(k + 16 * x);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const float4 q = *reinterpret_cast<const float4*>(qs + r * D + 16 * x + 4 * c);
        dot[r] = fmaf(q.x, y.x, fmaf(q.y, y.y, fmaf(q.z, y.z, fmaf(q.w, y.w, dot[r]))));
      }
    }
    float p[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      dot[r] += __shfl_xor_sync(0xffffffffu, dot[r], 1);
      dot[r] += __shfl_xor_sync(0xffffffffu, dot[r], 2);
      const int t = len - a.Nq + (row0 + r) % a.Nq;
      const float v = r < rows && u < end && sees(t, u, a.left, a.sink) ? dot[r] * sc : -INFINITY;
      const float mn = fmaxf(m[r], v), mu = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m[r] - mu);
      p[r] = exp2f(v - mu);
      m[r] = mn;
      l[r] = l[r] * f + p[r];
#pragma unroll
      for (int d = 0; d < 4 * X; ++d) o[r][d] *= f;
    }
    const float* vv = vp + (long long)key * a.vs[2] + 4 * c;
#pragma unroll
    for (int x = 0; x < X; ++x) {
      const float4 y = *reinterpret_cast<const float4*>(vv + 16 * x);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        o[r][4 * x] = fmaf(p[r], y.x, o[r][4 * x]);
        o[r][4 * x + 1] = fmaf(p[r], y.y, o[r][4 * x + 1]);
        o[r][4 * x + 2] = fmaf(p[r], y.z, o[r][4 * x + 2]);
        o[r][4 * x + 3] = fmaf(p[r], y.w, o[r][4 * x + 3]);
      }
    }
  }
  // join the eight lane groups of the warp
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    float top = m[r];
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float f = m[r] == -INFINITY ? 0.f : exp2f(m[r] - top);
    float sum = l[r] * f;
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
#pragma unroll
    for (int i = 0; i < 4 * X; ++i) {
      float v = f == 0.f ? 0.f : o[r][i] * f;
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
      if (g == 0) part[(warp * ROWS + r) * D + 16 * (i >> 2) + 4 * c + (i & 3)] = v;
    }
    if (lane == 0) {
      pm[warp * ROWS + r] = share_max(top, sum);
      pl[warp * ROWS + r] = sum;
    }
  }
  join<float, D, ROWS, kWarps>(part, pm, pl, rows, q_rows + row0, a);
}

// A cache [B, Hk, cap, D] through its strides; boxes of `keys` rows x 64 columns.
bool cache_map(CUtensorMap* map, const void* ptr, const long long* stride, const DecodeAttn& a, int D, int keys) {
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)a.cap, (cuuint64_t)a.Hk, (cuuint64_t)a.B};
  cuuint64_t st[3];
  for (int i = 0; i < 3; ++i) {
    st[i] = (cuuint64_t)stride[2 - i] * 2;
    if (dims[i + 1] == 1) st[i] = (cuuint64_t)D * 2;  // not used
  }
  const cuuint32_t box[4] = {64, (cuuint32_t)keys, 1, 1};
  return encode_bf16_map(map, ptr, 4, dims, st, box);
}

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), const DecodeAttn& a, const DecodePlan& plan, int threads, int smem,
                   cudaStream_t s, const Args&... args) {
  if (smem > 0) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * a.Hk * plan.cluster) * plan.tiles, (unsigned)plan.groups);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)plan.cluster;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, int D>
cudaError_t launch_d(const DecodeAttn& a, const DecodePlan& plan, cudaStream_t s, const char** why) {
  cudaError_t e;
  if constexpr (sizeof(T) == 2) {
    CUtensorMap mk, mv;
    if (!cache_map(&mk, a.k, a.ks, a, D, Ring<D>::kKeys) || !cache_map(&mv, a.v, a.vs, a, D, Ring<D>::kKeys)) {
      *why = "cuTensorMapEncodeTiled refused the caches' strides";
      return cudaErrorInvalidValue;
    }
    e = launch(window_decode_mma_kernel<D>, a, plan, 32 * kWarpsMma, Ring<D>::kBytes, s, mk, mv, a);
  } else {
    e = launch(window_decode_f32_kernel<D>, a, plan, 32 * kWarpsF32, 0, s, a);
  }
  if (e != cudaSuccess || plan.groups == 1) return e;
  return launch_next(decode_join_kernel<T, D>, (unsigned)(a.B * a.H * a.Nq), D, 0, s, a);
}

}  // namespace

// CTAs that share one key head's keys, each warp keeping two steps of the
// longest stream or more.  Below 32 MB of keys and values (about 5 us at the
// rate of HBM) a second launch and the trip through memory cost more than a
// cluster's looser packing.  Above, the number n for which the rounds of CTAs
// end soonest: `enough` of the `places` keep HBM busy, so a round of fewer takes
// as long as one of that many, and a round costs its CTAs / n.  Each CTA more
// costs about 1 % in its start and its share of the join.
DecodePlan decode_plan(bool bf16, int B, int H, int Hk, int Nq, int cap, int D, int left, int sink) {
  DecodePlan p;
  const int rows = bf16 ? 16 : 256 / D, keys = bf16 ? (D == 128 ? 16 : 32) : 8, warps = bf16 ? kWarpsMma : kWarpsF32;
  const int places = 148 * (bf16 ? 1 : 2), enough = bf16 ? 64 : places;
  p.tiles = ceil_div(H / Hk * Nq, rows);
  const long long heads = (long long)B * Hk, work = heads * p.tiles;
  const long long longest = left >= Window::kNoBound ? cap : std::min<long long>(cap, (long long)left + Nq + sink);
  const int most = (int)std::max(1ll, std::min(64ll, longest / (2ll * warps * keys)));
  p.groups = p.cluster = 1;
  if (heads * longest * D * (bf16 ? 4 : 8) >= 32ll << 20) {
    double best = 1e30;
    for (int n = 1; n <= most; ++n) {
      const long long rest = work * n % places;
      const double t = (double)(work * n - rest + (rest ? std::max<long long>(rest, enough) : 0)) / n * (1.0 + 0.01 * n);
      if (t < best) {
        best = t;
        p.groups = n;
      }
    }
  } else {
    while (p.cluster < 8 && 2 * p.cluster <= most && work * 2 * p.cluster <= places) p.cluster *= 2;
  }
  return p;
}

cudaError_t launch_window_decode(const DecodeAttn& a, const DecodePlan& plan, bool bf16, int D, cudaStream_t s,
                                 const char** why) {
  if (bf16)
    return D == 64 ? launch_d<__nv_bfloat16, 64>(a, plan, s, why) : launch_d<__nv_bfloat16, 128>(a, plan, s, why);
  return D == 64 ? launch_d<float, 64>(a, plan, s, why) : launch_d<float, 128>(a, plan, s, why);
}

}  // namespace dsa
