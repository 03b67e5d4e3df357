// Window attention backward on Blackwell tensor cores (sm_100a), bf16, D = 64
// or 128.  With P the softmax of each query over its visible keys (from the
// forward's lse) and delta = rowsum(dO * O):
//   dS = P * (dP - delta), dP = dO V^T;
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO,
// dK and dV summed over the query heads that share the key head.
//
// Two kernels, one CTA per tile of 128 rows:
//   dq    one query tile against the key tiles it sees;
//   dkdv  one key tile against the query tiles that see it, for each query
//         head of its group in turn: every sum has a fixed order, no atomics.
// Per tile pair the S-type products go to tensor memory as fp32, the
// element-wise pass writes packed bf16 terms back into S's columns, and the
// gradient products take them from there.  For dQ, dS goes in as two terms,
// hi = bf16(x) and lo = bf16(x - hi): it sums to zero along a row, and where
// the keys share a common part (they do, in trained attention) dQ is a small
// difference of large sums that one bf16 term would lose.  dK and dV are sums
// over queries, whose terms have no such bond: P and dS go in as one term each
// (half a step, at most 2^-8 of each, as P in the forward).
//
// Each tile pair runs as two halves of 64 columns: warps 0-3 own half 0 and
// warps 4-7 half 1 (one row per thread), each half with its own barriers, so
// while one half is in its element-wise pass the tensor cores work for the
// other.  Warp 8 issues the MMAs, warp 9 the TMA loads into a ring of two
// stages (three at D = 64).  Tensor memory: S 0-127, dP 128-255, gradients from
// 256.  Every mbarrier wait is bounded; a timeout sets the device error word
// and the CTA winds down.
#include "bwd_tiles.cuh"
#include "tile_map.cuh"
#include "window_attn.cuh"

namespace dsa {
namespace {

using namespace bwd;

constexpr int kThreads = 320;
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColP = 128, kColG = 256;
constexpr float kLog2e = 1.4426950408889634f;

// Barriers, with room for three ring stages; kBarR: a half's dP is read out of
// tensor memory (D = 64), kBarP: its terms are written.
enum : int { kBarFixed = 0, kBarRing = 1, kBarFree = 4, kBarS = 7, kBarP = 9, kBarR = 11, kBarDrain = 13,
             kNumBars = 14 };

template <int D>
struct Smem {
  static constexpr int kTile = BB * D * 2;
  static constexpr int kStages = D == 64 ? 3 : 2;       // of the streamed tiles
  static constexpr int kFixA = 0, kFixB = kTile;        // the CTA's own two tiles
  static constexpr int kRingA = 2 * kTile;
  static constexpr int kRingB = kRingA + kStages * kTile;
  static constexpr int kVec = kRingB + kStages * kTile;  // float [2][-lse2 | -delta][128] (dkdv)
  static constexpr int kBar = kVec + 2 * 2 * BB * 4;
  static constexpr int kSlot = kBar + 8 * kNumBars;
  static constexpr int kBytes = kSlot + 16;
};

struct BwdParams {
  Window w;
  int group;       // query heads per key head
  int tiles;       // tiles per head of the CTA's side
  float scale, scale_log2;
  const float *lse, *delta;
};

// bits 0 .. v-1
__device__ __forceinline__ uint32_t below(int v) { return v <= 0 ? 0u : v >= 32 ? 0xffffffffu : (1u << v) - 1u; }

// What the kernels share: barriers, tensor memory, teardown.
struct Cta {
  uint32_t base, bars, tmem;
  uint8_t* smem;
  volatile int* abort_flag;
  int warp, lane;
  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8u * (uint32_t)i; }
};

template <int D>
__device__ __forceinline__ bool cta_begin(Cta& c, uint8_t* smem, unsigned* err) {
  using L = Smem<D>;
  c.smem = smem;
  c.base = smem_u32(smem);
  c.warp = threadIdx.x >> 5;
  c.lane = threadIdx.x & 31;
  if (c.base & 1023u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) flag_error(err, kErrAlign);
    return false;
  }
  c.bars = c.base + L::kBar;
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + L::kSlot);
  c.abort_flag = reinterpret_cast<volatile int*>(smem + L::kSlot + 4);
  if (c.warp == kMmaWarp) {
    if (c.lane == 0) {
      // a half's four warps arrive on kBarP and kBarR
      for (int i = 0; i < kNumBars; ++i) mbar_init(c.bar(i), i >= kBarP && i < kBarR + 2 ? 4u : 1u);
      *c.abort_flag = 0;
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(smem_u32(slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  c.tmem = *slot;
  return true;
}

// After a role gave up, copies and MMAs may still be in flight: they finish
// (bounded) before shared and tensor memory are released.
template <int D>
__device__ __forceinline__ void cta_end(const Cta& c, int n, int issued) {
  constexpr int ST = Smem<D>::kStages;
  tc_fence_before();
  __syncthreads();
  if (*c.abort_flag) {
    if (c.warp == kMmaWarp && n > 0) {
      if (elect_one()) {
        mma_commit(c.bar(kBarDrain));
        mbar_wait(c.bar(kBarDrain), 0u);
      }
      __syncwarp();
    } else if (c.warp == kLoadWarp && c.lane == 0 && n > 0) {
      for (int b = issued > ST ? issued - ST : 0; b < issued; ++b)
        mbar_wait(c.bar(kBarRing + b % ST), (uint32_t)(b / ST) & 1u);
      mbar_wait(c.bar(kBarFixed), 0u);
    }
    tc_fence_before();
    __syncthreads();
  }
  if (c.warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(c.tmem, kTmemCols);
  }
}

__device__ __forceinline__ void give_up(const Cta& c, unsigned* err) {
  *c.abort_flag = 1;
  if (c.lane == 0) flag_error(err, kErrTimeout);
}

// S and dP of a half are in registers (the waits); with `tell`, the MMA issuer
// learns that dP's columns are free.
__device__ __forceinline__ void read_out(const Cta& c, int h, uint32_t (&sv)[2][32], uint32_t (&pv)[2][32], bool tell) {
#pragma unroll
  for (int cc = 0; cc < 2; ++cc) {
    tmem_wait_ld_regs(sv[cc]);
    tmem_wait_ld_regs(pv[cc]);
  }
  if (tell) {
    tc_fence_before();
    __syncwarp();
    if (c.lane == 0) mbar_arrive(c.bar(kBarR + h));
  }
}

// The loader's part: the fixed tiles of row f0 of head fh, then for it < n
// the two streamed tiles of head(it), row(it).
template <int D, typename Where>
__device__ __forceinline__ int load_tiles(const Cta& c, const CUtensorMap* fa, const CUtensorMap* fb, int f0, int fh,
                                          const CUtensorMap* sa, const CUtensorMap* sb, int n, Where where,
                                          unsigned* err) {
  using L = Smem<D>;
  constexpr uint32_t kTileBytes = L::kTile;
  int issued = 0;
  mbar_expect_tx(c.bar(kBarFixed), 2 * kTileBytes);
  tma_tile<D>(c.base + L::kFixA, fa, f0, fh, c.bar(kBarFixed));
  tma_tile<D>(c.base + L::kFixB, fb, f0, fh, c.bar(kBarFixed));
  for (int it = 0; it < n; ++it) {
    const int s = it % L::kStages;
    int head, row;
    where(it, head, row);
    if (!mbar_wait(c.bar(kBarFree + s), ((uint32_t)(it / L::kStages) & 1u) ^ 1u) || *c.abort_flag) {
      give_up(c, err);
      break;
    }
    mbar_expect_tx(c.bar(kBarRing + s), 2 * kTileBytes);
    tma_tile<D>(c.base + L::kRingA + s * kTileBytes, sa, row, head, c.bar(kBarRing + s));
    tma_tile<D>(c.base + L::kRingB + s * kTileBytes, sb, row, head, c.bar(kBarRing + s));
    issued = it + 1;
  }
  return issued;
}

// The MMA issuer's part: S = A a^T and dP = B b^T (A, B fixed, a, b streamed)
// in halves of 64 streamed rows; `grads(half, stage, accumulate)` once a half's
// terms are written.  The terms lie in S's columns, so the next pair's S
// follows the gradient products (the MMAs of one thread run in order).  dP's
// columns are free as soon as they are read: with three ring stages (D = 64)
// the next pair's dP runs while the half is in its element-wise pass (kEarly);
// with two its tiles would not have landed.
template <int D, typename Grads>
__device__ __forceinline__ void issue_mmas(const Cta& c, int n, Grads grads, unsigned* err) {
  using L = Smem<D>;
  constexpr uint32_t kTileBytes = L::kTile;
  constexpr bool kEarly = L::kStages == 3;
  const uint32_t base = __shfl_sync(0xffffffffu, c.base, 0), tmem = __shfl_sync(0xffffffffu, c.tmem, 0);
  const uint64_t dA = smem_desc_sw128(base + L::kFixA, 16, 1024), dB = smem_desc_sw128(base + L::kFixB, 16, 1024);
  const uint64_t da = smem_desc_sw128(base + L::kRingA, 16, 1024), db = smem_desc_sw128(base + L::kRingB, 16, 1024);
  int st = 0, st1 = 0;    // ring stages of this pair and of the next
  uint32_t ring_ph = 0;   // phase of the next pair's stage
  bool ok = warp_all(mbar_wait(c.bar(kBarFixed), 0u)) && warp_all(mbar_wait(c.bar(kBarRing), 0u));
  auto scores = [&](int stage, int h) {
    mma_rows_half<D>(tmem + kColS + 64 * h, dA, da + (uint64_t)(stage * (kTileBytes >> 4)), h);
  };
  auto dprobs = [&](int stage, int h) {
    mma_rows_half<D>(tmem + kColP + 64 * h, dB, db + (uint64_t)(stage * (kTileBytes >> 4)), h);
  };
  if (ok) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (elect_one()) {
        scores(0, h);
        dprobs(0, h);
        mma_commit(c.bar(kBarS + h));
      }
      __syncwarp();
    }
  }
  for (int it = 0; it < n && ok; ++it) {
    const bool more = it + 1 < n;
    const uint32_t ph = (uint32_t)it & 1u;
    st1 = st + 1;
    if (st1 == L::kStages) {
      st1 = 0;
      ring_ph ^= 1u;
    }
    if (kEarly && more) {
      if (!(ok = warp_all(mbar_wait(c.bar(kBarRing + st1), ring_ph)))) break;
      if (!(ok = warp_all(mbar_wait(c.bar(kBarR), ph)) && warp_all(mbar_wait(c.bar(kBarR + 1), ph)))) break;
      tc_fence_after();
      if (elect_one()) {  // both halves at once: half as many MMAs
        const uint64_t b0 = db + (uint64_t)(st1 * (kTileBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + kColP, dB + kstep<D>(kk), b0 + kstep<D>(kk), idesc_bf16_f32(BB, BB, false), kk > 0 ? 1u : 0u);
      }
      __syncwarp();
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!(ok = ok && warp_all(mbar_wait(c.bar(kBarP + h), ph)))) break;
      tc_fence_after();
      if (elect_one()) {
        grads(h, (uint64_t)(st * (kTileBytes >> 4)), it > 0 || h > 0);
        if (h == 1) mma_commit(c.bar(kBarFree + st));
      }
      __syncwarp();
      if (more) {
        if (!kEarly && h == 0 && !(ok = warp_all(mbar_wait(c.bar(kBarRing + st1), ring_ph)))) break;
        if (elect_one()) {
          scores(st1, h);
          if (!kEarly) dprobs(st1, h);
          mma_commit(c.bar(kBarS + h));
        }
        __syncwarp();
      }
    }
    st = st1;
  }
  if (!ok) give_up(c, err);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
window_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO, const BwdParams p,
                 __nv_bfloat16* __restrict__ dq, unsigned* err) {
  using L = Smem<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Cta c;
  if (!cta_begin<D>(c, smem, err)) return;
  const int bh = blockIdx.x / p.tiles, q0 = (blockIdx.x - bh * p.tiles) * BB;
  const int q1 = min(q0 + BB, p.w.Nq);
  const KeyTiles<BB> kt = KeyTiles<BB>::of(p.w, q0, q1);
  const int n = kt.count();
  int issued = 0;

  if (c.warp == kLoadWarp) {
    if (c.lane == 0 && n > 0)
      issued = load_tiles<D>(c, &tmQ, &tmO, q0, bh, &tmK, &tmV, n, [&](int it, int& head, int& row) {
        head = bh / p.group;
        row = kt.tile(it) * BB;
      }, err);
  } else if (c.warp == kMmaWarp) {
    if (n > 0) {
      const uint32_t tmem = __shfl_sync(0xffffffffu, c.tmem, 0);
      const uint64_t dKm = smem_desc_sw128(__shfl_sync(0xffffffffu, c.base, 0) + L::kRingA, kSubBytes, 1024);
      issue_mmas<D>(c, n, [&](int h, uint64_t off, bool accumulate) {
        mma_grad_half<D>(tmem + kColG, tmem + kColS, dKm + off, h, accumulate);  // dQ += dS K
      }, err);
    }
  } else {
    const int h = c.warp >> 2, row = 32 * (c.warp & 3) + c.lane;
    const uint32_t lanes = (uint32_t)(32 * (c.warp & 3)) << 16;
    const bool valid = q0 + row < q1;
    const size_t tok = (size_t)bh * p.w.Nq + q0 + row;
    // -lse (base 2) and -delta of the row; rows past the last query, and rows
    // that see no key, get -inf, so their P is 0
    const float ls = valid ? p.lse[tok] : -INFINITY;
    const float nl = ls > -INFINITY ? -ls * kLog2e : -INFINITY, nd = valid ? -p.delta[tok] : 0.f;
    const uint64_t sc2 = pack_f32x2(p.scale_log2, p.scale_log2), nl2 = pack_f32x2(nl, nl), nd2 = pack_f32x2(nd, nd);
    const int t = p.w.off + q0 + row, hi = p.w.hi(t), lo = p.w.lo(t);
    bool ok = true;
    for (int it = 0; it < n; ++it) {
      const int k0 = kt.tile(it) * BB;
      const bool whole = all_visible(p.w, q0, q1, k0, k0 + BB);
      if (!(ok = warp_all(mbar_wait(c.bar(kBarS + h), (uint32_t)it & 1u)))) break;
      tc_fence_after();
      uint32_t sv[2][32], pv[2][32];
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        tmem_ld32(c.tmem + lanes + kColS + 64 * h + 32 * cc, sv[cc]);
        tmem_ld32(c.tmem + lanes + kColP + 64 * h + 32 * cc, pv[cc]);
      }
      read_out(c, h, sv, pv, D == 64);
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const uint32_t col = 64u * h + 32u * cc;
        if (!whole) {
          const int k = k0 + (int)col;
          const uint32_t m = below(hi - k) & (~below(lo - k) | below(p.w.sink - k));
#pragma unroll
          for (int u = 0; u < 32; ++u)
            if (!((m >> u) & 1u)) {
              sv[cc][u] = 0xff800000u;  // -inf: P = 0
              pv[cc][u] = 0u;
            }
        }
        uint32_t dh[16], dl[16];
#pragma unroll
        for (int m = 0; m < 16; ++m) {
          float t0, t1, g0, g1;
          unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(sv[cc][2 * m]), __uint_as_float(sv[cc][2 * m + 1])), sc2, nl2),
                       t0, t1);
          const uint64_t p2 = pack_f32x2(exp2_approx(t0), exp2_approx(t1));
          const uint64_t d2 = add_f32x2(pack_f32x2(__uint_as_float(pv[cc][2 * m]), __uint_as_float(pv[cc][2 * m + 1])), nd2);
          unpack_f32x2(mul_f32x2(p2, d2), g0, g1);
          split_pair(g0, g1, dh[m], dl[m]);
        }
        tmem_st16(c.tmem + lanes + kColS + col, dh);
        tmem_st16(c.tmem + lanes + kColS + col + 16, dl);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (c.lane == 0) mbar_arrive(c.bar(kBarP + h));
    }
    if (ok && n > 0) ok = warp_all(mbar_wait(c.bar(kBarFree + (n - 1) % L::kStages), (uint32_t)((n - 1) / L::kStages) & 1u));
    if (!ok) {
      give_up(c, err);
    } else {
      tc_fence_after();
      // half h writes its half of the columns
#pragma unroll
      for (int g32 = 0; g32 < D / 64; ++g32) {
        const int col = h * (D / 2) + 32 * g32;
        uint32_t g[32];
        if (n > 0) {
          tmem_ld32(c.tmem + lanes + kColG + col, g);
          tmem_wait_ld_regs(g);
        } else {
#pragma unroll
          for (int u = 0; u < 32; ++u) g[u] = 0u;
        }
        if (valid) store_row_chunk(dq + tok * D + col, g, p.scale);
      }
    }
  }
  cta_end<D>(c, n, issued);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
window_dkdv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO, const BwdParams p,
                   __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv, unsigned* err) {
  using L = Smem<D>;
  constexpr uint32_t kColV = kColG, kColK = kColG + D;
  extern __shared__ __align__(1024) uint8_t smem[];
  Cta c;
  if (!cta_begin<D>(c, smem, err)) return;
  const int kv = blockIdx.x / p.tiles, k0 = (blockIdx.x - kv * p.tiles) * BB;
  const int k1 = min(k0 + BB, p.w.Nk);
  const QueryRun run = QueryRun::of(p.w, k0, k1);
  const int i0 = run.q0 / BB, per = run.q1 > run.q0 ? ceil_div(run.q1, BB) - i0 : 0;
  const int n = per * p.group;  // query tiles per head, head after head
  int issued = 0;

  if (c.warp == kLoadWarp) {
    if (c.lane == 0 && n > 0)
      issued = load_tiles<D>(c, &tmK, &tmV, k0, kv, &tmQ, &tmO, n, [&](int it, int& head, int& row) {
        const int g = it / per;
        head = kv * p.group + g;
        row = (i0 + it - g * per) * BB;
      }, err);
  } else if (c.warp == kMmaWarp) {
    if (n > 0) {
      const uint32_t tmem = __shfl_sync(0xffffffffu, c.tmem, 0), base = __shfl_sync(0xffffffffu, c.base, 0);
      const uint64_t dQm = smem_desc_sw128(base + L::kRingA, kSubBytes, 1024);
      const uint64_t dOm = smem_desc_sw128(base + L::kRingB, kSubBytes, 1024);
      issue_mmas<D>(c, n, [&](int h, uint64_t off, bool accumulate) {
        mma_grad_half<D, false>(tmem + kColV, tmem + kColS, dOm + off, h, accumulate);       // dV += P^T dO
        mma_grad_half<D, false>(tmem + kColK, tmem + kColS + 16, dQm + off, h, accumulate);  // dK += dS^T Q
      }, err);
    }
  } else {
    // thread = key row; columns = the query tile's queries, half h of them
    const int h = c.warp >> 2, row = 32 * (c.warp & 3) + c.lane, wt = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(32 * (c.warp & 3)) << 16;
    float* vec = reinterpret_cast<float*>(c.smem + L::kVec);
    const uint64_t sc2 = pack_f32x2(p.scale_log2, p.scale_log2);
    const int u = k0 + row;
    // -lse (base 2) and -delta of this half's 64 queries: threads 0-63 of the
    // four warps fetch the one, 64-127 the other, a tile pair ahead
    auto fetch = [&](int it) -> float {
      const int g = it / per, q = (i0 + it - g * per) * BB + 64 * h + (wt & 63);
      const size_t tok = (size_t)(kv * p.group + g) * p.w.Nq + q;
      const bool in = q < p.w.Nq;
      if (wt >= 64) return in ? -p.delta[tok] : 0.f;
      const float ls = in ? p.lse[tok] : -INFINITY;
      return ls > -INFINITY ? -ls * kLog2e : -INFINITY;
    };
    float next = n > 0 ? fetch(0) : 0.f;
    bool ok = true;
    for (int it = 0; it < n; ++it) {
      const int q0 = (i0 + it % per) * BB;
      const bool whole = all_visible(p.w, q0, min(q0 + BB, p.w.Nq), k0, k1);
      float* nl = vec + (it & 1) * 2 * BB;
      float* nd = nl + BB;
      (wt < 64 ? nl : nd)[64 * h + (wt & 63)] = next;
      if (it + 1 < n) next = fetch(it + 1);
      // the barrier of the half's four warps publishes the values and makes a
      // timed-out wait a decision of all four
      const bool late = !warp_all(mbar_wait(c.bar(kBarS + h), (uint32_t)it & 1u));
      if (named_bar_or(1 + h, 128, late)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t sv[2][32], pv[2][32];
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        tmem_ld32(c.tmem + lanes + kColS + 64 * h + 32 * cc, sv[cc]);
        tmem_ld32(c.tmem + lanes + kColP + 64 * h + 32 * cc, pv[cc]);
      }
      read_out(c, h, sv, pv, D == 64);
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const uint32_t col = 64u * h + 32u * cc;
        if (!whole) {
          // query i of the tile sees key u iff t >= u - right and (u < sink or t <= u + left)
          const int t0 = p.w.off + q0 + (int)col;
          const uint32_t m = ~below(u - p.w.right - t0) & (u < p.w.sink ? 0xffffffffu : below(u + p.w.left + 1 - t0));
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!((m >> e) & 1u)) {
              sv[cc][e] = 0xff800000u;
              pv[cc][e] = 0u;
            }
        }
        uint32_t ph[16], dh[16];
#pragma unroll
        for (int m = 0; m < 16; ++m) {
          const int qq = (int)col + 2 * m;  // even: the pairs are 8-byte aligned
          float t0, t1, g0, g1;
          unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(sv[cc][2 * m]), __uint_as_float(sv[cc][2 * m + 1])), sc2,
                                 *reinterpret_cast<const uint64_t*>(nl + qq)), t0, t1);
          const float p0 = exp2_approx(t0), p1 = exp2_approx(t1);
          ph[m] = pack_bf16(p0, p1);
          const uint64_t d2 = add_f32x2(pack_f32x2(__uint_as_float(pv[cc][2 * m]), __uint_as_float(pv[cc][2 * m + 1])),
                                        *reinterpret_cast<const uint64_t*>(nd + qq));
          unpack_f32x2(mul_f32x2(pack_f32x2(p0, p1), d2), g0, g1);
          dh[m] = pack_bf16(g0, g1);
        }
        tmem_st16(c.tmem + lanes + kColS + col, ph);
        tmem_st16(c.tmem + lanes + kColS + col + 16, dh);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (c.lane == 0) mbar_arrive(c.bar(kBarP + h));
    }
    if (ok && n > 0) ok = warp_all(mbar_wait(c.bar(kBarFree + (n - 1) % L::kStages), (uint32_t)((n - 1) / L::kStages) & 1u));
    if (!ok) {
      give_up(c, err);
    } else {
      tc_fence_after();
      // half 0 writes dV, half 1 dK
      __nv_bfloat16* dst = (h ? dk : dv) + ((size_t)kv * p.w.Nk + u) * D;
#pragma unroll
      for (int g32 = 0; g32 < D / 32; ++g32) {
        uint32_t g[32];
        if (n > 0) {
          tmem_ld32(c.tmem + lanes + (h ? kColK : kColV) + 32 * g32, g);
          tmem_wait_ld_regs(g);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) g[e] = 0u;
        }
        if (u < k1) store_row_chunk(dst + 32 * g32, g, h ? p.scale : 1.0f);
      }
    }
  }
  cta_end<D>(c, n, issued);
}

template <int D>
cudaError_t launch_d(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mo,
                     const WindowAttn& a, cudaStream_t s) {
  const int smem = Smem<D>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(window_dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(window_dkdv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  BwdParams p{a.w, a.H / a.Hk, ceil_div(a.w.Nq, BB), a.scale, a.scale * kLog2e, a.lse, a.delta};
  window_dq_kernel<D><<<a.B * a.H * p.tiles, kThreads, smem, s>>>(mq, mk, mv, mo, p, static_cast<__nv_bfloat16*>(a.dq),
                                                                  a.err);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  p.tiles = ceil_div(a.w.Nk, BB);
  window_dkdv_kernel<D><<<a.B * a.Hk * p.tiles, kThreads, smem, s>>>(
      mq, mk, mv, mo, p, static_cast<__nv_bfloat16*>(a.dk), static_cast<__nv_bfloat16*>(a.dv), a.err);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_bwd_sm100(const WindowAttn& a, cudaStream_t s, const char** why) {
  CUtensorMap mq, mk, mv, mo;
  if (!make_bf16_tile_map(&mq, a.q, a.B * a.H, a.w.Nq, a.D) || !make_bf16_tile_map(&mk, a.k, a.B * a.Hk, a.w.Nk, a.D) ||
      !make_bf16_tile_map(&mv, a.v, a.B * a.Hk, a.w.Nk, a.D) ||
      !make_bf16_tile_map(&mo, a.dout, a.B * a.H, a.w.Nq, a.D)) {
    if (why) *why = "cuTensorMapEncodeTiled failed or is unavailable";
    return cudaErrorInvalidValue;
  }
  return a.D == 64 ? launch_d<64>(mq, mk, mv, mo, a, s) : launch_d<128>(mq, mk, mv, mo, a, s);
}

}  // namespace dsa
