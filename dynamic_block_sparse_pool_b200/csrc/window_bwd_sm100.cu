// Window attention backward on Blackwell tensor cores (sm_100a), bf16, D = 64
// or 128.  With P the softmax of each query over its visible keys (from the
// forward's lse) and delta = rowsum(dO * O):
//   dS = P * (dP - delta), dP = dO V^T;
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO,
// dK and dV summed over the query heads that share the key head.
//
// One CTA per tile of 128 rows:
//   dq    one query tile against the key tiles it sees;
//   dkdv  one key tile against the query tiles that see it, for each query
//         head of its group in turn: every sum has a fixed order, no atomics.
//         A tile that many more queries see than the others (one with sinks) is
//         cut into several CTAs, whose fp32 shares window_join adds in order.
// Both kinds are CTAs of one launch.
// Per tile pair the S-type products go to tensor memory as fp32, the
// element-wise pass writes packed bf16 terms back into S's columns, and the
// gradient products take them from there.  For dQ, dS goes in as two terms,
// hi = bf16(x) and lo = bf16(x - hi): it sums to zero along a row, and where
// the keys share a common part (they do, in trained attention) dQ is a small
// difference of large sums that one bf16 term would lose.  dK and dV are sums
// over queries, whose terms have no such bond: P and dS go in as one term each
// (half a step, at most 2^-8 of each, as P in the forward).
//
// The element-wise pass (eight warps: one row per thread, warps 0-3 the first 64
// columns, warps 4-7 the others) is what bounds the kernels, so everything else
// goes on beside it.
//   Where tensor memory holds two buffers of S (all but dK/dV at D = 128): while
//   pair e is in its element-wise pass, S of e + 1 is done already and dP of
//   e + 1 runs as soon as dP of e has been read; the gradient products of e run
//   under the pass of e + 1, and S of e + 2 follows them into the buffer of e
//   (the MMAs of one thread run in order).
//   With one buffer each half's S and dP of e + 1 follow the half's gradient
//   products of e, so one half's pass goes on while the other half waits.
// Warp 8 issues the MMAs, warp 9 the TMA loads into two rings, one for each
// streamed tensor.  Every mbarrier wait is bounded; a timeout sets the device
// error word and the CTA winds down.
//
// Measured, 17,776 tokens, 8 heads, D = 64, every token in sight of 5,400 others
// and a prefix of 226, each kind alone: dq 430 us (511 with one buffer of S), dkdv
// 470 (617).  A pair of dq takes 1,990 cycles: exp2 1,024 on its unit, the MMAs 1,024
// (4 products), and the pass some 640 beside exp2 for waiting, reading tensor
// memory and handing over, which its two warps per scheduler, in phase, do not
// cover.  A delay of half the warps by a third of a pass, so that one half computes
// while the other reads, costs 5 %.  48 heads: 4.9 ms in all (575 TFLOP/s) with L2
// flushed between calls, 5.5 ms (515) back to back under the power cap.
// 8,192 tokens, 16 query heads on 4, D = 128, causal over 2,048, four sinks: dq
// 229 us, dkdv 270 (357 with the sinks' tile uncut and last, 376 with dP ahead
// of the gradients), 0.47 ms in all (640 TFLOP/s); causal without a window
// 0.82 ms (840).
#include <algorithm>

#include "bwd_tiles.cuh"
#include "tile_map.cuh"
#include "window_attn.cuh"

namespace dsa {
namespace {

using namespace bwd;

constexpr int kThreads = 384;
constexpr int kMmaWarp = 8, kLoadWarp = 9;
// Warps 10 and 11 only fill up the third warpgroup: of its registers (168 a thread
// at launch) the element-wise warps take what it does not need.
template <int D> constexpr int kElementRegs = D == 64 ? 216 : 208;  // (208 at D = 64: 3 % slower, 216 at 128: 2 %)
template <int D> constexpr int kOtherRegs = D == 64 ? 72 : 88;
static_assert(256 * kElementRegs<64> + 128 * kOtherRegs<64> <= 168 * kThreads);
static_assert(256 * kElementRegs<128> + 128 * kOtherRegs<128> <= 168 * kThreads);
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;

// Barriers, with room for three stages of each ring.  kBarS (+ half, with one
// buffer of S): S and dP of a pair are done; kBarR, with two buffers: dP is read
// out of tensor memory (eight warps); kBarP + 2 (pair % 2) (+ half, with one): the
// terms are written.  With two buffers of S a warp may be done with pair e + 1
// before another one is with e, so their arrivals must not meet on one barrier;
// e + 2 it cannot reach, since S and dP of it wait for every warp's kBarR of e + 1.
enum : int { kBarFixed = 0, kBarRingA = 1, kBarRingB = 4, kBarFreeA = 7, kBarFreeB = 10, kBarS = 13, kBarR = 15,
             kBarP = 16, kBarDrain = 20, kNumBars = 21 };

// Tensor and shared memory of a kernel with NG gradient accumulators.  The
// streamed tile A is read by S and by a gradient product, two pairs apart where
// S has two buffers; B by dP and, with NG = 2, by a gradient product.  A tile
// that is needed before the gradient products of the pair before it are done has
// a third stage, so that its load does not wait for them.
template <int D, int NG>
struct Layout {
  static constexpr bool kTwoS = 3 * BB + NG * D <= (int)kTmemCols;
  static constexpr uint32_t kColP = kTwoS ? 2 * BB : BB, kColG = kColP + BB;  // dP, gradients (S at 0)
  static constexpr int kTile = BB * D * 2;
  static constexpr int kStagesA = kTwoS ? 3 : 2, kStagesB = kTwoS && NG == 2 ? 3 : 2;
  static constexpr int kFixA = 0, kFixB = kTile;          // the CTA's own two tiles
  static constexpr int kRingA = 2 * kTile;
  static constexpr int kRingB = kRingA + kStagesA * kTile;
  static constexpr int kVec = kRingB + kStagesB * kTile;  // float [2][-lse2 | -delta][128] (dkdv)
  static constexpr int kBar = kVec + (NG == 2 ? 2 * 2 * BB * 4 : 0);
  static constexpr int kSlot = kBar + 8 * kNumBars;
  static constexpr int kBytes = kSlot + 16;
  static __device__ __forceinline__ uint32_t s_col(int it) { return kTwoS ? (uint32_t)(BB * (it & 1)) : 0u; }
};

struct BwdParams {
  Window w;
  BwdCut cut;      // dkdv
  float* shares;   // dkdv: [slot][dV, dK][128][D]
  int group;       // query heads per key head
  int tiles_q, tiles_k;  // tiles per head
  float scale, scale_log2;
  const float *lse, *delta;
  int heads;       // B H
  bool by_tile;    // dq: order_by_tile
  unsigned ctas_k; // CTAs of dkdv; the others are dq's
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

template <typename L>
__device__ __forceinline__ bool cta_begin(Cta& c, uint8_t* smem, unsigned* err) {
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
      for (int i = 0; i < kNumBars; ++i) mbar_init(c.bar(i), i == kBarR ? 8u : i >= kBarP && i < kBarP + 4 ? (L::kTwoS ? 8u : 4u) : 1u);
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
template <typename L>
__device__ __forceinline__ void cta_end(const Cta& c, int n, int issued_a, int issued_b) {
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
      for (int b = max(0, issued_a - L::kStagesA); b < issued_a; ++b)
        mbar_wait(c.bar(kBarRingA + b % L::kStagesA), (uint32_t)(b / L::kStagesA) & 1u);
      for (int b = max(0, issued_b - L::kStagesB); b < issued_b; ++b)
        mbar_wait(c.bar(kBarRingB + b % L::kStagesB), (uint32_t)(b / L::kStagesB) & 1u);
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

// S and dP of half h in registers; then dP's columns are free.
template <typename L>
__device__ __forceinline__ void read_half(const Cta& c, uint32_t lanes, uint32_t s_col, int h, uint32_t (&sv)[2][32],
                                          uint32_t (&pv)[2][32]) {
#pragma unroll
  for (int cc = 0; cc < 2; ++cc) {
    tmem_ld32(c.tmem + lanes + s_col + 64 * h + 32 * cc, sv[cc]);
    tmem_ld32(c.tmem + lanes + L::kColP + 64 * h + 32 * cc, pv[cc]);
  }
#pragma unroll
  for (int cc = 0; cc < 2; ++cc) {
    tmem_wait_ld_regs(sv[cc]);
    tmem_wait_ld_regs(pv[cc]);
  }
  if (L::kTwoS) {
    tc_fence_before();
    __syncwarp();
    if (c.lane == 0) mbar_arrive(c.bar(kBarR));
  }
}

// The loader's part: the fixed tiles of row f0 of head fh, then for it < n the
// two streamed tiles of head(it), row(it).
template <int D, typename L, typename Where>
__device__ __forceinline__ void load_tiles(const Cta& c, const CUtensorMap* fa, const CUtensorMap* fb, int f0, int fh,
                                           const CUtensorMap* sa, const CUtensorMap* sb, int n, Where where,
                                           int& issued_a, int& issued_b, unsigned* err) {
  constexpr uint32_t kTileBytes = L::kTile;
  mbar_expect_tx(c.bar(kBarFixed), 2 * kTileBytes);
  tma_tile<D>(c.base + L::kFixA, fa, f0, fh, c.bar(kBarFixed));
  tma_tile<D>(c.base + L::kFixB, fb, f0, fh, c.bar(kBarFixed));
  for (int it = 0; it < n; ++it) {
    const int a = it % L::kStagesA, b = it % L::kStagesB;
    int head, row;
    where(it, head, row);
    if (!mbar_wait(c.bar(kBarFreeA + a), ((uint32_t)(it / L::kStagesA) & 1u) ^ 1u) || *c.abort_flag) {
      give_up(c, err);
      return;
    }
    mbar_expect_tx(c.bar(kBarRingA + a), kTileBytes);
    tma_tile<D>(c.base + L::kRingA + a * kTileBytes, sa, row, head, c.bar(kBarRingA + a));
    ++issued_a;
    if (!mbar_wait(c.bar(kBarFreeB + b), ((uint32_t)(it / L::kStagesB) & 1u) ^ 1u) || *c.abort_flag) {
      give_up(c, err);
      return;
    }
    mbar_expect_tx(c.bar(kBarRingB + b), kTileBytes);
    tma_tile<D>(c.base + L::kRingB + b * kTileBytes, sb, row, head, c.bar(kBarRingB + b));
    ++issued_b;
  }
}

// The MMA issuer's part: S = A a^T and dP = B b^T (A, B fixed, a, b streamed),
// and `grads(half, column of S, stage of a, stage of b, accumulate)` once the
// terms are written.
template <int D, int NG, typename Grads>
__device__ __forceinline__ void issue_mmas(const Cta& c, int n, Grads grads, unsigned* err) {
  using L = Layout<D, NG>;
  constexpr uint32_t kTileBytes = L::kTile, kIdesc = idesc_bf16_f32(BB, BB, false);
  const uint32_t base = __shfl_sync(0xffffffffu, c.base, 0), tmem = __shfl_sync(0xffffffffu, c.tmem, 0);
  const uint64_t dA = smem_desc_sw128(base + L::kFixA, 16, 1024), dB = smem_desc_sw128(base + L::kFixB, 16, 1024);
  const uint64_t da = smem_desc_sw128(base + L::kRingA, 16, 1024), db = smem_desc_sw128(base + L::kRingB, 16, 1024);
  auto landed = [&](int ring, int it, int stages) {
    return warp_all(mbar_wait(c.bar(ring + it % stages), (uint32_t)(it / stages) & 1u));
  };
  auto product = [&](uint32_t d, uint64_t x, uint64_t y) {
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) mma_ss(d, x + kstep<D>(kk), y + kstep<D>(kk), kIdesc, kk > 0 ? 1u : 0u);
  };
  auto stage_a = [&](int it) { return (uint64_t)((it % L::kStagesA) * (kTileBytes >> 4)); };
  auto scores = [&](int it) { product(tmem + L::s_col(it), dA, da + stage_a(it)); };
  auto stage_b = [&](int it) { return (uint64_t)((it % L::kStagesB) * (kTileBytes >> 4)); };
  auto dprobs = [&](int it) { product(tmem + L::kColP, dB, db + stage_b(it)); };
  bool ok = warp_all(mbar_wait(c.bar(kBarFixed), 0u)) && landed(kBarRingA, 0, L::kStagesA) &&
            landed(kBarRingB, 0, L::kStagesB);
  if (ok) {
    if (elect_one()) {
      scores(0);
      dprobs(0);
      mma_commit(c.bar(kBarS));
      if (!L::kTwoS) mma_commit(c.bar(kBarS + 1));
      if (NG == 1) mma_commit(c.bar(kBarFreeB));
    }
    __syncwarp();
    if (L::kTwoS && n > 1 && (ok = landed(kBarRingA, 1, L::kStagesA))) {
      if (elect_one()) scores(1);
      __syncwarp();
    }
  }
  for (int it = 0; it < n && ok; ++it) {
    const bool more = it + 1 < n;
    if constexpr (L::kTwoS) {
      if (more) {
        if (!(ok = warp_all(mbar_wait_both(c.bar(kBarRingB + (it + 1) % L::kStagesB),
                                           (uint32_t)((it + 1) / L::kStagesB) & 1u, c.bar(kBarR), (uint32_t)it & 1u))))
          break;
        tc_fence_after();
        if (elect_one()) {
          dprobs(it + 1);
          mma_commit(c.bar(kBarS));
          if (NG == 1) mma_commit(c.bar(kBarFreeB + (it + 1) % L::kStagesB));
        }
        __syncwarp();
      }
      const uint32_t done = c.bar(kBarP + 2 * (it & 1)), parity = (uint32_t)(it >> 1) & 1u;
      const bool ahead = it + 2 < n;
      if (!(ok = warp_all(ahead ? mbar_wait_both(c.bar(kBarRingA + (it + 2) % L::kStagesA),
                                                 (uint32_t)((it + 2) / L::kStagesA) & 1u, done, parity)
                                : mbar_wait(done, parity))))
        break;
      tc_fence_after();
      if (elect_one()) {
        grads(0, L::s_col(it), stage_a(it), stage_b(it), it > 0);
        grads(1, L::s_col(it), stage_a(it), stage_b(it), true);
        mma_commit(c.bar(kBarFreeA + it % L::kStagesA));
        if (NG == 2) mma_commit(c.bar(kBarFreeB + it % L::kStagesB));
        if (ahead) scores(it + 2);
      }
      __syncwarp();
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!(ok = ok && warp_all(mbar_wait(c.bar(kBarP + 2 * (it & 1) + h), (uint32_t)(it >> 1) & 1u)))) break;
        tc_fence_after();
        if (elect_one()) {
          grads(h, 0u, stage_a(it), stage_b(it), it > 0 || h > 0);
          if (h == 1) mma_commit(c.bar(kBarFreeA + it % L::kStagesA));
          if (h == 1) mma_commit(c.bar(kBarFreeB + it % L::kStagesB));
        }
        __syncwarp();
        if (more) {  // the half's S and dP follow at once
          if (h == 0 && !(ok = landed(kBarRingA, it + 1, L::kStagesA) && landed(kBarRingB, it + 1, L::kStagesB))) break;
          if (elect_one()) {
            mma_rows_half<D>(tmem + 64 * h, dA, da + stage_a(it + 1), h);
            mma_rows_half<D>(tmem + L::kColP + 64 * h, dB, db + stage_b(it + 1), h);
            mma_commit(c.bar(kBarS + h));
          }
          __syncwarp();
        }
      }
    }
  }
  if (!ok) give_up(c, err);
}

template <int D>
__device__ __forceinline__ void dq_tile(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                        const CUtensorMap& tmO, const BwdParams& p, unsigned block, uint8_t* smem,
                                        __nv_bfloat16* __restrict__ dq, unsigned* err) {
  using L = Layout<D, 1>;
  Cta c;
  if (!cta_begin<L>(c, smem, err)) return;
  wait_for_previous();
  const int run = p.by_tile ? p.heads : p.tiles_q, o = block / run, r = block - o * run;
  const int bh = p.by_tile ? r : o, q0 = (p.tiles_q - 1 - (p.by_tile ? o : r)) * BB;
  const int q1 = min(q0 + BB, p.w.Nq);
  const KeyTiles<BB> kt = KeyTiles<BB>::of(p.w, q0, q1);
  const int n = kt.count();
  int issued_a = 0, issued_b = 0;

  if (c.warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs<D>));
    if (c.warp == kLoadWarp) {
      if (c.lane == 0 && n > 0)
        load_tiles<D, L>(c, &tmQ, &tmO, q0, bh, &tmK, &tmV, n, [&](int it, int& head, int& row) {
          head = bh / p.group;
          row = kt.tile(it) * BB;
        }, issued_a, issued_b, err);
    } else if (c.warp == kMmaWarp) {
      if (n > 0) {
        const uint32_t tmem = __shfl_sync(0xffffffffu, c.tmem, 0);
        const uint64_t dKm = smem_desc_sw128(__shfl_sync(0xffffffffu, c.base, 0) + L::kRingA, kSubBytes, 1024);
        issue_mmas<D, 1>(c, n, [&](int h, uint32_t s_col, uint64_t a, uint64_t, bool accumulate) {
          mma_grad_half<D>(tmem + L::kColG, tmem + s_col, dKm + a, h, accumulate);  // dQ += dS K
        }, err);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kElementRegs<D>));
    const int h = c.warp >> 2, row = 32 * (c.warp & 3) + c.lane;
    const uint32_t lanes = (uint32_t)(32 * (c.warp & 3)) << 16;
    const bool valid = q0 + row < q1;
    const size_t tok = (size_t)bh * p.w.Nq + q0 + row;
    // -lse (base 2) and -delta of the row; rows past the last query, and rows
    // that see no key, get -inf, so their P is 0 (lse = NaN, from a NaN that the
    // row met, stays: its P is NaN)
    const float ls = valid ? p.lse[tok] : -INFINITY;
    const float nl = ls != -INFINITY ? -ls * kLog2e : -INFINITY, nd = valid ? -p.delta[tok] : 0.f;
    const uint64_t sc2 = pack_f32x2(p.scale_log2, p.scale_log2), nl2 = pack_f32x2(nl, nl), nd2 = pack_f32x2(nd, nd);
    const int t = p.w.off + q0 + row, hi = p.w.hi(t), lo = p.w.lo(t);
    bool ok = true;
    for (int it = 0; it < n; ++it) {
      const int k0 = kt.tile(it) * BB;
      const bool whole = all_visible(p.w, q0, q1, k0, k0 + BB);
      if (!(ok = warp_all(mbar_wait(c.bar(kBarS + (L::kTwoS ? 0 : h)), (uint32_t)it & 1u)))) break;
      tc_fence_after();
      const uint32_t s_col = L::s_col(it);
      uint32_t sv[2][32], pv[2][32];
      read_half<L>(c, lanes, s_col, h, sv, pv);
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
        tmem_st16(c.tmem + lanes + s_col + col, dh);
        tmem_st16(c.tmem + lanes + s_col + col + 16, dl);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (c.lane == 0) mbar_arrive(c.bar(kBarP + 2 * (it & 1) + (L::kTwoS ? 0 : h)));
    }
    if (ok && n > 0) ok = warp_all(mbar_wait(c.bar(kBarFreeA + (n - 1) % L::kStagesA), (uint32_t)((n - 1) / L::kStagesA) & 1u));
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
          tmem_ld32(c.tmem + lanes + L::kColG + col, g);
          tmem_wait_ld_regs(g);
        } else {
#pragma unroll
          for (int u = 0; u < 32; ++u) g[u] = 0u;
        }
        if (valid) store_row_chunk(dq + tok * D + col, g, p.scale);
      }
    }
  }
  cta_end<L>(c, n, issued_a, issued_b);
}

template <int D>
__device__ __forceinline__ void dkdv_tile(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                          const CUtensorMap& tmO, const BwdParams& p, unsigned block, uint8_t* smem,
                                          __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv,
                                          unsigned* err) {
  using L = Layout<D, 2>;
  constexpr uint32_t kColV = L::kColG, kColK = L::kColG + D;
  int kv, tile, part;
  p.cut.place(block, p.tiles_k, kv, tile, part);
  const int k0 = tile * BB, k1 = min(k0 + BB, p.w.Nk);
  const QueryRun run = QueryRun::of(p.w, k0, k1);
  const int i0 = run.q0 / BB, per = run.tiles<BB>();
  // pairs e0 .. e0 + n - 1 of the tile: query tiles per head, head after head
  const int e0 = part * p.cut.chunk(tile), n = min(per * p.group - e0, p.cut.chunk(tile));
  if (part > 0 && n <= 0) return;  // (part 0 writes its zeros)
  Cta c;
  if (!cta_begin<L>(c, smem, err)) return;
  wait_for_previous();
  int issued_a = 0, issued_b = 0;

  if (c.warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs<D>));
    if (c.warp == kLoadWarp) {
      if (c.lane == 0 && n > 0)
        load_tiles<D, L>(c, &tmK, &tmV, k0, kv, &tmQ, &tmO, n, [&](int it, int& head, int& row) {
          const int g = (e0 + it) / per;
          head = kv * p.group + g;
          row = (i0 + e0 + it - g * per) * BB;
        }, issued_a, issued_b, err);
    } else if (c.warp == kMmaWarp) {
      if (n > 0) {
        const uint32_t tmem = __shfl_sync(0xffffffffu, c.tmem, 0), base = __shfl_sync(0xffffffffu, c.base, 0);
        const uint64_t dQm = smem_desc_sw128(base + L::kRingA, kSubBytes, 1024);
        const uint64_t dOm = smem_desc_sw128(base + L::kRingB, kSubBytes, 1024);
        issue_mmas<D, 2>(c, n, [&](int h, uint32_t s_col, uint64_t a, uint64_t b, bool accumulate) {
          mma_grad_half<D, false>(tmem + kColV, tmem + s_col, dOm + b, h, accumulate);       // dV += P^T dO
          mma_grad_half<D, false>(tmem + kColK, tmem + s_col + 16, dQm + a, h, accumulate);  // dK += dS^T Q
        }, err);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kElementRegs<D>));
    // thread = key row; columns = the query tile's queries, half h of them
    const int h = c.warp >> 2, row = 32 * (c.warp & 3) + c.lane, wt = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(32 * (c.warp & 3)) << 16;
    float* vec = reinterpret_cast<float*>(c.smem + L::kVec);
    const uint64_t sc2 = pack_f32x2(p.scale_log2, p.scale_log2);
    const int u = k0 + row;
    // -lse (base 2) and -delta of this half's 64 queries: threads 0-63 of the
    // four warps fetch the one, 64-127 the other, a tile pair ahead (of query
    // tile i0 + qi of head g)
    int g = n > 0 ? e0 / per : 0, qi = e0 - g * per;
    // what is loaded is touched a pair later only: the load's latency stays hidden
    const float* src = wt < 64 ? p.lse : p.delta;
    auto fetch = [&]() -> float {
      const int q = (i0 + qi) * BB + 64 * h + (wt & 63);
      float x = wt < 64 ? -INFINITY : 0.f;
      if (q < p.w.Nq) x = src[(size_t)(kv * p.group + g) * p.w.Nq + q];
      return x;
    };
    float next = n > 0 ? fetch() : 0.f;
    bool ok = true;
    for (int it = 0; it < n; ++it) {
      const int q0 = (i0 + qi) * BB;
      const bool whole = all_visible(p.w, q0, min(q0 + BB, p.w.Nq), k0, k1);
      float* nl = vec + (it & 1) * 2 * BB;
      float* nd = nl + BB;
      (wt < 64 ? nl : nd)[64 * h + (wt & 63)] = wt >= 64 ? -next : next != -INFINITY ? -next * kLog2e : -INFINITY;
      if (++qi == per) {
        qi = 0;
        ++g;
      }
      if (it + 1 < n) next = fetch();
      // the barrier of the half's four warps publishes the values and makes a
      // timed-out wait a decision of all four
      const bool late = !warp_all(mbar_wait(c.bar(kBarS + (L::kTwoS ? 0 : h)), (uint32_t)it & 1u));
      if (named_bar_or(1 + h, 128, late)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t s_col = L::s_col(it);
      uint32_t sv[2][32], pv[2][32];
      read_half<L>(c, lanes, s_col, h, sv, pv);
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
        tmem_st16(c.tmem + lanes + s_col + col, ph);
        tmem_st16(c.tmem + lanes + s_col + col + 16, dh);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (c.lane == 0) mbar_arrive(c.bar(kBarP + 2 * (it & 1) + (L::kTwoS ? 0 : h)));
    }
    if (ok && n > 0) ok = warp_all(mbar_wait(c.bar(kBarFreeA + (n - 1) % L::kStagesA), (uint32_t)((n - 1) / L::kStagesA) & 1u));
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
        if (p.cut.shared(tile)) {  // this CTA's share, for window_join_kernel
          float4* sh = reinterpret_cast<float4*>(
              p.shares + ((p.cut.slot(kv, tile, part) * 2 + h) * BB + row) * D + 32 * g32);
#pragma unroll
          for (int x = 0; x < 8; ++x)
            sh[x] = make_float4(__uint_as_float(g[4 * x]), __uint_as_float(g[4 * x + 1]), __uint_as_float(g[4 * x + 2]),
                                __uint_as_float(g[4 * x + 3]));
        } else if (u < k1) {
          store_row_chunk(dst + 32 * g32, g, h ? p.scale : 1.0f);
        }
      }
    }
  }
  cta_end<L>(c, n, issued_a, issued_b);
}

// dkdv's CTAs, then dq's, which fill in where those run out: 1,003 tokens, 4
// heads on 2, D = 64: 44 -> 32 us, 8,192 tokens, 16 heads on 4, D = 128, causal:
// 1,020 -> 815 us.  (At D = 64 the compiler spills a little more for having both:
// 1 % slower than two launches where there are dozens of waves of CTAs.)
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
window_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO, const BwdParams p,
                  __nv_bfloat16* __restrict__ dq, __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv,
                  unsigned* err) {
  extern __shared__ __align__(1024) uint8_t smem[];
  let_next_start();
  if (blockIdx.x < p.ctas_k)
    dkdv_tile<D>(tmQ, tmK, tmV, tmO, p, blockIdx.x, smem, dk, dv, err);
  else
    dq_tile<D>(tmQ, tmK, tmV, tmO, p, blockIdx.x - p.ctas_k, smem, dq, err);
}

// dK and dV of the tiles that several CTAs share, summed in order: four columns
// of a row per thread.  Grid: x = heads * tiles that are cut, y = kJoinCtas<D>.
template <int D>
constexpr int kJoinCtas = 2 * BB * (D / 4) / 256;

template <int D>
__global__ void __launch_bounds__(256)
window_join_kernel(const BwdParams p, __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv) {
  wait_for_previous();
  const int cut = p.cut.cut_tiles(), kv = blockIdx.x / cut, tile = p.cut.cut_tile(blockIdx.x - kv * cut);
  const int k0 = tile * BB, k1 = min(k0 + BB, p.w.Nk);
  const int n = QueryRun::of(p.w, k0, k1).tiles<BB>() * p.group, parts = max(1, ceil_div(n, p.cut.chunk(tile)));
  const int i = blockIdx.y * 256 + threadIdx.x, h = i / (BB * (D / 4)), r = i / (D / 4) % BB, d = 4 * (i % (D / 4));
  if (k0 + r >= k1) return;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = 0; c < parts; ++c) {
    const float4 x =
        *reinterpret_cast<const float4*>(p.shares + ((p.cut.slot(kv, tile, c) * 2 + h) * BB + r) * D + d);
    s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
  }
  const float mul = h ? p.scale : 1.f;
  uint2 o;
  o.x = pack_bf16(s.x * mul, s.y * mul);
  o.y = pack_bf16(s.z * mul, s.w * mul);
  *reinterpret_cast<uint2*>((h ? dk : dv) + ((size_t)kv * p.w.Nk + k0 + r) * D + d) = o;
}

template <int D>
cudaError_t launch_d(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mo,
                     const WindowAttn& a, cudaStream_t s) {
  const int smem = std::max(Layout<D, 1>::kBytes, Layout<D, 2>::kBytes);
  cudaError_t e = cudaFuncSetAttribute(window_bwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  BwdParams p;
  p.w = a.w;
  p.cut = bwd_cut(a.B, a.H, a.Hk, a.w);
  p.shares = a.shares;
  p.group = a.H / a.Hk;
  p.tiles_q = ceil_div(a.w.Nq, BB);
  p.tiles_k = ceil_div(a.w.Nk, BB);
  p.scale = a.scale;
  p.scale_log2 = a.scale * kLog2e;
  p.lse = a.lse;
  p.delta = a.delta;
  p.heads = a.B * a.H;
  p.by_tile = order_by_tile(a);
  p.ctas_k = (unsigned)p.cut.ctas(p.tiles_k);
  auto *dq = static_cast<__nv_bfloat16*>(a.dq), *dk = static_cast<__nv_bfloat16*>(a.dk),
       *dv = static_cast<__nv_bfloat16*>(a.dv);
  e = launch_next(window_bwd_kernel<D>, p.ctas_k + (unsigned)(p.heads * p.tiles_q), kThreads, smem, s, mq, mk, mv, mo, p,
                  dq, dk, dv, a.err);
  if (e != cudaSuccess) return e;
  const int cut = p.cut.cut_tiles();
  return cut ? launch_next(window_join_kernel<D>, dim3(a.B * a.Hk * cut, kJoinCtas<D>), 256, 0, s, p, dk, dv) : e;
}

}  // namespace

// Pairs of a key tile.
static int tile_pairs(const Window& w, int t, int group) {
  return QueryRun::of(w, t * BB, std::min((t + 1) * BB, w.Nk)).tiles<BB>() * group;
}

// A tile with sinks sees every query, the others a window of them: each kind is
// cut where its longest tile has more than one and a half times an SM's share of
// all pairs (a pair takes about 1.5 us, a CTA's start and its share 4 us, so not
// below eight pairs).
BwdChunks bwd_chunks(int B, int H, int Hk, const Window& w) {
  const int tiles = ceil_div(w.Nk, BB), group = H / Hk;
  BwdChunks c;
  c.sink_tiles = ceil_div(w.sink, BB);
  int longest[2] = {0, 0};
  long long all = 0;
  for (int t = 0; t < tiles; ++t) {
    const int n = tile_pairs(w, t, group);
    all += n;
    int& l = longest[t >= c.sink_tiles];
    l = std::max(l, n);
  }
  // (beyond 32 bits for tens of millions of tokens in sight of one another; a tile
  // that is cut has more pairs than that, so a part always fits)
  const long long share = std::max<long long>(8, (all * B * Hk + 147) / 148);
  for (int i = 0; i < 2; ++i) {
    const bool cut = 2ll * longest[i] > 3 * share;
    c.chunks[i] = cut ? (int)share : std::max(1, longest[i]);
    c.counts[i] = cut ? ceil_div(longest[i], c.chunks[i]) : 1;
  }
  c.heads = B * Hk;
  return c;
}

BwdCut bwd_cut(int B, int H, int Hk, const Window& w) {
  const int tiles = ceil_div(w.Nk, BB), group = H / Hk;
  BwdCut c;
  static_cast<BwdChunks&>(c) = bwd_chunks(B, H, Hk, w);
  for (int k = 0; k < 2; ++k) {
    c.from[k] = c.to[k] = k ? c.sink_tiles : 0;
    if (c.counts[k] == 1) continue;
    c.to[k] = k ? tiles : c.sink_tiles;
    while (tile_pairs(w, c.from[k], group) <= c.chunks[k]) ++c.from[k];  // (the longest tile stops both)
    while (tile_pairs(w, c.to[k] - 1, group) <= c.chunks[k]) --c.to[k];
  }
  return c;
}

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
