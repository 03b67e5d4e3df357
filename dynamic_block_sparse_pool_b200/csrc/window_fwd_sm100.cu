// Window attention forward on Blackwell tensor cores (sm_100a), bf16,
// D = 64 or 128: TMA loads, tcgen05 MMAs with fp32 accumulators in tensor
// memory, online softmax on CUDA cores, warp-specialised and persistent.
//
// For every query: softmax over its visible keys (window.cuh), in one pass
// over key tiles of 128 with a running reference m and sum l:
//   P = 2^(S scale log2e - m),  l += rowsum(P),  O += P V;  O / l at the end.
// m only moves when a tile's maximum exceeds it by more than 16 (base 2), and
// then l and O are rescaled: P stays below 2^16, where bf16 and fp32 are as
// precise as below 1, and O and l share the reference, so the result is the
// softmax all the same.  P is rounded to bf16 for the second product (at most
// half a step, 2^-8 of each weight; l sums the unrounded values).
//
// An item is two neighbouring tiles of 128 queries of one head (one, where
// items would not fill the SMs), so a key tile in shared memory serves both
// and shared-memory traffic per MMA stays below what the tensor cores need.
// One CTA per SM takes one item of every gridDim.x, in an order that keeps
// concurrent windows in L2 (order_by_tile) and, where it can, deals long and
// short items out evenly: 8,192 tokens, 16 heads on 4, D = 128, causal without a
// window 352 -> 248 us (1,109 TFLOP/s).  384 threads:
//   warps 0-3  softmax and output of query tile A, one row per thread
//   warps 4-7  the same for tile B
//   warps 8, 9 MMA issuers of tile A and tile B (8 also allocates tensor
//              memory): an MMA and a wait cost an issuer as many cycles as the
//              tensor cores take for them, so each tile has its own
//   warp  10   TMA loader: the two Q tiles, then K and V tiles through a ring
//   (warp 11 only completes the warpgroup that gives registers up)
// Tensor memory: S_A, S_B (128 columns each; P overwrites S in place as
// packed bf16), O_A, O_B.  While tile A is in its softmax the tensor cores
// run tile B's PV and next S, and the other way round.  The MMAs of one
// thread run in order, so S(i+1) overwrites the buffer of P(i) after PV(i)
// has read it, and a finished S(i+1) also means that PV(i) is done: the
// softmax warps may rescale O.  The last PV has a barrier of its own (the
// next item's first S may be done before every softmax warp has noticed, and
// one barrier for both would run a phase ahead of it); the next item's first
// PV waits for their P, which they write after they have read O out.
//
// Masks: a key tile that every row of the query tile sees in full needs
// none; in the others hidden scores become -inf before the maximum, so what
// a hidden key holds (NaN included) does not matter for S.  A row whose keys
// are all hidden so far keeps m = -inf and uses 0 in its place, so its P is 0.
// Every mbarrier wait is bounded; a timeout sets the device error word and
// the CTA winds down.
//
// Measured, D = 128: 75,600 tokens, 40 heads, 7,200 to either side 21.1 ms (1,005
// TFLOP/s), 2 x 8,192 tokens, 32 heads on 8, causal over 2,048 with four sinks
// 0.51 ms (945) with L2 flushed between calls, 0.57 (841) back to back under the
// power cap.  The tensor cores work 55 % of the cycles: an MMA issuer takes
// as long as its MMAs, and the softmax of a tile (exp2, a quarter of the issue
// slots) hides behind the other tile's MMAs only in part.
#include "sm100.cuh"
#include "tile_map.cuh"
#include "window.cuh"
#include "window_attn.cuh"

namespace dsa {
namespace {

using namespace sm100;

constexpr int BM = 128, BN = 128;
constexpr int kThreads = 384;
// Registers: 12 warps get 168 each at launch (64,512 in all); the softmax
// warps, which hold a row of S, take 208, the others keep 88 (256 * 208 +
// 128 * 88 = 64,512).
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr int kMmaWarp = 8, kLoadWarp = 10;  // MMA issuers: 8 (tile A), 9 (tile B)
constexpr uint32_t kTmemCols = 512, kColO = 256;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kStep = 16.f;  // the reference moves when a maximum exceeds it by more

template <int D>
struct Smem {
  static constexpr int kTile = BM * D * 2;        // one [128 x D] bf16 tile
  static constexpr int kSub = BM * 64 * 2;        // one 128B-swizzled [128 x 64] part
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kQ = 0;                    // two tiles
  static constexpr int kRing = 2 * kTile;
  static constexpr int kBar = kRing + kStages * kTile;
  // barriers: per query tile Q landed, Q free; ring landed / free; per query
  // tile S done, its last PV done, and (by half) P written; teardown
  static constexpr int kQFull = 0, kQFree = 2, kFull = 4, kFree = kFull + kStages,
                       kS = kFree + kStages, kO = kS + 2, kP = kO + 2, kDrain = kP + 4,
                       kNumBars = kDrain + 2;
  static constexpr int kSlot = kBar + 8 * kNumBars;
  static constexpr int kBytes = kSlot + 16;
};

__device__ __forceinline__ bool warp_all(bool v) { return __all_sync(0xffffffffu, v); }

__device__ __forceinline__ float exp2_mufu(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct FwdParams {
  Window w;
  int H, group;       // query heads, query heads per key head
  int pairs;          // query tiles per item (1 or 2)
  int items_per_head;
  int items;
  int heads;          // B H
  bool by_tile;       // order of the items: head within query tile
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
};

// An item: head, first query, the key tiles of each query tile and of both.
struct Item {
  int bh, kv, q0;
  KeyTiles<BN> a, b, all;
  __device__ __forceinline__ Item(const FwdParams& p, int i) {
    const int run = p.by_tile ? p.heads : p.items_per_head, o = i / run, r = i - o * run;
    bh = p.by_tile ? r : o;
    q0 = (p.items_per_head - 1 - (p.by_tile ? o : r)) * (BM * p.pairs);
    kv = bh / p.group;  // (b H + h) / group = b Hk + h / group
    a = KeyTiles<BN>::of(p.w, q0, min(q0 + BM, p.w.Nq));
    b = p.pairs == 2 ? KeyTiles<BN>::of(p.w, q0 + BM, min(q0 + 2 * BM, p.w.Nq)) : KeyTiles<BN>::none();
    all = KeyTiles<BN>::join(a, b);
  }
};

// The CTA's r-th item: every other round backwards, so that who gets the longer
// item of one round gets the shorter one of the next.
__device__ __forceinline__ int item_at(int r) {
  return r * gridDim.x + (r & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, int row, int head,
                                          uint32_t bar) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) tma_load_3d(dst + c * Smem<D>::kSub, map, c * 64, row, head, bar);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
window_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const FwdParams p, unsigned* err) {
  using L = Smem<D>;
  constexpr int ST = L::kStages;
  constexpr uint32_t kTileBytes = L::kTile;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  if (base & 1023u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) flag_error(err, kErrAlign);
    return;
  }
  const uint32_t bars = base + L::kBar;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kSlot + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == kMmaWarp) {
    if (lane == 0) {
      for (int i = 0; i < L::kNumBars; ++i) {
        uint32_t count = 1;
        if (i >= L::kP && i < L::kP + 4) count = 4;                          // softmax warps
        if (i >= L::kFree && i < L::kFree + ST) count = 2;   // MMA issuers
        mbar_init(bar(i), count);
      }
      *abort_flag = 0;
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  if (warp == kLoadWarp && lane == 0) {
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  uint32_t issued = 0, q_issued = 0;  // loader: ring tiles issued, items whose Q tiles are
  int q_last = -1;                    // the query tile whose Q was loaded last
  bool had_mma = false;
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
      // ------------------------------------------------------------------ loader
      if (lane == 0) {
        bool ok = true;
        for (int r = 0, i; (i = item_at(r)) < p.items && ok; ++r) {
          const Item it(p, i);
          const int n = it.all.count();
          if (n == 0) continue;
          // Q's buffers are free once the last S of the tile's previous item is
          // done; K(0) goes between them, so tile A need not wait for tile B
          auto load_q = [&](int x) {
            ok = ok && (q_issued == 0 || mbar_wait(bar(L::kQFree + x), (q_issued - 1) & 1u)) && !*abort_flag;
            if (!ok) return;
            mbar_expect_tx(bar(L::kQFull + x), kTileBytes);
            // a second tile behind the last query reads as zeros
            load_tile<D>(base + L::kQ + x * kTileBytes, &tmQ, it.q0 + BM * x, it.bh, bar(L::kQFull + x));
            q_last = x;
          };
          // K(0), then K(e), V(e - 1) in the order the MMA issuers take them
          load_q(0);
          for (int e = 0; e <= 2 * n - 1 && ok; ++e) {
            if (e == 1) {
              load_q(1);
              if (!ok) break;
              ++q_issued;
            }
            const bool is_k = e == 0 || ((e & 1) && e < 2 * n - 1);
            const int blk = is_k ? (e + 1) / 2 : e == 2 * n - 1 ? n - 1 : e / 2 - 1;
            const uint32_t s = issued % ST;
            if (!(ok = mbar_wait(bar(L::kFree + s), ((issued / ST) & 1u) ^ 1u) && !*abort_flag)) break;
            mbar_expect_tx(bar(L::kFull + s), kTileBytes);
            load_tile<D>(base + L::kRing + s * kTileBytes, is_k ? &tmK : &tmV, it.all.tile(blk) * BN, it.kv,
                         bar(L::kFull + s));
            ++issued;
          }
        }
        if (!ok) {
          *abort_flag = 1;
          flag_error(err, kErrTimeout);
        }
      }
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
      // ------------------------------------------------------------- MMA issuers
      // One warp per query tile.  The whole warp runs the loop on values that
      // every lane knows to be the same (broadcasts, votes), so descriptors and
      // addresses are computed once per warp in uniform registers; one
      // elected lane issues the MMAs and commits.
      const int x = __shfl_sync(0xffffffffu, warp - kMmaWarp, 0);
      constexpr uint32_t kIdescS = idesc_bf16_f32(BM, BN, false);
      constexpr uint32_t kIdescO = idesc_bf16_f32(BM, D, true);
      const uint32_t ubase = __shfl_sync(0xffffffffu, base, 0), utmem = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t tS = utmem + 128u * x, tO = utmem + kColO + (uint32_t)D * x;
      const uint64_t dq = smem_desc_sw128(ubase + L::kQ + x * kTileBytes, 16, 1024);
      const uint64_t dk = smem_desc_sw128(ubase + L::kRing, 16, 1024);
      const uint64_t dv = smem_desc_sw128(ubase + L::kRing, L::kSub, 1024);
      const uint32_t ubars = ubase + L::kBar;
      auto ubar = [&](int i) { return ubars + 8u * (uint32_t)i; };
      auto kstep = [](int kk) -> uint64_t {  // 16 columns of D in a K-major tile
        return (uint64_t)(((kk >> 2) * L::kSub + (kk & 3) * 32) >> 4);
      };
      uint32_t ring = 0, ring_ph = 0;  // the next ring tile's stage and phase
      uint32_t p_ph = 0, q_ph = 0;     // phases of the next P tile and Q load
      bool ok = true;
      auto advance = [&](uint32_t& st, uint32_t& ph, uint32_t by) {
        st += by;
        if (st >= ST) {
          st -= ST;
          ph ^= 1u;
        }
      };
      for (int r = 0, i; (i = item_at(r)) < p.items && ok; ++r) {
        const Item it(p, i);
        const int n = __shfl_sync(0xffffffffu, it.all.count(), 0);
        if (n == 0) continue;
        // key tile positions e at which this query tile is active: two runs
        const KeyTiles<BN> mine = x ? it.b : it.a;
        const int f = __shfl_sync(0xffffffffu, min(mine.first, n), 0);
        const int r0 = __shfl_sync(0xffffffffu, mine.begin - it.all.begin + it.all.first, 0);
        const int r1 = __shfl_sync(0xffffffffu, mine.end - it.all.begin + it.all.first, 0);
        const int first = f > 0 ? 0 : r0, last = (r1 > r0 ? r1 : f) - 1;
        if (!(ok = warp_all(mbar_wait(ubar(L::kQFull + x), q_ph)))) break;
        q_ph ^= 1u;
        had_mma = true;
        uint32_t ks = ring, kph = ring_ph;  // K(e)
        uint32_t vs = ring, vph = ring_ph;  // V(e - 1)
        bool pend = false;                  // P(e - 1) is on its way
        // ring order: K(0), K(1), V(0), K(2), V(1), ..., K(n - 1), V(n - 2), V(n - 1)
        for (int e = 0; e <= n; ++e) {
          if (e == 1) {
            advance(ks, kph, 1);
            advance(vs, vph, n == 1 ? 1 : 2);
          } else if (e > 1) {
            advance(ks, kph, 2);
            advance(vs, vph, e == n ? 1 : 2);
          }
          if (e < n && !(ok = warp_all(mbar_wait(ubar(L::kFull + ks), kph)))) break;
          if (e > 0 && !(ok = warp_all(mbar_wait(ubar(L::kFull + vs), vph)))) break;
          const uint64_t k0 = dk + (uint64_t)(ks * (kTileBytes >> 4)), v0 = dv + (uint64_t)(vs * (kTileBytes >> 4));
          const bool act = e < n && (e < f || (e >= r0 && e < r1));
          if (pend) {
            // O (+)= P(e - 1) V(e - 1), a half of the keys at a time; the tile's
            // first PV overwrites O
            const uint32_t more = e - 1 > first;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (!(ok = ok && warp_all(mbar_wait(ubar(L::kP + 2 * x + h), p_ph)))) break;
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
                  mma_ts(tO, tS + 8u * kk, v0 + (uint64_t)((kk * 2048) >> 4), kIdescO, kk > 0 ? 1u : more);
              }
              __syncwarp();
            }
            if (!ok) break;
            p_ph ^= 1u;
          }
          if (act) {
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                mma_ss(tS, dq + kstep(kk), k0 + kstep(kk), kIdescS, kk > 0 ? 1u : 0u);
            }
            __syncwarp();
          }
          // S(e) is done; the tile's last PV has its own barrier: the next
          // item's first S may follow before every softmax warp has seen it
          if (act) {
            if (elect_one()) mma_commit(ubar(L::kS + x));
          } else if (pend && e > last) {
            if (elect_one()) mma_commit(ubar(L::kO + x));
          }
          pend = act;
          // (with the other tile's issuer: two arrivals free a tile)
          if (elect_one()) {
            if (e > 0) mma_commit(ubar(L::kFree + vs));
            if (e < n) mma_commit(ubar(L::kFree + ks));
            if (e == n - 1) mma_commit(ubar(L::kQFree + x));
          }
          __syncwarp();
        }
        // the next item's K(0) follows V(n - 1)
        ring = vs;
        ring_ph = vph;
        advance(ring, ring_ph, 1);
      }
      if (!ok && lane == 0) {
        *abort_flag = 1;
        flag_error(err, kErrTimeout);
      }
    }
  } else {
    // ----------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int x = warp >> 2;
    const int row = 32 * (warp & 3) + lane;
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + lane_off + 128u * x, tO = tmem + lane_off + kColO + (uint32_t)D * x;
    const float scale = p.scale_log2;
    uint32_t seen = 0, o_ph = 0;  // phases of S taken so far, phase of the next complete O
    bool ok = true;
    for (int r = 0, i; (i = item_at(r)) < p.items && ok; ++r) {
      const Item it(p, i);
      const KeyTiles<BN> mine = x ? it.b : it.a;
      const int q0 = it.q0 + BM * x, q1 = min(q0 + BM, p.w.Nq);
      if (q0 >= q1 || x >= p.pairs) continue;
      const int t = p.w.off + q0 + row;
      const int lo = p.w.lo(t), hi = p.w.hi(t);
      const int n = mine.count();
      float mref = -INFINITY, l = 0.f;
      for (int e = 0; e < n; ++e) {
        const int k0 = mine.tile(e) * BN;
        if (!(ok = warp_all(mbar_wait(bar(L::kS + x), seen & 1u)))) break;
        ++seen;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, s[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_wait_ld_regs(s[c]);
        if (!all_visible(p.w, q0, q1, k0, k0 + BN)) {
          const int chi = hi - k0, clo = lo - k0, csk = p.w.sink - k0;
          auto below = [](int v) { return v <= 0 ? 0u : v >= 32 ? 0xffffffffu : (1u << v) - 1u; };
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t m = below(chi - 32 * c) & (~below(clo - 32 * c) | below(csk - 32 * c));
#pragma unroll
            for (int u = 0; u < 32; ++u)
              if (!((m >> u) & 1u)) s[c][u] = 0xff800000u;  // -inf
          }
        }
        float m4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          m4[c] = __uint_as_float(s[c][0]);
#pragma unroll
          for (int u = 1; u + 1 < 32; u += 2)
            m4[c] = max3f(m4[c], __uint_as_float(s[c][u]), __uint_as_float(s[c][u + 1]));
          m4[c] = fmaxf(m4[c], __uint_as_float(s[c][31]));
        }
        const float m = max3f(m4[0], m4[1], fmaxf(m4[2], m4[3])) * scale;
        const bool move = m > mref + kStep || (mref == -INFINITY && m > mref);
        if (__any_sync(0xffffffffu, move)) {
          const float alpha = move ? exp2f(mref - m) : 1.f;  // 0 where the row had no keys yet
          if (move) mref = m;
          l *= alpha;
          if (e > 0) {
            // O holds the sum through the previous key tile (16 columns at a
            // time: the row of S stays in registers meanwhile)
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld16_wait(tO + 16 * c, o);
#pragma unroll
              for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * alpha);
              tmem_st16(tO + 16 * c, o);
            }
          }
        }
        const float nm = mref == -INFINITY ? 0.f : -mref;
        const uint64_t sc2 = pack_f32x2(scale, scale), nm2 = pack_f32x2(nm, nm);
        uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            float a, b;
            unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[c][2 * u]), __uint_as_float(s[c][2 * u + 1])), sc2, nm2),
                         a, b);
            a = exp2_mufu(a);
            b = exp2_mufu(b);
            sum2[u & 1] = add_f32x2(sum2[u & 1], pack_f32x2(a, b));
            const __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b);
            pk[u] = *reinterpret_cast<const uint32_t*>(&h2);
          }
          tmem_st16(tS + 16 * c, pk);
          if (c & 1) {  // half of the keys: the MMA issuer may start on them
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kP + 2 * x + (c >> 1)));
          }
        }
        float a, b;
        unpack_f32x2(add_f32x2(sum2[0], sum2[1]), a, b);
        l += a + b;
      }
      if (!ok) break;
      if (n > 0) {  // O is complete
        if (!(ok = warp_all(mbar_wait(bar(L::kO + x), o_ph)))) break;
        o_ph ^= 1u;
        tc_fence_after();
      }
      const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // NaN stays NaN
      const bool valid = q0 + row < q1;
      const size_t tok = (size_t)it.bh * p.w.Nq + q0 + row;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32(tO + 32 * c, o);
          tmem_wait_ld_regs(o);
        }
#pragma unroll
        for (int w8 = 0; w8 < 4; ++w8) {
          uint32_t h[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float a = __uint_as_float(o[8 * w8 + 2 * u]) * inv, b = __uint_as_float(o[8 * w8 + 2 * u + 1]) * inv;
            const __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b);
            h[u] = l == 0.f ? 0u : *reinterpret_cast<const uint32_t*>(&h2);
          }
          if (valid)
            *reinterpret_cast<uint4*>(p.out + tok * D + 32 * c + 8 * w8) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
      if (valid && p.lse) p.lse[tok] = l == 0.f ? -INFINITY : (mref + log2f(l)) * kLn2;
      tc_fence_before();
    }
    if (!ok) {
      *abort_flag = 1;
      if (lane == 0) flag_error(err, kErrTimeout);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // A role gave up: let every copy and MMA in flight finish (bounded)
    // before shared and tensor memory are released.
    if (had_mma) {  // the MMA issuers
      if (lane == 0) {
        mma_commit(bar(L::kDrain + warp - kMmaWarp));
        mbar_wait(bar(L::kDrain + warp - kMmaWarp), 0u);
      }
      __syncwarp();
    } else if (warp == kLoadWarp && lane == 0) {
      for (uint32_t b = issued > ST ? issued - ST : 0; b < issued; ++b)
        mbar_wait(bar(L::kFull + b % ST), (b / ST) & 1u);
      // (tile A is one load ahead of tile B between the two)
      const uint32_t qa = q_issued + (q_last == 0 ? 1u : 0u);
      if (qa > 0) mbar_wait(bar(L::kQFull), (qa - 1) & 1u);
      if (q_issued > 0) mbar_wait(bar(L::kQFull + 1), (q_issued - 1) & 1u);
    }
    tc_fence_before();
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
cudaError_t launch_d(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                     const FwdParams& p, int num_sms, unsigned* err, cudaStream_t s) {
  const int smem = Smem<D>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(window_fwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  window_fwd_kernel<D><<<min(p.items, num_sms), kThreads, smem, s>>>(mq, mk, mv, p, err);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_fwd_sm100(const WindowAttn& a, cudaStream_t s, const char** why) {
  const int BH = a.B * a.H;
  CUtensorMap mq, mk, mv;
  if (!make_bf16_tile_map(&mq, a.q, BH, a.w.Nq, a.D) || !make_bf16_tile_map(&mk, a.k, a.B * a.Hk, a.w.Nk, a.D) ||
      !make_bf16_tile_map(&mv, a.v, a.B * a.Hk, a.w.Nk, a.D)) {
    if (why) *why = "cuTensorMapEncodeTiled failed or is unavailable";
    return cudaErrorInvalidValue;
  }
  FwdParams p;
  p.w = a.w;
  p.H = a.H;
  p.group = a.H / a.Hk;
  // two query tiles per item, unless single ones are needed to fill the SMs
  const int tiles = ceil_div(a.w.Nq, BM);
  p.pairs = (long long)BH * ceil_div(tiles, 2) >= a.num_sms ? 2 : 1;
  p.items_per_head = ceil_div(tiles, p.pairs);
  p.items = BH * p.items_per_head;
  p.heads = BH;
  p.by_tile = order_by_tile(a);
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  return a.D == 64 ? launch_d<64>(mq, mk, mv, p, a.num_sms, a.err, s)
                   : launch_d<128>(mq, mk, mv, p, a.num_sms, a.err, s);
}

}  // namespace dsa
