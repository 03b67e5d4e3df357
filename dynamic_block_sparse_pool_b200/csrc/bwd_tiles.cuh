// Tiles and products of the tensor-core backward passes: blocks of 128 rows,
// bf16 operands, P and dS as one or two bf16 terms each.
#pragma once

#include "sm100.cuh"

namespace dsa {
namespace bwd {

using namespace sm100;

constexpr int BB = 128;            // rows of a block (queries and keys)
constexpr int kSubBytes = BB * 64 * 2;  // one 128B-swizzled [128 x 64] sub-tile

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ bool warp_all(bool v) { return __all_sync(0xffffffffu, v); }

template <int D>
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int row, int bh,
                                         uint32_t bar) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) tma_load_3d(dst + c * kSubBytes, map, c * 64, row, bh, bar);
}

// K step kk (16 elements along D) of a K-major tile, as a descriptor offset
template <int D>
__device__ __forceinline__ uint64_t kstep(int kk) {
  return (uint64_t)(((kk >> 2) * kSubBytes + (kk & 3) * 32) >> 4);
}

// bf16 pair (lo element first) as one 32-bit word
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// x = hi + lo with hi = bf16(x), lo = bf16(x - hi), for a pair of values
__device__ __forceinline__ void split_pair(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = pack_bf16(a - __low2float(h), b - __high2float(h));
}

// S-type product for half h of the block's columns: D[tmem, 64 columns] =
// A B_h^T, A a [128 x D] tile and B_h rows 64h .. 64h + 63 of another, both
// K-major (64 rows of 128 bytes per 64-column sub-tile: 8192 bytes on).
template <int D>
__device__ __forceinline__ void mma_rows_half(uint32_t d, uint64_t a0, uint64_t b0, int h) {
  constexpr uint32_t kIdesc = idesc_bf16_f32(BB, BB / 2, false);
  const uint64_t bh = b0 + (uint64_t)((h * (BB / 2) * 128) >> 4);
  mma_ss(d, a0 + kstep<D>(0), bh + kstep<D>(0), kIdesc, 0u);
#pragma unroll
  for (int kk = 1; kk < D / 16; ++kk) mma_ss_acc(d, a0 + kstep<D>(kk), bh + kstep<D>(kk), kIdesc);
}

// gradient product over half h of the K dimension: D[tmem] (+)= (hi + lo)
// [tmem, rows x K steps 4h .. 4h + 3, packed as above] B, B a [128 x D] tile
// read MN-major (its rows are the K dimension)
// (kLo = false: hi alone)
template <int D, bool kLo = true>
__device__ __forceinline__ void mma_grad_half(uint32_t d, uint32_t a, uint64_t b0, int h,
                                              bool accumulate) {
  constexpr uint32_t kIdesc = idesc_bf16_f32(BB, D, true);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int kk = 4 * h + q;
    const uint32_t ah = a + 32u * (uint32_t)(kk >> 1) + 8u * (uint32_t)(kk & 1);
    const uint64_t b = b0 + (uint64_t)((kk * 2048) >> 4);
    if (q == 0 && !accumulate)
      mma_ts(d, ah, b, kIdesc, 0u);
    else
      mma_ts_acc(d, ah, b, kIdesc);
    if (kLo) mma_ts_acc(d, ah + 16u, b, kIdesc);
  }
}

// Stores 32 fp32 accumulator columns of this thread's row, times `mul`, as bf16.
__device__ __forceinline__ void store_row_chunk(__nv_bfloat16* dst, const uint32_t (&g)[32], float mul) {
  uint4* d4 = reinterpret_cast<uint4*>(dst);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint4 o;
    o.x = pack_bf16(__uint_as_float(g[8 * w + 0]) * mul, __uint_as_float(g[8 * w + 1]) * mul);
    o.y = pack_bf16(__uint_as_float(g[8 * w + 2]) * mul, __uint_as_float(g[8 * w + 3]) * mul);
    o.z = pack_bf16(__uint_as_float(g[8 * w + 4]) * mul, __uint_as_float(g[8 * w + 5]) * mul);
    o.w = pack_bf16(__uint_as_float(g[8 * w + 6]) * mul, __uint_as_float(g[8 * w + 7]) * mul);
    d4[w] = o;
  }
}

}  // namespace bwd
}  // namespace dsa
