// Rows of D = 64 or 128 values held by D / 8 neighbouring threads, eight
// consecutive values each: loads, stores and sums used by the per-head norm
// with rotation and by the 8-bit activation rows.
//
// 8-bit rows: one fp32 scale = amax / 127 for each row and int8 codes =
// round-half-even(x * (127 / amax)), every operation rounded to fp32, so a
// program that repeats the three operations gets the same codes.  A code is
// off by at most half a step: amax / 254 (against amax / 16 next to amax for
// e4m3, whose smaller steps near zero win only for rows with far outliers).
// amax is taken on the magnitude bits, which order NaN above infinity above
// every finite value: a row with a non-finite value gets scale NaN and comes
// back as NaN throughout.  A row whose amax is below 2^-119 (127 / amax
// would overflow) is held as zeros.
#pragma once

#include "common.cuh"

namespace dsa {
namespace rows8 {

// What a load of eight values brings in, before it is converted.
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> { uint4 v; };
template <> struct Raw<float> { uint4 v, w; };
template <> struct Raw<int8_t> { uint2 v; float scale; };

// Rows are read once and written once: no reuse to keep in L1.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, Raw<__nv_bfloat16>& r) {
  r.v = __ldcs(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ void load8(const float* p, Raw<float>& r) {
  r.v = __ldcs(reinterpret_cast<const uint4*>(p));
  r.w = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
}
__device__ __forceinline__ void load8(const int8_t* p, Raw<int8_t>& r) {
  r.v = __ldcs(reinterpret_cast<const uint2*>(p));
}

__device__ __forceinline__ void unpack_bf16(uint32_t w, float& lo, float& hi) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void values8(const Raw<__nv_bfloat16>& r, float (&x)[8]) {
  unpack_bf16(r.v.x, x[0], x[1]);
  unpack_bf16(r.v.y, x[2], x[3]);
  unpack_bf16(r.v.z, x[4], x[5]);
  unpack_bf16(r.v.w, x[6], x[7]);
}
__device__ __forceinline__ void values8(const Raw<float>& r, float (&x)[8]) {
  x[0] = __uint_as_float(r.v.x); x[1] = __uint_as_float(r.v.y);
  x[2] = __uint_as_float(r.v.z); x[3] = __uint_as_float(r.v.w);
  x[4] = __uint_as_float(r.w.x); x[5] = __uint_as_float(r.w.y);
  x[6] = __uint_as_float(r.w.z); x[7] = __uint_as_float(r.w.w);
}
__device__ __forceinline__ void values8(const Raw<int8_t>& r, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = (float)(int8_t)(r.v.x >> (8 * e)) * r.scale;
    x[4 + e] = (float)(int8_t)(r.v.y >> (8 * e)) * r.scale;
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                            pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Sum over the TPR (8 or 16) neighbouring threads of a row, in all of them.
template <int TPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < TPR; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The row's codes and scale from its threads' values (see above).
template <int TPR>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float& scale) {
  uint32_t top = 0;  // magnitude bits: integer order is the order of magnitudes
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
  for (int o = 1; o < TPR; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float amax = __uint_as_float(top);
  float inv = 0.f;
  scale = 0.f;
  if (top >= 0x7f800000u) {
    scale = __uint_as_float(0x7fc00000u);
  } else if (amax >= 0x1p-119f) {
    scale = __fdiv_rn(amax, 127.0f);
    inv = __fdiv_rn(127.0f, amax);
  }
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    w[e >> 2] |= ((uint32_t)__float2int_rn(__fmul_rn(x[e], inv)) & 0xffu) << (8 * (e & 3));
  return make_uint2(w[0], w[1]);
}

}  // namespace rows8
}  // namespace dsa
