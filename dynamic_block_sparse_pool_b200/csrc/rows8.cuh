// Rows of D = 64 or 128 values held by D / 8 neighbouring threads, eight
// consecutive values each: loads, stores and sums used by the per-head norm
// with rotation and by the 8-bit activation rows.
//
// 8-bit rows: one fp32 scale = amax / 127 for each row and int8 codes =
// round-half-even(x * (127 / amax)), every operation rounded to fp32, so a
// program that repeats the three operations gets the same codes.  A code is
// off by at most half a step: amax / 254 (against amax / 28 next to amax for
// e4m3 with amax at its largest value, 448, where a step is 32; its smaller steps
// near zero win only for rows with far outliers).
// amax is taken on the magnitude bits, which order NaN above infinity above
// every finite value: a row with a non-finite value gets scale NaN and comes
// back as NaN throughout.  A row whose amax is below 2^-119 is held as zeros:
// its scale, amax / 127, would not be a normal fp32 number.
#pragma once

#include "common.cuh"
#include "sm100.cuh"

namespace dsa {
namespace rows8 {

// A thread's eight values as four packed pairs: sm_100's fp32x2 instructions
// halve the issue slots, which bound these kernels as much as memory does.
typedef uint64_t Pair;
__device__ __forceinline__ Pair pair(float lo, float hi) { return pack_f32x2(lo, hi); }
__device__ __forceinline__ Pair both(float v) { return pack_f32x2(v, v); }
__device__ __forceinline__ float added(Pair p) {
  float a, b;
  unpack_f32x2(p, a, b);
  return a + b;
}

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

__device__ __forceinline__ Pair unpack_bf16(uint32_t w) {
  return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ void values(const Raw<__nv_bfloat16>& r, Pair (&x)[4]) {
  x[0] = unpack_bf16(r.v.x);
  x[1] = unpack_bf16(r.v.y);
  x[2] = unpack_bf16(r.v.z);
  x[3] = unpack_bf16(r.v.w);
}
__device__ __forceinline__ void values(const Raw<float>& r, Pair (&x)[4]) {
  x[0] = pair(__uint_as_float(r.v.x), __uint_as_float(r.v.y));
  x[1] = pair(__uint_as_float(r.v.z), __uint_as_float(r.v.w));
  x[2] = pair(__uint_as_float(r.w.x), __uint_as_float(r.w.y));
  x[3] = pair(__uint_as_float(r.w.z), __uint_as_float(r.w.w));
}
// The codes, without their scale, and without a conversion instruction (they
// run at an eighth of the FMA rate): the byte c + 128 as the low mantissa byte
// of 2^23 is the float 2^23 + 128 + c; subtracting 2^23 + 128 is exact.
__device__ __forceinline__ void values(const Raw<int8_t>& r, Pair (&x)[4]) {
  const uint32_t w[2] = {r.v.x ^ 0x80808080u, r.v.y ^ 0x80808080u};
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const uint32_t v = w[m >> 1], k = 2 * (m & 1);
    x[m] = add_f32x2(pair(__uint_as_float(__byte_perm(v, 0x4b000000u, 0x7440u + k)),
                          __uint_as_float(__byte_perm(v, 0x4b000000u, 0x7441u + k))), both(-8388736.0f));
  }
}
// What the values have to be multiplied by.
template <typename T>
__device__ __forceinline__ float scale_of(const Raw<T>&) { return 1.f; }
__device__ __forceinline__ float scale_of(const Raw<int8_t>& r) { return r.scale; }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(Pair p) {
  float a, b;
  unpack_f32x2(p, a, b);
  return pack_bf16(a, b);
}
__device__ __forceinline__ void store(__nv_bfloat16* p, const Pair (&x)[4]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0]), pack_bf16(x[1]), pack_bf16(x[2]), pack_bf16(x[3]));
}
__device__ __forceinline__ void store(float* p, const Pair (&x)[4]) {
  float v[8];
#pragma unroll
  for (int m = 0; m < 4; ++m) unpack_f32x2(x[m], v[2 * m], v[2 * m + 1]);
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// The same loads into shared memory, asynchronously (16-byte slots, one or two
// per load, kThreads apart): what is in flight costs no registers, and as
// every thread reads back only its own slots, no barrier is needed.
template <typename T> struct Slots { static constexpr int kCount = sizeof(T) == 4 ? 2 : 1; };

__device__ __forceinline__ uint32_t shared_at(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// Sum over the TPR (8 or 16) neighbouring threads of a row, in all of them.
template <int TPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < TPR; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Bits of the largest magnitude of eight values (integer order is the order
// of magnitudes, NaN above infinity).
__device__ __forceinline__ uint32_t top_bits(const Raw<__nv_bfloat16>& r) {
  constexpr uint32_t kMag = 0x7fff7fffu;
  const uint32_t m = __vmaxu2(__vmaxu2(r.v.x & kMag, r.v.y & kMag), __vmaxu2(r.v.z & kMag, r.v.w & kMag));
  return max(m << 16, m & 0xffff0000u);
}
__device__ __forceinline__ uint32_t top_bits(const Raw<float>& r) {
  constexpr uint32_t kMag = 0x7fffffffu;
  return max(max(max(r.v.x & kMag, r.v.y & kMag), max(r.v.z & kMag, r.v.w & kMag)),
             max(max(r.w.x & kMag, r.w.y & kMag), max(r.w.z & kMag, r.w.w & kMag)));
}

// Over the row's threads.
template <int TPR>
__device__ __forceinline__ uint32_t row_top(uint32_t top) {
#pragma unroll
  for (int o = 1; o < TPR; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  return top;
}

// Scales of U rows, from the rows' largest magnitudes (see above): thread 2 u of
// a row's threads returns row u's scale, amax / 127, and inv[u] = 127 / amax is
// for all of them.  (2 U threads make one division each, so that 2 U divisions
// cost the issue slots of one.)
template <int TPR, int U>
__device__ __forceinline__ float scales8(const uint32_t (&top)[U], int sub, float (&inv)[U]) {
  static_assert(2 * U <= TPR);
  uint32_t t = top[0];
#pragma unroll
  for (int u = 1; u < U; ++u) t = (sub >> 1) == u ? top[u] : t;
  const float amax = __uint_as_float(t);
  const bool some = t < 0x7f800000u && amax >= 0x1p-119f;
  float q = some ? __fdiv_rn(sub & 1 ? 127.0f : amax, sub & 1 ? amax : 127.0f) : 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) inv[u] = __shfl_sync(0xffffffffu, q, 2 * u + 1, TPR);
  return t >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : q;
}

// A thread's codes of a row with inv = 127 / amax.
__device__ __forceinline__ uint2 encode8(const Pair (&x)[4], float inv) {
  // round-half-even by the adder: 1.5 * 2^23 + v keeps the integer nearest to v
  // (ties to even) in its low bits, here the low byte as |v| <= 127
  uint32_t t[8];
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    float a, b;  // (not packed: the product has to be rounded before the sum)
    unpack_f32x2(x[m], a, b);
    t[2 * m] = __float_as_uint(__fadd_rn(__fmul_rn(a, inv), 12582912.0f));
    t[2 * m + 1] = __float_as_uint(__fadd_rn(__fmul_rn(b, inv), 12582912.0f));
  }
  return make_uint2(
      __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410),
      __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410));
}

}  // namespace rows8
}  // namespace dsa
