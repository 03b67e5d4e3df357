// Activation rows of D values held in 8 bits (rows8.cuh says how), and back.
//
// Bound by memory: one pass, each row read once and written once.  D / 8
// threads per row, eight values each, so a warp moves two rows (D = 128) or
// four (D = 64) per step with 16-byte accesses.  Measured, 3.0 million rows of
// 128 in bf16, there and back: 368 us, 6.4 TB/s of counted bytes.
#include <algorithm>

#include "rows8.cuh"

namespace dsa {
namespace {

using namespace rows8;

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // loads in flight per thread

// Grid: one CTA per kThreads / (D / 8) * kUnroll rows.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
pack8_kernel(const T* __restrict__ x, long long rows, int8_t* __restrict__ codes,
             float* __restrict__ scales) {
  constexpr int TPR = D / 8, RPC = kThreads / TPR;
  const int sub = threadIdx.x % TPR;
  const long long r0 = (long long)blockIdx.x * (RPC * kUnroll) + threadIdx.x / TPR;
  Raw<T> raw[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long r = min(r0 + u * RPC, rows - 1);
    load8(x + r * D + 8 * sub, raw[u]);
  }
  uint32_t top[kUnroll];
  float inv[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) top[u] = row_top<TPR>(top_bits(raw[u]));
  const float scale = scales8<TPR>(top, sub, inv);
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    Pair v[4];
    values(raw[u], v);
    const long long r = r0 + u * RPC;
    if (r < rows) {
      *reinterpret_cast<uint2*>(codes + r * D + 8 * sub) = encode8(v, inv[u]);
      if (sub == 2 * u) scales[r] = scale;
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
unpack8_kernel(const int8_t* __restrict__ codes, const float* __restrict__ scales, long long rows,
               T* __restrict__ x) {
  constexpr int TPR = D / 8, RPC = kThreads / TPR;
  const int sub = threadIdx.x % TPR;
  const long long r0 = (long long)blockIdx.x * (RPC * kUnroll) + threadIdx.x / TPR;
  Raw<int8_t> raw[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long r = min(r0 + u * RPC, rows - 1);
    load8(codes + r * D + 8 * sub, raw[u]);
    raw[u].scale = scales[r];
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    Pair v[4];
    values(raw[u], v);
#pragma unroll
    for (int m = 0; m < 4; ++m) v[m] = mul_f32x2(v[m], both(raw[u].scale));
    const long long r = r0 + u * RPC;
    if (r < rows) store(x + r * D + 8 * sub, v);
  }
}

template <typename T, int D>
cudaError_t pack_t(const void* x, long long rows, int8_t* codes, float* scales, cudaStream_t s) {
  const long long per = kThreads / (D / 8) * kUnroll;
  pack8_kernel<T, D><<<(unsigned)((rows + per - 1) / per), kThreads, 0, s>>>(
      static_cast<const T*>(x), rows, codes, scales);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t unpack_t(const int8_t* codes, const float* scales, long long rows, void* x,
                     cudaStream_t s) {
  const long long per = kThreads / (D / 8) * kUnroll;
  unpack8_kernel<T, D><<<(unsigned)((rows + per - 1) / per), kThreads, 0, s>>>(
      codes, scales, rows, static_cast<T*>(x));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_pack8(const void* x, bool bf16, long long rows, int D, int8_t* codes,
                         float* scales, cudaStream_t s) {
  if (bf16)
    return D == 64 ? pack_t<__nv_bfloat16, 64>(x, rows, codes, scales, s)
                   : pack_t<__nv_bfloat16, 128>(x, rows, codes, scales, s);
  return D == 64 ? pack_t<float, 64>(x, rows, codes, scales, s)
                 : pack_t<float, 128>(x, rows, codes, scales, s);
}

cudaError_t launch_unpack8(const int8_t* codes, const float* scales, bool bf16, long long rows,
                           int D, void* x, cudaStream_t s) {
  if (bf16)
    return D == 64 ? unpack_t<__nv_bfloat16, 64>(codes, scales, rows, x, s)
                   : unpack_t<__nv_bfloat16, 128>(codes, scales, rows, x, s);
  return D == 64 ? unpack_t<float, 64>(codes, scales, rows, x, s)
                 : unpack_t<float, 128>(codes, scales, rows, x, s);
}

}  // namespace dsa
