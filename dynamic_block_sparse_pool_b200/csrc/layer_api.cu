// C ABI of the calls around the attention (declared in include/dsa.h): the
// per-head norm with rotation, the window attention and the 8-bit activation
// rows.  Argument checks and dispatch; no call allocates device memory or
// synchronises the host.
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "dsa.h"
#include "norm_rope.cuh"

namespace dsa {
dsa_status api_checked_device(unsigned** err_word);
void api_set_last_error(const char* msg);
}  // namespace dsa

namespace {

dsa_status fail(dsa_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
dsa_status fail(dsa_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  dsa::api_set_last_error(buf);
  return st;
}

dsa_status launched(cudaError_t e, const char* where) {
  return e == cudaSuccess ? DSA_OK : fail(DSA_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool known(dsa_dtype dt) { return dt == DSA_F32 || dt == DSA_BF16; }

// Strides of token-major rows: non-negative multiples of `unit` elements.
dsa_status check_strides(const int64_t* st, int unit, const char* what) {
  for (int i = 0; i < 6; ++i)
    if (st[i] < 0 || st[i] % unit)
      return fail(DSA_ERR_INVALID_ARG, "%s[%d] = %lld: strides must be non-negative multiples of %d elements",
                  what, i, (long long)st[i], unit);
  return DSA_OK;
}

// What the forward and the backward of the norm with rotation share.
dsa_status check_norm_rope(const void* xq, const void* xk, const float* xq_scale,
                           const float* xk_scale, const int64_t* x_strides, dsa_dtype dt, int B,
                           int N, int Hq, int Hk, int D, const float* wq, const float* wk,
                           float eps, const float* table, const int32_t* pos, int pos_per_batch,
                           const int32_t* axes, int halves) {
  if (!xq || !xk || !x_strides || !table || !pos || !axes)
    return fail(DSA_ERR_INVALID_ARG, "null xq, xk, x_strides, table, pos or axes");
  if (!known(dt)) return fail(DSA_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
  if ((xq_scale == nullptr) != (xk_scale == nullptr))
    return fail(DSA_ERR_INVALID_ARG, "xq_scale and xk_scale must both be set or both be NULL");
  if (B < 1 || N < 1) return fail(DSA_ERR_INVALID_ARG, "B and N must be >= 1 (got %d, %d)", B, N);
  if ((long long)B * N > INT_MAX) return fail(DSA_ERR_INVALID_ARG, "B*N exceeds 2^31 - 1");
  if (Hq < 1 || Hk < 1 || Hq > 65535 || Hk > 65535)
    return fail(DSA_ERR_INVALID_ARG, "Hq and Hk must be 1..65535 (got %d, %d)", Hq, Hk);
  if (D != 64 && D != 128) return fail(DSA_ERR_INVALID_ARG, "head_dim D must be 64 or 128 (got %d)", D);
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(DSA_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if ((pos_per_batch != 0 && pos_per_batch != 1) || (halves != 0 && halves != 1))
    return fail(DSA_ERR_INVALID_ARG, "pos_per_batch and halves must be 0 or 1");
  long long sum = 0, entries = 0;
  for (int a = 0; a < 3; ++a) {
    if (axes[a] < 0 || (axes[a] > 0 && axes[3 + a] < 1))
      return fail(DSA_ERR_INVALID_ARG, "axis %d: %d pairs over a table of %d positions", a, axes[a], axes[3 + a]);
    sum += axes[a];
    if (axes[a] > 0) entries += (long long)axes[a] * axes[3 + a];
  }
  if (sum > D / 2) return fail(DSA_ERR_INVALID_ARG, "%lld rotated pairs exceed D/2 = %d", sum, D / 2);
  if (entries > (1 << 30)) return fail(DSA_ERR_INVALID_ARG, "the rotation tables exceed 2^30 entries");
  const size_t a = xq_scale ? 8 : 16;
  if (!aligned(xq, a) || !aligned(xk, a) || !aligned(xq_scale, 4) || !aligned(xk_scale, 4) ||
      !aligned(wq, 4) || !aligned(wk, 4) || !aligned(table, 8) || !aligned(pos, 4))
    return fail(DSA_ERR_INVALID_ARG, "misaligned pointer");
  return check_strides(x_strides, xq_scale ? 8 : dt == DSA_BF16 ? 8 : 4, "x_strides");
}

dsa::RopeArgs rope_args(const float* table, const int32_t* pos, int pos_per_batch, int N,
                        const int32_t* axes) {
  dsa::RopeArgs r;
  r.table = reinterpret_cast<const float2*>(table);
  r.pos = pos;
  r.pos_bstride = pos_per_batch ? 3ll * N : 0;
  for (int a = 0; a < 3; ++a) {
    r.pairs[a] = axes[a];
    r.len[a] = axes[a] > 0 ? axes[3 + a] : 0;
  }
  return r;
}

}  // namespace

extern "C" {

dsa_status dsa_rope_table(int positions, int pairs, float theta, float* table) {
  dsa::api_set_last_error("");
  if (!table) return fail(DSA_ERR_INVALID_ARG, "null table");
  if (positions < 1 || pairs < 1 || pairs > 64)
    return fail(DSA_ERR_INVALID_ARG, "need positions >= 1 and pairs in 1..64 (got %d, %d)", positions, pairs);
  if ((long long)positions * pairs > (1 << 30)) return fail(DSA_ERR_INVALID_ARG, "the table exceeds 2^30 entries");
  if (!(theta > 0.f) || !std::isfinite(theta)) return fail(DSA_ERR_INVALID_ARG, "theta must be finite and > 0");
  for (int i = 0; i < pairs; ++i) {
    const double f = std::pow((double)theta, -(double)i / pairs);
    for (long long p = 0; p < positions; ++p) {
      table[(p * pairs + i) * 2] = (float)std::cos((double)p * f);
      table[(p * pairs + i) * 2 + 1] = (float)std::sin((double)p * f);
    }
  }
  return DSA_OK;
}

dsa_status dsa_qk_norm_rope(const void* xq, const void* xk, const float* xq_scale,
                            const float* xk_scale, const int64_t* x_strides, dsa_dtype dt, int B,
                            int N, int Hq, int Hk, int D, const float* wq, const float* wk,
                            float eps, const float* table, const int32_t* pos, int pos_per_batch,
                            const int32_t* axes, int halves, void* q, void* k, int8_t* xq8,
                            float* xq8_scale, int8_t* xk8, float* xk8_scale, void* stream) {
  dsa::api_set_last_error("");
  dsa_status st = check_norm_rope(xq, xk, xq_scale, xk_scale, x_strides, dt, B, N, Hq, Hk, D, wq, wk,
                                  eps, table, pos, pos_per_batch, axes, halves);
  if (st != DSA_OK) return st;
  if (!q || !k) return fail(DSA_ERR_INVALID_ARG, "null q or k");
  const int saves = (xq8 != nullptr) + (xk8 != nullptr) + (xq8_scale != nullptr) + (xk8_scale != nullptr);
  if (saves != 0 && saves != 4)
    return fail(DSA_ERR_INVALID_ARG, "xq8, xq8_scale, xk8 and xk8_scale must all be set or all be NULL");
  if (saves && xq_scale) return fail(DSA_ERR_INVALID_ARG, "8-bit rows are already given: nothing to save");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(xq8, 8) || !aligned(xk8, 8) ||
      !aligned(xq8_scale, 4) || !aligned(xk8_scale, 4))
    return fail(DSA_ERR_INVALID_ARG, "q and k must be 16-byte aligned, codes 8-byte, scales 4-byte aligned");
  dsa::NormRopeFwd f;
  if ((st = dsa::api_checked_device(&f.err)) != DSA_OK) return st;
  f.xq = xq; f.xk = xk; f.xq_scale = xq_scale; f.xk_scale = xk_scale;
  f.qb = x_strides[0]; f.qn = x_strides[1]; f.qh = x_strides[2];
  f.kb = x_strides[3]; f.kn = x_strides[4]; f.kh = x_strides[5];
  f.bf16 = dt == DSA_BF16;
  f.B = B; f.N = N; f.Hq = Hq; f.Hk = Hk; f.D = D;
  f.wq = wq; f.wk = wk; f.eps = eps;
  f.rope = rope_args(table, pos, pos_per_batch, N, axes);
  f.halves = halves != 0;
  f.q = q; f.k = k;
  f.xq8 = xq8; f.xk8 = xk8; f.xq8_scale = xq8_scale; f.xk8_scale = xk8_scale;
  return launched(dsa::launch_qk_norm_rope(f, static_cast<cudaStream_t>(stream)), "qk_norm_rope launch");
}

size_t dsa_qk_norm_rope_bwd_workspace_size(int D) {
  return D == 64 || D == 128 ? (size_t)dsa::kNormRopeBwdCtas * 2 * D * sizeof(float) : 0;
}

dsa_status dsa_qk_norm_rope_bwd(const void* dq, const void* dk, const void* xq, const void* xk,
                                const float* xq_scale, const float* xk_scale,
                                const int64_t* x_strides, dsa_dtype dt, int B, int N, int Hq,
                                int Hk, int D, const float* wq, const float* wk, float eps,
                                const float* table, const int32_t* pos, int pos_per_batch,
                                const int32_t* axes, int halves, void* dxq, void* dxk,
                                const int64_t* dx_strides, float* dwq, float* dwk,
                                void* workspace, size_t ws_bytes, void* stream) {
  dsa::api_set_last_error("");
  dsa_status st = check_norm_rope(xq, xk, xq_scale, xk_scale, x_strides, dt, B, N, Hq, Hk, D, wq, wk,
                                  eps, table, pos, pos_per_batch, axes, halves);
  if (st != DSA_OK) return st;
  if (!dq || !dk || !dxq || !dxk || !dx_strides || !workspace)
    return fail(DSA_ERR_INVALID_ARG, "null dq, dk, dxq, dxk, dx_strides or workspace");
  if ((st = check_strides(dx_strides, dt == DSA_BF16 ? 8 : 4, "dx_strides")) != DSA_OK) return st;
  if (!aligned(dq, 16) || !aligned(dk, 16) || !aligned(dxq, 16) || !aligned(dxk, 16) ||
      !aligned(workspace, 16) || !aligned(dwq, 4) || !aligned(dwk, 4))
    return fail(DSA_ERR_INVALID_ARG, "gradients and workspace must be 16-byte aligned, dwq and dwk 4-byte aligned");
  if (ws_bytes < dsa_qk_norm_rope_bwd_workspace_size(D))
    return fail(DSA_ERR_INVALID_ARG, "workspace of %zu bytes is below the %zu needed", ws_bytes,
                dsa_qk_norm_rope_bwd_workspace_size(D));
  dsa::NormRopeBwd f;
  if ((st = dsa::api_checked_device(&f.err)) != DSA_OK) return st;
  f.gq = dq; f.gk = dk;
  f.xq = xq; f.xk = xk; f.xq_scale = xq_scale; f.xk_scale = xk_scale;
  f.qb = x_strides[0]; f.qn = x_strides[1]; f.qh = x_strides[2];
  f.kb = x_strides[3]; f.kn = x_strides[4]; f.kh = x_strides[5];
  f.bf16 = dt == DSA_BF16;
  f.B = B; f.N = N; f.Hq = Hq; f.Hk = Hk; f.D = D;
  f.wq = wq; f.wk = wk; f.eps = eps;
  f.rope = rope_args(table, pos, pos_per_batch, N, axes);
  f.halves = halves != 0;
  f.dxq = dxq; f.dxk = dxk;
  f.dqb = dx_strides[0]; f.dqn = dx_strides[1]; f.dqh = dx_strides[2];
  f.dkb = dx_strides[3]; f.dkn = dx_strides[4]; f.dkh = dx_strides[5];
  f.dwq = dwq; f.dwk = dwk;
  f.part = static_cast<float*>(workspace);
  return launched(dsa::launch_qk_norm_rope_bwd(f, static_cast<cudaStream_t>(stream)), "qk_norm_rope_bwd launch");
}

static dsa_status check_rows8(const void* x, dsa_dtype dt, size_t rows, int D, const void* codes,
                              const float* scales) {
  if (!x || !codes || !scales) return fail(DSA_ERR_INVALID_ARG, "null x, codes or scales");
  if (!known(dt)) return fail(DSA_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
  if (D != 64 && D != 128) return fail(DSA_ERR_INVALID_ARG, "head_dim D must be 64 or 128 (got %d)", D);
  if (rows < 1 || rows > (1ull << 36)) return fail(DSA_ERR_INVALID_ARG, "rows must be 1..2^36 (got %zu)", rows);
  if (!aligned(x, 16) || !aligned(codes, 8) || !aligned(scales, 4))
    return fail(DSA_ERR_INVALID_ARG, "x must be 16-byte aligned, codes 8-byte, scales 4-byte aligned");
  return DSA_OK;
}

dsa_status dsa_pack8(const void* x, dsa_dtype dt, size_t rows, int D, int8_t* codes,
                     float* scales, void* stream) {
  dsa::api_set_last_error("");
  dsa_status st = check_rows8(x, dt, rows, D, codes, scales);
  unsigned* err = nullptr;
  if (st != DSA_OK || (st = dsa::api_checked_device(&err)) != DSA_OK) return st;
  return launched(dsa::launch_pack8(x, dt == DSA_BF16, (long long)rows, D, codes, scales,
                                    static_cast<cudaStream_t>(stream)), "pack8 launch");
}

dsa_status dsa_unpack8(const int8_t* codes, const float* scales, dsa_dtype dt, size_t rows, int D,
                       void* x, void* stream) {
  dsa::api_set_last_error("");
  dsa_status st = check_rows8(x, dt, rows, D, codes, scales);
  unsigned* err = nullptr;
  if (st != DSA_OK || (st = dsa::api_checked_device(&err)) != DSA_OK) return st;
  return launched(dsa::launch_unpack8(codes, scales, dt == DSA_BF16, (long long)rows, D, x,
                                      static_cast<cudaStream_t>(stream)), "unpack8 launch");
}

}  // extern "C"
