// C ABI of the calls around the attention (declared in include/dsa.h): the
// per-head norm with rotation, the window attention and the 8-bit activation
// rows.  Argument checks and dispatch; no call allocates device memory or
// synchronises the host.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "dsa.h"
#include "norm_rope.cuh"
#include "window_attn.cuh"

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
  if (e == cudaSuccess) return DSA_OK;
  cudaGetLastError();  // reported here: the next call's launch shall not find it
  return fail(DSA_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

dsa_status sm_count(int* n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  return launched(e, "cudaDeviceGetAttribute");
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
  if ((long long)B * N > INT_MAX - 65536) return fail(DSA_ERR_INVALID_ARG, "B*N exceeds 2^31 - 65537");
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

dsa_status check_heads(int B, int H, int Hk, int D, float scale, int sink, dsa_dtype dt) {
  if (!known(dt)) return fail(DSA_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
  if (B < 1 || H < 1 || Hk < 1) return fail(DSA_ERR_INVALID_ARG, "B, H, Hk must be >= 1 (got %d, %d, %d)", B, H, Hk);
  if ((long long)B * H > 65535) return fail(DSA_ERR_INVALID_ARG, "B*H = %lld exceeds 65535", (long long)B * H);
  if (H % Hk) return fail(DSA_ERR_INVALID_ARG, "H = %d must be a multiple of Hk = %d", H, Hk);
  if (D != 64 && D != 128) return fail(DSA_ERR_INVALID_ARG, "head_dim D must be 64 or 128 (got %d)", D);
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(DSA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (sink < 0) return fail(DSA_ERR_INVALID_ARG, "sink must be >= 0 (got %d)", sink);
  return DSA_OK;
}

int bound(int v) { return v < 0 || v > dsa::Window::kNoBound ? dsa::Window::kNoBound : v; }

// Checks and arguments that the window attention's passes share.
dsa_status window_shape(dsa::WindowAttn& a, dsa_dtype dt, int B, int H, int Hk, int Nq, int Nk, int D, float scale,
                        int q_offset, int left, int right, int sink) {
  dsa_status st = check_heads(B, H, Hk, D, scale, sink, dt);
  if (st != DSA_OK) return st;
  if (Nq < 1 || Nk < 1 || Nq > (1 << 27) || Nk > (1 << 27))
    return fail(DSA_ERR_INVALID_ARG, "Nq and Nk must be 1..2^27 (got %d, %d)", Nq, Nk);
  if (q_offset > (1 << 28) || q_offset < -(1 << 28))
    return fail(DSA_ERR_INVALID_ARG, "q_offset must be within 2^28 of 0 (got %d)", q_offset);
  const long long tiles = (std::max(Nq, Nk) + 63ll) / 64;
  if ((long long)B * H * tiles > INT_MAX) return fail(DSA_ERR_INVALID_ARG, "too many query or key tiles");
  a = {};
  a.B = B; a.H = H; a.Hk = Hk; a.D = D;
  a.w = {Nq, Nk, q_offset, bound(left), bound(right), std::min(sink, Nk)};
  a.scale = scale;
  return DSA_OK;
}

dsa_status window_args(dsa::WindowAttn& a, const void* q, const void* k, const void* v, dsa_dtype dt, int B, int H,
                       int Hk, int Nq, int Nk, int D, float scale, int q_offset, int left, int right, int sink) {
  dsa_status st = window_shape(a, dt, B, H, Hk, Nq, Nk, D, scale, q_offset, left, right, sink);
  if (st != DSA_OK) return st;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16))
    return fail(DSA_ERR_INVALID_ARG, "q, k and v must be 16-byte aligned");
  a.q = q; a.k = k; a.v = v;
  if ((st = dsa::api_checked_device(&a.err)) != DSA_OK) return st;
  return sm_count(&a.num_sms);
}

size_t delta_bytes(const dsa::WindowAttn& a) { return ((size_t)a.B * a.H * a.w.Nq * sizeof(float) + 15) / 16 * 16; }

size_t window_bwd_bytes(const dsa::WindowAttn& a, dsa_dtype dt) {
  if (dt == DSA_F32) return delta_bytes(a) + dsa::simt_share_floats(a.B, a.H, a.Hk, a.w, a.D) * sizeof(float);
  const size_t slots = dsa::bwd_cut(a.B, a.H, a.Hk, a.w).slots();
  return delta_bytes(a) + slots * 2 * 128 * a.D * sizeof(float);
}

}  // namespace

extern "C" {

dsa_status dsa_window_attn_fwd(const void* q, const void* k, const void* v, dsa_dtype dt, int B,
                               int H, int Hk, int Nq, int Nk, int D, float scale, int q_offset,
                               int left, int right, int sink, void* out, float* lse,
                               void* stream) {
  dsa::api_set_last_error("");
  if (!q || !k || !v || !out) return fail(DSA_ERR_INVALID_ARG, "null q, k, v or out");
  if (!aligned(out, 16) || !aligned(lse, 4))
    return fail(DSA_ERR_INVALID_ARG, "out must be 16-byte aligned, lse 4-byte aligned");
  dsa::WindowAttn a;
  dsa_status st = window_args(a, q, k, v, dt, B, H, Hk, Nq, Nk, D, scale, q_offset, left, right, sink);
  if (st != DSA_OK) return st;
  a.out = out;
  a.lse = lse;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const char* why = nullptr;
  const cudaError_t e = dt == DSA_BF16 ? dsa::launch_window_fwd_sm100(a, s, &why) : dsa::launch_window_fwd_simt(a, s);
  if (e != cudaSuccess && why) return fail(DSA_ERR_CUDA, "window_attn_fwd: %s", why);
  return launched(e, "window_attn_fwd launch");
}

size_t dsa_window_attn_bwd_workspace_size(dsa_dtype dt, int B, int H, int Hk, int Nq, int Nk, int D, int q_offset,
                                          int left, int right, int sink) {
  dsa::api_set_last_error("");
  dsa::WindowAttn a;
  if (window_shape(a, dt, B, H, Hk, Nq, Nk, D, 1.f, q_offset, left, right, sink) != DSA_OK) return 0;
  return window_bwd_bytes(a, dt);
}

dsa_status dsa_window_attn_bwd(const void* q, const void* k, const void* v, const void* out,
                               const void* dout, const float* lse, dsa_dtype dt, int B, int H,
                               int Hk, int Nq, int Nk, int D, float scale, int q_offset, int left,
                               int right, int sink, void* dq, void* dk, void* dv, void* workspace,
                               size_t ws_bytes, void* stream) {
  dsa::api_set_last_error("");
  if (!q || !k || !v || !out || !dout || !lse || !dq || !dk || !dv || !workspace)
    return fail(DSA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(out, 16) || !aligned(dout, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) ||
      !aligned(workspace, 16) || !aligned(lse, 4))
    return fail(DSA_ERR_INVALID_ARG, "tensors and workspace must be 16-byte aligned, lse 4-byte aligned");
  dsa::WindowAttn a;
  dsa_status st = window_args(a, q, k, v, dt, B, H, Hk, Nq, Nk, D, scale, q_offset, left, right, sink);
  if (st != DSA_OK) return st;
  if (ws_bytes < window_bwd_bytes(a, dt))
    return fail(DSA_ERR_INVALID_ARG, "workspace of %zu bytes is below the %zu needed", ws_bytes,
                window_bwd_bytes(a, dt));
  a.o = out; a.dout = dout;
  a.lse = const_cast<float*>(lse);
  a.dq = dq; a.dk = dk; a.dv = dv;
  a.delta = static_cast<float*>(workspace);
  a.shares = a.delta + delta_bytes(a) / sizeof(float);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const char* why = nullptr;
  cudaError_t e = dsa::launch_row_delta(out, dout, dt == DSA_BF16, (long long)B * H * Nq, D, a.delta, s);
  if (e == cudaSuccess)
    e = dt == DSA_BF16 ? dsa::launch_window_bwd_sm100(a, s, &why) : dsa::launch_window_bwd_simt(a, s);
  if (e != cudaSuccess && why) return fail(DSA_ERR_CUDA, "window_attn_bwd: %s", why);
  return launched(e, "window_attn_bwd launch");
}

static dsa_status check_decode(dsa_dtype dt, int B, int H, int Hk, int Nq, int cap, int D, float scale, int sink) {
  dsa_status st = check_heads(B, H, Hk, D, scale, sink, dt);
  if (st != DSA_OK) return st;
  if (Nq < 1 || Nq > 128) return fail(DSA_ERR_INVALID_ARG, "Nq must be 1..128 (got %d)", Nq);
  if (cap < 1 || cap > (1 << 27)) return fail(DSA_ERR_INVALID_ARG, "cap must be 1..2^27 (got %d)", cap);
  return DSA_OK;
}

static size_t decode_ws_bytes(const dsa::DecodePlan& p, int B, int H, int Nq, int D) {
  return p.groups == 1 ? 0 : (size_t)p.groups * B * H * Nq * (D + 2) * sizeof(float);
}

size_t dsa_window_attn_decode_workspace_size(dsa_dtype dt, int B, int H, int Hk, int Nq, int cap, int D, int left,
                                             int sink) {
  dsa::api_set_last_error("");
  if (check_decode(dt, B, H, Hk, Nq, cap, D, 1.f, sink) != DSA_OK) return 0;
  return decode_ws_bytes(dsa::decode_plan(dt == DSA_BF16, B, H, Hk, Nq, cap, D, bound(left), std::min(sink, cap)), B,
                         H, Nq, D);
}

dsa_status dsa_window_attn_decode(const void* q, const void* k, const void* v,
                                  const int64_t* kv_strides, dsa_dtype dt, int B, int H, int Hk,
                                  int Nq, int cap, int D, float scale, const int32_t* lens,
                                  int left, int sink, void* out, float* lse, void* workspace,
                                  size_t ws_bytes, void* stream) {
  dsa::api_set_last_error("");
  if (!q || !k || !v || !kv_strides || !lens || !out)
    return fail(DSA_ERR_INVALID_ARG, "null q, k, v, kv_strides, lens or out");
  dsa_status st = check_decode(dt, B, H, Hk, Nq, cap, D, scale, sink);
  if (st != DSA_OK) return st;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(lens, 4) ||
      !aligned(lse, 4) || !aligned(workspace, 16))
    return fail(DSA_ERR_INVALID_ARG, "q, k, v, out and workspace must be 16-byte aligned, lens and lse 4-byte aligned");
  if ((st = check_strides(kv_strides, dt == DSA_BF16 ? 8 : 4, "kv_strides")) != DSA_OK) return st;
  const int dims[3] = {B, Hk, cap};
  for (int i = 0; i < 6; ++i)
    if (dims[i % 3] > 1 && (kv_strides[i] < D || kv_strides[i] >= (1ll << 38)))
      return fail(DSA_ERR_INVALID_ARG, "kv_strides[%d] = %lld: rows must not overlap", i, (long long)kv_strides[i]);
  dsa::DecodeAttn a = {};
  a.B = B; a.H = H; a.Hk = Hk; a.group = H / Hk; a.Nq = Nq; a.cap = cap;
  a.scale = scale;
  a.left = bound(left);
  a.sink = std::min(sink, cap);
  const dsa::DecodePlan plan = dsa::decode_plan(dt == DSA_BF16, B, H, Hk, Nq, cap, D, a.left, a.sink);
  const size_t need = decode_ws_bytes(plan, B, H, Nq, D);
  if (need > 0 && (!workspace || ws_bytes < need))
    return fail(DSA_ERR_INVALID_ARG, "workspace of %zu bytes is below the %zu needed", workspace ? ws_bytes : 0, need);
  a.groups = plan.groups;
  a.ws = static_cast<float*>(workspace);
  a.q = q; a.k = k; a.v = v;
  for (int i = 0; i < 3; ++i) {
    a.ks[i] = kv_strides[i];
    a.vs[i] = kv_strides[3 + i];
  }
  a.lens = lens;
  a.out = out;
  a.lse = lse;
  if ((st = dsa::api_checked_device(&a.err)) != DSA_OK) return st;
  const char* why = nullptr;
  const cudaError_t e =
      dsa::launch_window_decode(a, plan, dt == DSA_BF16, D, static_cast<cudaStream_t>(stream), &why);
  if (e != cudaSuccess && why) return fail(DSA_ERR_CUDA, "window_attn_decode: %s", why);
  return launched(e, "window_attn_decode launch");
}

dsa_status dsa_rope_table(int positions, int pairs, float theta, float* table, void* stream) {
  const double base = theta;
  return dsa_rope_table_f64(positions, pairs, &base, table, stream);
}

dsa_status dsa_rope_table_f64(int positions, int pairs, const double* theta, float* table, void* stream) {
  dsa::api_set_last_error("");
  if (!table || !theta) return fail(DSA_ERR_INVALID_ARG, "null table or theta");
  if (positions < 1 || pairs < 1 || pairs > 64)
    return fail(DSA_ERR_INVALID_ARG, "need positions >= 1 and pairs in 1..64 (got %d, %d)", positions, pairs);
  if ((long long)positions * pairs > (1 << 30)) return fail(DSA_ERR_INVALID_ARG, "the table exceeds 2^30 entries");
  if (!(*theta > 0.0) || !std::isfinite(*theta)) return fail(DSA_ERR_INVALID_ARG, "theta must be finite and > 0");
  if (!aligned(table, 8)) return fail(DSA_ERR_INVALID_ARG, "table must be 8-byte aligned");
  unsigned* err = nullptr;
  const dsa_status st = dsa::api_checked_device(&err);
  if (st != DSA_OK) return st;
  return launched(dsa::launch_rope_table(positions, pairs, *theta, reinterpret_cast<float2*>(table),
                                         static_cast<cudaStream_t>(stream)), "rope_table launch");
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
  return D == 64 || D == 128 ? (size_t)dsa::kNormRopeBwdCtas * D * sizeof(float) : 0;
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
