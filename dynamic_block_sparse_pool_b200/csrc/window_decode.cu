// Window attention of a few new tokens over a cache of keys and values.
//
// Query i of Nq stands at position t = len - Nq + i of its stream and sees
// the keys u <= t with u < sink or u >= t - left (window.cuh with right = 0);
// len is read from device memory, so one captured launch serves a growing
// cache.
//
// Bound by memory: the visible keys and values are read once (2 D values per
// key for 4 D Nq H / Hk operations).  A cluster of 1, 2, 4 or 8 CTAs of four
// warps takes one key head and up to kRows of its rows (the query heads of
// the group times the new tokens), so the group shares every key that is
// read.  Every warp of the cluster takes steps of kKeys keys in turn, keeps
// its own running maximum, sum and output in registers, and the warps'
// results are joined in shared memory, then across the cluster through
// distributed shared memory: one launch, no workspace, fixed order.
//
// bf16: products on mma.sync (16 rows; at these sizes its rate is far above
// what memory feeds).  Both operands come straight from global memory in
// 16-byte loads: the order of the summed dimension is free, so lane (g, c)
// takes elements 8c .. 8c+7 of each 32 of key g's row for two k-steps, and Q
// is loaded in the same order; for P V the order of the output columns is
// free, so lane group g takes D/8 neighbouring columns of a value row and
// two rows' elements are paired by byte permutes.  While a step's softmax and
// P V run, the next step's keys are on their way.
// fp32: dot products on CUDA cores, four lanes per key; each lane group of
// four keeps the softmax of its own keys.
//
// Rows of the cache that no query sees are not read (a step's lanes past the
// end of a run read its last key again), so they may hold anything.
#include <cooperative_groups.h>

#include <algorithm>

#include "window_attn.cuh"

namespace dsa {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
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

// The warps' rows, their maxima and sums in shared memory -> the outputs.
// part: [kWarps][ROWS][D] outputs relative to m, m and l: [kWarps][ROWS].
// Warp 0's place then holds the CTA's, and each CTA of the cluster finishes
// its share of the rows from all of them.
template <typename T, int D, int ROWS>
__device__ __forceinline__ void join(float* part, float* pm, float* pl, int rows, int row0, int nq, T* out, float* lse,
                                     size_t q_rows, int group_row0) {
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
    pm[r] = m;
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
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const size_t row = q_rows + group_row0 + r;
    T* o = out + row * D + d;
    o[0] = Elem<T>::from_f(acc.x * inv);
    o[1] = Elem<T>::from_f(acc.y * inv);
    o[2] = Elem<T>::from_f(acc.z * inv);
    o[3] = Elem<T>::from_f(acc.w * inv);
    if (lse && d == 0) lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The stream's length, 0 (and reported) where it is outside [0, cap].
__device__ __forceinline__ int stream_len(const DecodeAttn& a, int b) {
  const int len = a.lens[b];
  if (len >= 0 && len <= a.cap) return len;
  if (threadIdx.x == 0) flag_error(a.err, kErrLength);
  return 0;
}

// Grid: x = cluster size * key heads of all streams, y = tiles of 16 rows.
template <int D>
__global__ void __launch_bounds__(kThreads, 2)
window_decode_mma_kernel(const DecodeAttn a) {
  constexpr int ROWS = 16, K = 16;
  constexpr int KS = D / 32;      // 16-byte loads of a key row per lane
  constexpr int NT = D / 8;       // column tiles of 8 of the output
  constexpr int VW = D / 64;      // 16-byte loads of a value row per lane
  __shared__ __align__(16) float part[kWarps * ROWS * D];
  __shared__ float pm[kWarps * ROWS], pl[kWarps * ROWS];
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = cluster.num_blocks(), rank = cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int kvh = blockIdx.x / cs, b = kvh / a.Hk, kh = kvh - b * a.Hk;
  const int all = a.group * a.Nq, row0 = blockIdx.y * ROWS, rows = min(ROWS, all - row0);
  const int len = stream_len(a, b);
  const Steps<K> st(len, a.Nq, a.left, a.sink);
  // rows of the group are contiguous in q: (head, token)
  const size_t q_rows = ((size_t)b * a.H + (size_t)kh * a.group) * a.Nq;
  const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(a.k) + b * a.ks[0] + kh * a.ks[1];
  const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(a.v) + b * a.vs[0] + kh * a.vs[1];

  uint4 qa[KS], qb[KS];  // rows g and g + 8
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (q_rows + row0) * D + 32 * s + 8 * c;
    qa[s] = g < rows ? *reinterpret_cast<const uint4*>(q + g * D) : make_uint4(0, 0, 0, 0);
    qb[s] = g + 8 < rows ? *reinterpret_cast<const uint4*>(q + (g + 8) * D) : make_uint4(0, 0, 0, 0);
  }
  const int ta = len - a.Nq + (row0 + g) % a.Nq, tb = len - a.Nq + (row0 + g + 8) % a.Nq;
  const int t_first = len - a.Nq, t_last = len - 1;
  const float sc = a.scale * kLog2e;

  float o[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  float ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;

  uint4 kr[2][KS], vr[4][VW];
  auto load_k = [&](int s) {
    int base, end;
    st.at(s, base, end);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const __nv_bfloat16* p = kp + (long long)min(base + 8 * t + g, end - 1) * a.ks[2] + 8 * c;
#pragma unroll
      for (int x = 0; x < KS; ++x) kr[t][x] = __ldcs(reinterpret_cast<const uint4*>(p + 32 * x));
    }
  };
  auto load_v = [&](int s) {
    int base, end;
    st.at(s, base, end);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int key = min(base + 2 * c + (r & 1) + 8 * (r >> 1), end - 1);
      const __nv_bfloat16* p = vp + (long long)key * a.vs[2] + NT * g;
#pragma unroll
      for (int x = 0; x < VW; ++x) vr[r][x] = __ldcs(reinterpret_cast<const uint4*>(p + 8 * x));
    }
  };
  const int stride = cs * kWarps;
  int s = rank * kWarps + warp;
  if (s < st.n) {
    load_k(s);
    load_v(s);
  }
  for (; s < st.n; s += stride) {
    float x[2][4] = {};
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        mma16816(x[t], qa[i].x, qb[i].x, qa[i].y, qb[i].y, kr[t][i].x, kr[t][i].y);
        mma16816(x[t], qa[i].z, qb[i].z, qa[i].w, qb[i].w, kr[t][i].z, kr[t][i].w);
      }
    const int next = s + stride;
    if (next < st.n) load_k(next);
    int base, end;
    st.at(s, base, end);
    const bool whole = base + K <= end && base + K - 1 <= t_first && (s < st.nf || base >= t_last - a.left);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int u = base + 8 * t + 2 * c + e;
        const bool in = u < end;
        x[t][e] = whole || (in && sees(ta, u, a.left, a.sink)) ? x[t][e] * sc : -INFINITY;
        x[t][2 + e] = whole || (in && sees(tb, u, a.left, a.sink)) ? x[t][2 + e] * sc : -INFINITY;
      }
    float na = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
    float nb = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      na = fmaxf(na, __shfl_xor_sync(0xffffffffu, na, d));
      nb = fmaxf(nb, __shfl_xor_sync(0xffffffffu, nb, d));
    }
    na = fmaxf(na, ma);
    nb = fmaxf(nb, mb);
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
    uint32_t pa[2], pb[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float p0 = exp2f(x[t][0] - ra), p1 = exp2f(x[t][1] - ra);
      const float p2 = exp2f(x[t][2] - rb), p3 = exp2f(x[t][3] - rb);
      la += p0 + p1;
      lb += p2 + p3;
      pa[t] = pack2(p0, p1);
      pb[t] = pack2(p2, p3);
    }
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      const uint32_t* v0 = reinterpret_cast<const uint32_t*>(&vr[0][w]);
      const uint32_t* v1 = reinterpret_cast<const uint32_t*>(&vr[1][w]);
      const uint32_t* v2 = reinterpret_cast<const uint32_t*>(&vr[2][w]);
      const uint32_t* v3 = reinterpret_cast<const uint32_t*>(&vr[3][w]);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int j = 8 * w + 2 * y;
        mma16816(o[j], pa[0], pb[0], pa[1], pb[1], __byte_perm(v0[y], v1[y], 0x5410), __byte_perm(v2[y], v3[y], 0x5410));
        mma16816(o[j + 1], pa[0], pb[0], pa[1], pb[1], __byte_perm(v0[y], v1[y], 0x7632),
                 __byte_perm(v2[y], v3[y], 0x7632));
      }
    }
    if (next < st.n) load_v(next);
  }
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    la += __shfl_xor_sync(0xffffffffu, la, d);
    lb += __shfl_xor_sync(0xffffffffu, lb, d);
  }
  // column tile j, column 2c + e of it is column NT (2c + e) + j of the row
  float* pw = part + warp * ROWS * D;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      pw[g * D + NT * (2 * c + e) + j] = o[j][e];
      pw[(g + 8) * D + NT * (2 * c + e) + j] = o[j][2 + e];
    }
  }
  if (c == 0) {
    pm[warp * ROWS + g] = ma;
    pm[warp * ROWS + g + 8] = mb;
    pl[warp * ROWS + g] = la;
    pl[warp * ROWS + g + 8] = lb;
  }
  join<__nv_bfloat16, D, ROWS>(part, pm, pl, rows, row0, a.Nq, static_cast<__nv_bfloat16*>(a.out), a.lse, q_rows, row0);
}

// Grid as above with tiles of 4 or 2 rows; lane (g, c): key g of a step of 8,
// elements 16 x + 4 c .. + 3 of its row.
template <int D>
constexpr int f32_rows() { return 256 / D; }  // 4 or 2: as many as registers hold

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
window_decode_f32_kernel(const DecodeAttn a) {
  constexpr int ROWS = f32_rows<D>(), K = 8, X = D / 16;
  __shared__ __align__(16) float part[kWarps * ROWS * D];
  __shared__ __align__(16) float qs[ROWS * D];
  __shared__ float pm[kWarps * ROWS], pl[kWarps * ROWS];
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = cluster.num_blocks(), rank = cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int kvh = blockIdx.x / cs, b = kvh / a.Hk, kh = kvh - b * a.Hk;
  const int all = a.group * a.Nq, row0 = blockIdx.y * ROWS, rows = min(ROWS, all - row0);
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
  for (int s = rank * kWarps + warp; s < st.n; s += cs * kWarps) {
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
      pm[warp * ROWS + r] = top;
      pl[warp * ROWS + r] = sum;
    }
  }
  join<float, D, ROWS>(part, pm, pl, rows, row0, a.Nq, static_cast<float*>(a.out), a.lse, q_rows, row0);
}

template <typename Kernel>
cudaError_t launch(Kernel kernel, const DecodeAttn& a, int rows_per, int keys, cudaStream_t s) {
  const int heads = a.B * a.Hk, tiles = ceil_div(a.group * a.Nq, rows_per);
  // Enough CTAs for two on each SM, as long as every warp keeps two steps of
  // the longest stream or more.
  const long long longest =
      a.left >= Window::kNoBound ? a.cap : std::min<long long>(a.cap, (long long)a.left + a.Nq + a.sink);
  int cs = 1;
  while (cs < 8 && (long long)heads * tiles * cs < 2 * a.num_sms && longest >= 4ll * cs * kWarps * keys) cs *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(heads * cs), (unsigned)tiles);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cs;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_window_decode(const DecodeAttn& a, bool bf16, int D, cudaStream_t s) {
  if (bf16)
    return D == 64 ? launch(window_decode_mma_kernel<64>, a, 16, 16, s)
                   : launch(window_decode_mma_kernel<128>, a, 16, 16, s);
  return D == 64 ? launch(window_decode_f32_kernel<64>, a, f32_rows<64>(), 8, s)
                 : launch(window_decode_f32_kernel<128>, a, f32_rows<128>(), 8, s);
}

}  // namespace dsa
