// Arguments of the window attention's kernels and their launchers.
#pragma once

#include "window.cuh"

namespace dsa {

// How the pairs of a key tile (128 keys) are cut among CTAs in the bf16 dK/dV
// kernel: tiles with sinks (kind 0) and the others (kind 1) alike among
// themselves.
struct BwdChunks {
  int heads, sink_tiles;
  int chunks[2], counts[2];  // pairs of a part, parts of a tile
  __host__ __device__ bool kind(int tile) const { return tile >= sink_tiles; }
  __host__ __device__ int chunk(int tile) const { return kind(tile) ? chunks[1] : chunks[0]; }
  __host__ __device__ int parts(int tile) const { return kind(tile) ? counts[1] : counts[0]; }
  // CTAs, and what CTA i of them does: the tiles with sinks of all heads come
  // first, since what is not cut of them takes longest
  __host__ __device__ int ctas(int tiles) const {
    return heads * (sink_tiles * counts[0] + (tiles - sink_tiles) * counts[1]);
  }
  __host__ __device__ void place(int i, int tiles, int& head, int& tile, int& part) const {
    const int first = heads * sink_tiles * counts[0];
    const bool k = i >= first;
    const int n = k ? counts[1] : counts[0], per = k ? tiles - sink_tiles : sink_tiles;
    if (k) i -= first;
    part = i % n;
    i /= n;
    head = i / per;
    tile = (k ? sink_tiles : 0) + i - head * per;
  }
};
BwdChunks bwd_chunks(int B, int H, int Hk, const Window& w);

// The same with the tiles that have shares (partial sums in the workspace): of
// each kind those from the first with more than one part to the last, which few
// queries over a long past make a small run of all tiles.
struct BwdCut : BwdChunks {
  int from[2], to[2];
  __host__ __device__ int run(bool k) const { return k ? to[1] - from[1] : to[0] - from[0]; }
  __host__ __device__ bool shared(int tile) const {
    return kind(tile) ? tile >= from[1] && tile < to[1] : tile >= from[0] && tile < to[0];
  }
  // tiles of a head that have shares, and the i-th of them
  __host__ __device__ int cut_tiles() const { return run(0) + run(1); }
  __host__ __device__ int cut_tile(int i) const { return i < run(0) ? from[0] + i : from[1] + i - run(0); }
  // place of a part's share: the kinds one after the other
  __host__ __device__ size_t slot(int head, int tile, int part) const {
    const bool k = kind(tile);
    const size_t first = k ? (size_t)heads * run(0) * counts[0] : 0;
    return first + ((size_t)head * run(k) + tile - (k ? from[1] : from[0])) * parts(tile) + part;
  }
  __host__ __device__ size_t slots() const {
    return (size_t)heads * ((size_t)run(0) * counts[0] + (size_t)run(1) * counts[1]);
  }
};
BwdCut bwd_cut(int B, int H, int Hk, const Window& w);

struct WindowAttn {
  int B, H, Hk, D;
  Window w;
  float scale;
  const void *q, *k, *v;      // [B, H or Hk, Nq or Nk, D]
  void* out;                  // [B, H, Nq, D]
  float* lse;                 // [B, H, Nq]; forward: NULL if not wanted
  // backward
  const void *o, *dout;       // the forward's output and its gradient
  void *dq, *dk, *dv;
  float* delta;               // workspace, [B, H, Nq]
  float* shares;              // workspace: sums of gradient tiles that several CTAs share
  int num_sms;
  unsigned* err;
};

// Order of the query tiles (of all heads): by head, so that CTAs that run at the
// same time read overlapping windows of few heads, or by tile, the last one
// first, where the windows of all heads together fit in half of L2.  With a
// causal mask the first tiles are the shortest, and so the CTAs end together.
inline bool order_by_tile(const WindowAttn& a) {
  const int window = a.w.left + a.w.right + 256;
  return (long long)a.B * a.Hk * (a.w.Nk < window ? a.w.Nk : window) * a.D * 4 <= 60ll << 20;
}

struct DecodeAttn {
  int B, H, Hk, group, Nq, cap;
  float scale;
  int left, sink;             // left: at most Window::kNoBound
  const void *q, *k, *v;      // q [B, H, Nq, D]; k, v [B, Hk, cap, D] through strides
  long long ks[3], vs[3];     // strides of stream, head, key, in elements
  const int32_t* lens;        // [B]: keys in the cache, the new tokens' among them
  void* out;                  // [B, H, Nq, D]
  float* lse;                 // [B, H, Nq], NULL if not wanted
  int groups;                 // CTAs per head that join through the workspace
  float* ws;                  // [groups][B H Nq][D], then [groups][B H Nq] (maximum, sum)
  unsigned* err;
};

// How the keys of one head are shared: `cluster` CTAs that join on the SMs, or
// `groups` that join through the workspace (one of the two is 1).
struct DecodePlan {
  int tiles, cluster, groups;  // tiles: of a group's rows
};
DecodePlan decode_plan(bool bf16, int B, int H, int Hk, int Nq, int cap, int D, int left, int sink);

cudaError_t launch_window_decode(const DecodeAttn& a, const DecodePlan& plan, bool bf16, int D, cudaStream_t s,
                                 const char** why);

// bf16 on tcgen05
cudaError_t launch_window_fwd_sm100(const WindowAttn& a, cudaStream_t s, const char** why);
cudaError_t launch_window_bwd_sm100(const WindowAttn& a, cudaStream_t s, const char** why);
// fp32 on CUDA cores
// How the pairs of a gradient's tiles are cut into chunks, one CTA each: tiles
// [from, to) have more than `chunk` of them and leave up to `parts` partial sums
// (shares) in the workspace; the others are one chunk and need no share.
struct SimtCut {
  int chunk, parts, from, to;
  __host__ __device__ int tiles() const { return to - from; }
  __host__ __device__ bool shared(int tile) const { return tile >= from && tile < to; }
  __host__ __device__ size_t slot(int head, int tile, int part) const {
    return ((size_t)head * tiles() + tile - from) * parts + part;
  }
  __host__ __device__ size_t slots(int heads) const { return (size_t)heads * tiles() * parts; }
};
// dQ's tiles; those of dK and dV with sinks (0) and without (1).
struct SimtChunks {
  SimtCut q, k[2];
  int sink_tiles;
};
SimtChunks simt_chunks(int B, int H, int Hk, const Window& w);
size_t simt_share_floats(int B, int H, int Hk, const Window& w, int D);
cudaError_t launch_window_fwd_simt(const WindowAttn& a, cudaStream_t s);
cudaError_t launch_window_bwd_simt(const WindowAttn& a, cudaStream_t s);

}  // namespace dsa
