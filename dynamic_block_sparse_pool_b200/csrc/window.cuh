// The mask of the window attention: key u is visible to the query at
// position t iff u <= t + right and (u < sink or u >= t - left), 0 <= u < Nk.
//
// For a tile of queries the visible keys lie in two runs of key tiles: the
// first ones (sinks) and the window's.  For a tile of keys the queries that
// see any of them are one run.  Both are arithmetic, so no index list is
// built or read.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace dsa {

struct Window {
  int Nq, Nk;
  int off;          // position of query 0
  int left, right;  // at most kNoBound, which bounds nothing
  int sink;

  static constexpr int kNoBound = 1 << 29;

  // keys [0, hi) are not in the query's future; keys [lo, hi) are its window
  __host__ __device__ int hi(int t) const { return max_(0, min_(Nk, t + right + 1)); }
  __host__ __device__ int lo(int t) const { return min_(max_(0, t - left), hi(t)); }

  static __host__ __device__ int min_(int a, int b) { return a < b ? a : b; }
  static __host__ __device__ int max_(int a, int b) { return a > b ? a : b; }
};

// Key tiles of BN keys that the queries [q0, q1) see: 0 .. first-1 and
// begin .. end-1 (begin >= first).
template <int BN>
struct KeyTiles {
  int first, begin, end;
  __host__ __device__ static KeyTiles none() { return {0, 0, 0}; }
  __host__ __device__ static KeyTiles of(const Window& w, int q0, int q1) {
    if (q1 <= q0) return none();
    const int t0 = w.off + q0, t1 = w.off + q1 - 1;
    const int hi = w.hi(t1), lo = Window::min_(Window::max_(0, t0 - w.left), hi);
    const int s = Window::min_(w.sink, hi);
    KeyTiles r;
    r.first = (s + BN - 1) / BN;
    r.end = (hi + BN - 1) / BN;
    r.begin = lo < hi ? Window::max_(lo / BN, r.first) : r.end;
    if (r.end < r.begin) r.end = r.begin;
    return r;
  }
  __host__ __device__ int count() const { return first + (end - begin); }
  __host__ __device__ int tile(int i) const { return i < first ? i : begin + (i - first); }
  __host__ __device__ bool has(int j) const { return j < first || (j >= begin && j < end); }
  // the tiles of two neighbouring query tiles together
  __host__ __device__ static KeyTiles join(const KeyTiles& a, const KeyTiles& b) {
    if (b.count() == 0) return a;
    if (a.count() == 0) return b;
    KeyTiles r;
    r.first = Window::max_(a.first, b.first);
    const bool wa = a.begin < a.end, wb = b.begin < b.end;
    r.begin = wa && wb ? Window::min_(a.begin, b.begin) : wa ? a.begin : b.begin;
    r.end = wa && wb ? Window::max_(a.end, b.end) : wa ? a.end : b.end;
    r.begin = Window::max_(r.begin, r.first);
    r.end = Window::max_(r.end, r.begin);
    return r;
  }
};

// Queries [q0, q1) that see any key of [k0, k1).
struct QueryRun {
  int q0, q1;
  __host__ __device__ static QueryRun of(const Window& w, int k0, int k1) {
    const int a = Window::max_(0, k0 - w.right - w.off);
    const int b = k0 < w.sink ? w.Nq : Window::min_(w.Nq, k1 - 1 + w.left - w.off + 1);
    return {a, Window::max_(a, b)};
  }
  // tiles of BM queries that the run touches
  template <int BM>
  __host__ __device__ int tiles() const { return q1 > q0 ? (q1 + BM - 1) / BM - q0 / BM : 0; }
};

// Whether every query of [q0, q1) sees every key of [k0, k1).
__host__ __device__ inline bool all_visible(const Window& w, int q0, int q1, int k0, int k1) {
  const int t0 = w.off + q0, t1 = w.off + q1 - 1;
  return k1 <= w.hi(t0) && (k0 >= t1 - w.left || k1 <= w.sink);
}

}  // namespace dsa
