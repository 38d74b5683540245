// flat_list.cuh -- the split of a ragged batch's tiles over a persistent grid:
// all tiles of all (sequence, KV head) segments form one flat list, and each
// CTA takes an even share of it.  Shared by the 8-bit decode and the paged
// decode; prefix[b] holds the units (below) of a KV head of the sequences before b.
#pragma once

#include <cstdint>

namespace gqa {
namespace {

// A tile's place in the flat (sequence, KV head, tile) order.  The order is
// counted in units: a segment of nt tiles takes nt + E, its tiles and E for
// what its end costs, so that an even split of the units is an even split of
// the work however short the segments are (64 ragged segments of up to 64
// tiles a head, g = 16: 150 -> 112 us when it came in).
struct FlatWalk {
  long long u, end;  // the unit at hand; the end of the part of the range it lies in
  int b, kvh, k, nt, pos;
};
// A CTA's range of units [t0, t1).  If its last segment begins inside it and
// goes on past t1, that part [tA, t1) is done first, then the rest; the CTA
// that has the segment's next part starts with it too.  So a split segment's
// parts are all done early, and their merge goes on behind the tiles that
// follow.  (tA = t1: nothing goes first.)
struct FlatRange {
  long long t0, tA, t1;
};
// To the first tile of the next segment (b = B past the last).
template <int E>
__device__ __forceinline__ void flat_segment(FlatWalk& w, const int* prefix, const int* spos,
                                              int B, int Hkv) {
  w.u += w.nt - w.k + E;
  w.k = 0;
  if (++w.kvh < Hkv) return;
  w.kvh = 0;
  do { ++w.b; } while (w.b < B && prefix[w.b + 1] == prefix[w.b]);
  if (w.b < B) {
    w.nt = prefix[w.b + 1] - prefix[w.b] - E;
    w.pos = spos[w.b];
  }
}
// The first tile at or after unit u.
template <int E>
__device__ __forceinline__ void flat_init(FlatWalk& w, long long u, const int* prefix,
                                           const int* spos, int B, int Hkv) {
  int lo = 0, hi = B - 1;  // largest b with Hkv*prefix[b] <= u
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((long long)Hkv * prefix[mid] <= u) lo = mid; else hi = mid - 1;
  }
  const int n = prefix[lo + 1] - prefix[lo];
  const uint32_t off = (uint32_t)(u - (long long)Hkv * prefix[lo]);
  w.u = u;
  w.b = lo;
  w.nt = n - E;
  w.kvh = (int)(off / (uint32_t)n);
  w.k = (int)(off % (uint32_t)n);
  w.pos = spos[lo];
  if (w.k >= w.nt) flat_segment<E>(w, prefix, spos, B, Hkv);
}
// CTA c's range.  An even share, but a boundary inside a segment of at most
// kShortTiles tiles moves to that segment's nearer end: such a segment is not
// worth a merge through L2 (340 of one or two tiles: 18.4 -> 11.8 us).  (A
// longer segment's parts stay where the even shares put them: cta_of.)
constexpr int kShortTiles = 4;
template <int E>
__device__ __forceinline__ long long flat_boundary(long long u, long long T, const int* prefix, int B,
                                               int Hkv, long long& f0, int& n) {
  f0 = u;
  n = 0;
  if (u >= T) return T;
  int lo = 0, hi = B - 1;  // largest b with Hkv*prefix[b] <= u
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((long long)Hkv * prefix[mid] <= u) lo = mid; else hi = mid - 1;
  }
  n = prefix[lo + 1] - prefix[lo];
  const int k = (int)((uint32_t)(u - (long long)Hkv * prefix[lo]) % (uint32_t)n);
  f0 = u - k;  // the segment's first unit; its tiles are f0 .. f0+n-E-1
  if (k > 0 && n - E <= kShortTiles) return 2 * k < n ? f0 : f0 + n;
  return u;
}
// T * c / G, in 32 bits where that will do (c <= G <= 2^8 or so).
__device__ __forceinline__ long long flat_share(long long T, int c, int G) {
  return T < (1ll << 22) ? (long long)((uint32_t)T * (uint32_t)c / (uint32_t)G) : T * c / G;
}
template <int E>
__device__ __forceinline__ void flat_range(FlatRange& r, long long T, int c, int G,
                                            const int* prefix, int B, int Hkv) {
  long long f0;
  int n;
  r.t0 = flat_boundary<E>(flat_share(T, c, G), T, prefix, B, Hkv, f0, n);
  r.t1 = flat_boundary<E>(flat_share(T, c + 1, G), T, prefix, B, Hkv, f0, n);
  // tiles of the segment both before t1 (from f0 on) and behind it; before f0,
  // the units up to t0 + E may end another segment and hold no tile
  r.tA = f0 < r.t1 && r.t1 < f0 + n - E && f0 > r.t0 + E ? f0 : r.t1;
}
// The range's first tile in this order.
template <int E>
__device__ __forceinline__ void flat_start(FlatWalk& w, const FlatRange& r, const int* prefix,
                                            const int* spos, int B, int Hkv) {
  flat_init<E>(w, r.tA < r.t1 ? r.tA : r.t0, prefix, spos, B, Hkv);
  w.end = r.t1;
}
// Past the end of the part that went first: to the rest of the range.
template <int E>
__device__ __forceinline__ void flat_turn(FlatWalk& w, const FlatRange& r, const int* prefix,
                                           const int* spos, int B, int Hkv) {
  if (w.u >= w.end && w.end == r.t1 && r.tA < r.t1) {
    flat_init<E>(w, r.t0, prefix, spos, B, Hkv);
    w.end = r.tA;
  }
}
template <int E>
__device__ __forceinline__ void flat_next(FlatWalk& w, const FlatRange& r, const int* prefix,
                                           const int* spos, int B, int Hkv) {
  ++w.u;
  if (++w.k == w.nt) flat_segment<E>(w, prefix, spos, B, Hkv);
  flat_turn<E>(w, r, prefix, spos, B, Hkv);
}

}  // namespace
}  // namespace gqa
