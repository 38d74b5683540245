// kv8_decode.cu -- split-KV decode attention over the 8-bit cache (e4m3 codes
// with a power-of-two scale per block of rows, KV head and operand), over all
// rows up to each position or over the rows of listed blocks only.
//
// For sequence b, query head h and KV head h/g, over the attended rows j:
//   s_j   = log2(e) scale * ks_j * (q . k8_j)    ks_j, vs_j: the scales of j's block
//   w_j   = 2^(s_j - M),  M = max_j (s_j + log2 vs_j)
//   out   = sum_j (w_j vs_j) v8_j / sum_j w_j
// which is softmax(s) (vs v8) relative to the row that contributes most, not
// the one that weighs most: w_j vs_j <= 1 enters the product on the scale of
// what it contributes, so fp16 parts carry it whatever the blocks' scales are.
// The sum of the w_j stays in fp32 and in range: with scales of
// 2^-60 to 2^60 its largest lies between 2^-60 and 2^60 of M, and a factor
// between two maxima, as far as 2^-120 and more, comes in two halves (moved):
// in one it would be zero below 2^-126, and weight lost with it.
//
// Bound by memory: a row costs 256 bytes for K and V, half of the bf16
// cache's.  4.3 GB (B=256, g=8) take 599 to 608 us, 7.2 TB/s; 268 MB (B=32) 45 to
// 47 us at g <= 8 and 54 at g = 16.  How:
//  * 128-row tiles (32 KB for K and V) stream through a shared-memory ring by
//    tiled TMA copies (128-byte swizzle: a row of codes is exactly one
//    swizzle span) issued by one producer warp; another fetches each 16-row
//    slice's scales, four tiles at a time, and leaves them beside the tile,
//    with flags for where a segment starts and ends.  The query rows come with
//    a segment's first tile.
//  * 8 consumer warps take 16 rows each.  e4m3 -> fp16 is exact and one
//    conversion instruction per two values; both products run on warp-level
//    MMAs (m16n8k16, fp16 in, fp32 out) with rows or dims as M and the heads
//    as N, so a KV head's g heads share one conversion of its codes.  q is
//    scaled per head by a power of two into fp16 (its 8 bits fit).
//  * The order of the dims in q.k and of the rows in both products is free, so
//    K's 16-byte pieces feed the A operand as they are, and V comes through
//    transposing 8-bit matrix loads; no bank conflicts, no code moved between
//    lanes.  The conversions are what the warps spend most of their issue
//    slots on (96 of about 270 instructions a slice).
//  * A flat list of all tiles is split evenly over the grid (one CTA per SM).
//    At a segment's end the consumers leave their partials in shared memory
//    and go on; two further warps merge them (512 x 8 segments of one tile:
//    55 -> 44 us).  A segment split over CTAs is merged by the CTA that
//    arrives last, in CTA order, so results do not depend on timing; short
//    ones are not split.  The last segment is the consumers' own to merge, and
//    its other part is fetched while they finish it (g = 8: 50 -> 46 us, g = 16:
//    58 -> 54).  For few segments a thread-block cluster takes each
//    (kv8_cluster.cuh).
#include <cooperative_groups.h>

#include <atomic>
#include <mutex>

#include "fp8.cuh"
#include "internal.h"
#include "decode_params.h"
#include "tcgen05.cuh"
#include "warp_ops.cuh"

namespace gqa {

namespace {

constexpr int kD = kDecodeD;
constexpr int kTile = 128;
constexpr int kSlices = kTile / 16;         // 16-row slices, one per consumer warp
constexpr int kOpBytes = kTile * kD;        // 16 KB per operand
constexpr int kStageBytes = 2 * kOpBytes;
constexpr int kWarps = kSlices;             // consumer warps
constexpr int kConsumers = kWarps * 32;
constexpr int kMergeThreads = 64;           // two warps that merge (flat list)
constexpr int kThreads = kConsumers + 64 + kMergeThreads;  // and two producer warps
constexpr int kClusterThreads = kConsumers + 64;
constexpr int kMaxStages = 6;
constexpr int kMiscInts = 48;  // [0] abort, [1] the last piece's other part is there, [2] last to
                               // arrive, [3] segments left over, [8..16) scan, [24..32) those
                               // segments, [32..48) the last piece
constexpr int kNoRow = 0x40000000;          // row of a slice that holds nothing
constexpr float kMInit = -3e38f;            // running maximum before any row
constexpr float kTau = 8.f;                 // the running maximum may lag by 2^kTau
constexpr float kShift = 6.f;               // probabilities sit at 2^kShift .. 2^(kShift+kTau)
constexpr int kMaxSmem = 227 * 1024;
constexpr int kWholeTiles = 4;              // segments this short are not split

constexpr int kRowsMask = 0xff;
constexpr int kStarts = 0x100;              // a piece starts with this tile
constexpr int kEnds = 0x200;                // and ends with this one
constexpr int kLast = 0x400;                // the CTA's last tile

struct SliceMeta {
  int rows;       // how many of the slice's rows count (0..16), and the tile's flags
  float ks;       // K scale
  float vs;       // V scale
  float lv;       // its log2
};

__device__ __forceinline__ SliceMeta slice_meta(int rows, float ks, float vs) {
  SliceMeta mt;
  mt.rows = rows;
  mt.ks = ks;
  mt.vs = vs;
  // log2 of a power of two comes out exact
  const uint32_t bits = __float_as_uint(vs);
  mt.lv = (float)((int)(bits >> 23) - 127) +
          log2f(__uint_as_float((bits & 0x7fffffu) | 0x3f800000u));
  return mt;
}

// A sum of weights relative to one maximum, relative to another that lies
// 2^-d away.
__device__ __forceinline__ float moved(float sum, float d) {
  const float half = ex2(0.5f * d);
  return sum * half * half;
}

struct Kv8Params {
  const uint16_t* q;
  const int32_t* positions;
  const float* k_scale;
  const float* v_scale;
  const int32_t* index;  // [B, Hkv, count], or null
  uint16_t* out;
  uint32_t* status;
  uint32_t* counters;
  float* part_ml;        // [slots][g][2]
  float* part_o;         // [slots][g][kD]
  int B, Hq, Hkv, L, g;
  int lb;                // log2 of the block's rows
  int nb;                // blocks of a cache
  int count;
  int stages;
  int test_skip;
  float qscale;          // scale * log2(e)
};

// Shared memory: the ring, per stage the q rows of a piece that starts there
// and the slices' scales, the warps' partials (twice where they are small),
// barriers, and per sequence the units before it and its position.
constexpr int kMergeRow = kD + 8;
__host__ __device__ constexpr int merge_heads(int g) { return (g + 1) & ~1; }
__host__ __device__ constexpr int merge_row(int warp, int h, int g) {
  return ((warp * 2 + (h & 1)) * (merge_heads(g) >> 1) + (h >> 1)) * kMergeRow;
}
__host__ __device__ constexpr int merge_floats(int g) {
  return kWarps * (merge_heads(g) * kMergeRow + 2 * g);
}
__host__ __device__ constexpr int merge_buffers(int g) { return g <= 8 ? 2 : 1; }
// The other part of the last piece's segment: its outputs, then (max, sum).
__host__ __device__ constexpr int other_floats(int g) { return g * (kD + 2) + (g & 1) * 2; }
inline size_t smem_bytes(int stages, int B, int g) {
  return (size_t)stages * (kStageBytes + g * kD * 2 + kSlices * sizeof(SliceMeta) + 16) + 7 * 8 +
         ((size_t)merge_buffers(g) * merge_floats(g) + other_floats(g)) * 4 + kMiscInts * 4 +
         ((size_t)2 * B + 1) * 4;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Untiled bulk copy of `bytes` (a multiple of 16) from global memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// A tile's place in the flat (sequence, KV head, tile) order.  The order is
// counted in units: a segment of nt tiles takes nt + E, its tiles and E for
// what its end costs, so that an even split of the units is an even split of
// the work however short the segments are (64 ragged segments of up to 64
// tiles a head, g = 16: 150 -> 112 us when it came in).
template <int NT> constexpr int kEndUnits = NT == 1 ? 1 : 3;
struct Walk8 {
  long long u, end;  // the unit at hand; the end of the part of the range it lies in
  int b, kvh, k, nt, pos;
};
// A CTA's range of units [t0, t1).  If its last segment begins inside it and
// goes on past t1, that part [tA, t1) is done first, then the rest; the CTA
// that has the segment's next part starts with it too.  So a split segment's
// parts are all done early, and their merge goes on behind the tiles that
// follow.  (tA = t1: nothing goes first.)
struct Range8 {
  long long t0, tA, t1;
};
// To the first tile of the next segment (b = B past the last).
template <int E>
__device__ __forceinline__ void walk8_segment(Walk8& w, const int* prefix, const int* spos,
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
__device__ __forceinline__ void walk8_init(Walk8& w, long long u, const int* prefix,
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
  if (w.k >= w.nt) walk8_segment<E>(w, prefix, spos, B, Hkv);
}
// CTA c's range.  An even share, but a boundary inside a segment of at most
// kShortTiles tiles moves to that segment's nearer end: such a segment is not
// worth a merge through L2 (340 of one or two tiles: 18.4 -> 11.8 us).  (A
// longer segment's parts stay where the even shares put them: cta_of.)
constexpr int kShortTiles = 4;
template <int E>
__device__ __forceinline__ long long boundary8(long long u, long long T, const int* prefix, int B,
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
template <int E>
__device__ __forceinline__ void range8_init(Range8& r, long long T, int c, int G,
                                            const int* prefix, int B, int Hkv) {
  long long f0;
  int n;
  r.t0 = boundary8<E>(T * c / G, T, prefix, B, Hkv, f0, n);
  r.t1 = boundary8<E>(T * (c + 1) / G, T, prefix, B, Hkv, f0, n);
  // tiles of the segment both before t1 (from f0 on) and behind it; before f0,
  // the units up to t0 + E may end another segment and hold no tile
  r.tA = f0 < r.t1 && r.t1 < f0 + n - E && f0 > r.t0 + E ? f0 : r.t1;
}
// The range's first tile in this order.
template <int E>
__device__ __forceinline__ void walk8_start(Walk8& w, const Range8& r, const int* prefix,
                                            const int* spos, int B, int Hkv) {
  walk8_init<E>(w, r.tA < r.t1 ? r.tA : r.t0, prefix, spos, B, Hkv);
  w.end = r.t1;
}
// Past the end of the part that went first: to the rest of the range.
template <int E>
__device__ __forceinline__ void walk8_turn(Walk8& w, const Range8& r, const int* prefix,
                                           const int* spos, int B, int Hkv) {
  if (w.u >= w.end && w.end == r.t1 && r.tA < r.t1) {
    walk8_init<E>(w, r.t0, prefix, spos, B, Hkv);
    w.end = r.tA;
  }
}
template <int E>
__device__ __forceinline__ void walk8_next(Walk8& w, const Range8& r, const int* prefix,
                                           const int* spos, int B, int Hkv) {
  ++w.u;
  if (++w.k == w.nt) walk8_segment<E>(w, prefix, spos, B, Hkv);
  walk8_turn<E>(w, r, prefix, spos, B, Hkv);
}

// 16 rows x 16 codes of two 16-code columns, transposed (lane l gives the
// address of row l % 16 of column block l / 16): r[2j] holds, for code c of
// block j (lane 4c + t), rows 4t .. 4t+3, and r[2j+1] the same for code c + 8.
__device__ __forceinline__ void ldmatrix_codes(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// One consumer warp: 16 rows of a tile for one KV head's g <= 8*NT heads.
// Lane 4c + t.
//  * S = K q^T: MMA row c is slice row key(c) = 4*(c/2) + c%2, row c+8 is
//    key(c) + 2, columns the heads.  MMA step w takes dims 32t + 4w .. +3 of
//    every lane t, so a lane's 32 bytes of a row are its operand and q is held
//    to match.
//  * P^T by 8x8 transposes: lane t gets rows 4t, 4t+1 and 4t+2, 4t+3.
//  * O^T += V^T P^T: the transposing matrix loads put those four rows' codes of
//    one dim in one register; MMA block i holds dims 16i + c (row c) and
//    16i + 8 + c (row c+8).
template <int NT>
struct Consumer8 {
  static constexpr bool kTwoParts = NT == 1;  // of a probability
  uint32_t qb[NT][8][2];
  float o[NT][8][4];
  float m[NT][2], l[NT][2], qk[NT][2];
  int c, t;

  // the g query rows of the segment, in shared memory
  __device__ __forceinline__ void load_q(const uint8_t* qs, int g, float qscale) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int h = 8 * n + c;
      uint4 u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        u[i] = h < g ? lds128(qs + h * (kD * 2) + 64 * t + 16 * i) : make_uint4(0u, 0u, 0u, 0u);
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w)
          amax = fmax3(amax, fabsf(bf16lo(word(u[i], w))), fabsf(bf16hi(word(u[i], w))));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // q * 2^(7-ex) lies below 2^8: exact in fp16 down to 2^-22 of the
      // head's largest element, and off by 2^-33 of it below
      const int ex = max((int)(__float_as_uint(amax) >> 23) - 127, -119);
      const float f = __uint_as_float((uint32_t)(127 + 7 - ex) << 23);
      const float un = __uint_as_float((uint32_t)(127 - 7 + ex) << 23) * qscale;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t x = word(u[i], w);
          qb[n][2 * i + (w >> 1)][w & 1] = pack_f16x2(bf16lo(x) * f, bf16hi(x) * f);
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) qk[n][e] = __shfl_sync(0xffffffffu, un, 4 * (2 * t + e));
    }
  }
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[n][e] = kMInit;
        l[n][e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[n][i][k] = 0.f;
    }
  }
  // 16 rows at Ks, Vs (the slice's first row in the tile), of which the
  // first `rows` count (rows >= 1); the others may hold anything.  FULL: all
  // of them count, and nothing is masked.
  __device__ __forceinline__ void slice(const uint8_t* Ks, const uint8_t* Vs, int rows,
                                        const SliceMeta& meta) {
    if (rows >= 16) slice_of<true>(Ks, Vs, 16, meta);
    else slice_of<false>(Ks, Vs, rows, meta);
  }
  template <bool FULL>
  __device__ __forceinline__ void slice_of(const uint8_t* Ks, const uint8_t* Vs, int rows,
                                        const SliceMeta& meta) {
    const int key = 4 * (c >> 1) + (c & 1);
    uint4 ka[2], kb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ka[i] = lds128(Ks + sw128(key, 2 * t + i));
      kb[i] = lds128(Ks + sw128(key + 2, 2 * t + i));
    }
    float s[NT][2][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[n][0][k] = s[n][1][k] = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const uint32_t wa = word(ka[w >> 2], w & 3), wb = word(kb[w >> 2], w & 3);
      const uint32_t a0 = e4m3x2_to_f16x2(wa), a2 = e4m3x2_to_f16x2(wa >> 16);
      const uint32_t a1 = e4m3x2_to_f16x2(wb), a3 = e4m3x2_to_f16x2(wb >> 16);
#pragma unroll
      for (int n = 0; n < NT; ++n)
        mma_f16(s[n][w & 1], a0, a1, a2, a3, qb[n][w][0], qb[n][w][1]);
    }
    uint32_t pb[NT][2], rest[2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float sc = s[n][0][k] + s[n][1][k];
        x[k] = FULL || key + (k & 2) < rows ? fmaf(sc, qk[n][k & 1] * meta.ks, meta.lv)
                                                 : -INFINITY;
      }
      const float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
      if (__any_sync(0xffffffffu, mx0 > m[n][0] + kTau || mx1 > m[n][1] + kTau)) {
        float mx[2] = {mx0, mx1};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1)
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], off));
          const float to = mx[e] > m[n][e] + kTau ? mx[e] : m[n][e];
          const float alpha = ex2(m[n][e] - to);
          l[n][e] = moved(l[n][e], m[n][e] - to);
          m[n][e] = to;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[n][i][e] *= alpha;
            o[n][i][2 + e] *= alpha;
          }
        }
      }
      // the weights, up to 2^(kShift + kTau) / vs, and what they count in the product
      const float ref[2] = {m[n][0] - kShift + meta.lv, m[n][1] - kShift + meta.lv};
      float pr[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) pr[k] = ex2(x[k] - ref[k & 1]);
      l[n][0] += pr[0] + pr[2];
      l[n][1] += pr[1] + pr[3];
#pragma unroll
      for (int k = 0; k < 4; ++k) pr[k] *= meta.vs;
      // Rounded to fp16; up to 8 heads what that leaves (22 bits together)
      // enters as well, for nothing where memory bounds the call (268 MB at
      // g = 8: 46.7 us without, 47.0 with; a CTA's tile 0.03 us more).  At more
      // heads the warps' own work does (g = 16: 53.5 and 59.2 us), and the one
      // rounding of 2^-12, an eighth of the bf16 output's, stays.
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t hi = pack_f16x2(pr[2 * k], pr[2 * k + 1]);
        pb[n][k] = movm_trans(hi);
        if (kTwoParts) {
          const float2 f = f16x2_to_f32x2(hi);
          rest[k] = movm_trans(pack_f16x2(pr[2 * k] - f.x, pr[2 * k + 1] - f.y));
        }
      }
    }
    // rows that do not count may be NaN: 0 * NaN would spread
    const int seen = rows - 4 * t;  // of this lane's four rows
    const uint32_t keep = FULL || seen >= 4 ? 0xffffffffu
                          : seen <= 0       ? 0u
                                            : (1u << (8 * seen)) - 1u;
    const int lane = 4 * c + t;
    const uint32_t v_row = smem_u32(Vs) + (lane & 15) * 128;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      uint32_t v[4];
      ldmatrix_codes(v, v_row + (((i + (lane >> 4)) ^ (lane & 7)) << 4));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t lo = FULL ? v[2 * j] : v[2 * j] & keep;
        const uint32_t hi = FULL ? v[2 * j + 1] : v[2 * j + 1] & keep;
        const uint32_t a0 = e4m3x2_to_f16x2(lo), a2 = e4m3x2_to_f16x2(lo >> 16);
        const uint32_t a1 = e4m3x2_to_f16x2(hi), a3 = e4m3x2_to_f16x2(hi >> 16);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_f16(o[n][i + j], a0, a1, a2, a3, pb[n][0], pb[n][1]);
          if (kTwoParts) mma_f16(o[n][i + j], a0, a1, a2, a3, rest[0], rest[1]);
        }
      }
    }
  }
  // This warp's (m, l, o) -> ml [warp][g][2], mo (merge_row): rows of even and
  // of odd heads apart and 136 floats long, so that a store's lanes (8 c, 4 t)
  // fall on 32 different banks.
  __device__ __forceinline__ void stash(float* mo, float* ml, int warp, int g) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[n][e];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        const int h = 8 * n + 2 * t + e;
        if (h < g) {
          float* dst = mo + merge_row(warp, h, g) + c;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dst[16 * i] = o[n][i][e];
            dst[16 * i + 8] = o[n][i][2 + e];
          }
          if (c == 0)
            *reinterpret_cast<float2*>(ml + (warp * g + h) * 2) = make_float2(m[n][e], sum);
        }
      }
  }
};

// The warps' partials of column i (head i / 32, four dims), in warp order: the
// maximum, and sum and unnormalised output relative to it.
__device__ __forceinline__ void merge_warps8(const float* mo, const float* mml, int i, int g,
                                             float& M, float& ls, float4& os) {
  const int h = i / (kD / 4), d = (i % (kD / 4)) * 4;
  float2 ml[kWarps];
  M = kMInit;
#pragma unroll
  for (int ww = 0; ww < kWarps; ++ww) {
    ml[ww] = *reinterpret_cast<const float2*>(mml + (ww * g + h) * 2);
    M = fmaxf(M, ml[ww].x);
  }
  ls = 0.f;
  os = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int ww = 0; ww < kWarps; ++ww) {
    const float e = ex2(ml[ww].x - M);
    const float4 x = *reinterpret_cast<const float4*>(mo + merge_row(ww, h, g) + d);
    ls += moved(ml[ww].y, ml[ww].x - M);
    os.x = fmaf(x.x, e, os.x);
    os.y = fmaf(x.y, e, os.y);
    os.z = fmaf(x.z, e, os.z);
    os.w = fmaf(x.w, e, os.w);
  }
}

// A segment split over CTAs c0 .. c0 + n - 1.
struct Part8 {
  size_t out_at;
  int c0, n;
};
static_assert(2 * sizeof(Part8) <= 8 * 4, "two fit behind misc[24]");
// The CTA's last piece: whole, or part `own` of a segment; have: the segment's
// only other part has arrived and lies in shared memory.
struct Last8 {
  Part8 pt;
  uint32_t* counter;
  int whole, own, have;
};
static_assert(sizeof(Last8) <= 16 * 4, "behind misc[32]");

__device__ __forceinline__ void store_column(const Kv8Params& p, size_t out_at, int col,
                                             const float4& o, float ls) {
  const float inv = ls == 0.f ? 0.f : 1.f / ls;
  if (!range_ok(col >= 0 && out_at + (size_t)col * 4 + 4 <= (size_t)p.B * p.Hq * kD, p.status))
    return;
  *reinterpret_cast<uint2*>(p.out + out_at + (size_t)col * 4) =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}
// Where part r of a segment lies: a CTA holds at most one segment's first part
// and at most one later part.
__device__ __forceinline__ int part_slot(const Part8& pt, int r) {
  return 2 * (pt.c0 + r) + (r == 0);
}
__device__ __forceinline__ bool slot_ok(const Kv8Params& p, int slot) {
  return range_ok(slot >= 0 && slot < 2 * kKv8MaxGrid, p.status);
}

// A column's output from few parts, in CTA order (absent ones: kMInit, zeros).
constexpr int kFewParts = 4;
__device__ __forceinline__ void join_parts(const Kv8Params& p, size_t out_at, int col,
                                           const float2 (&ml)[kFewParts],
                                           const float4 (&x)[kFewParts]) {
  float M = kMInit;
#pragma unroll
  for (int r = 0; r < kFewParts; ++r) M = fmaxf(M, ml[r].x);
  float ls = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int r = 0; r < kFewParts; ++r) {
    const float e = ex2(ml[r].x - M);
    ls += moved(ml[r].y, ml[r].x - M);
    o.x = fmaf(x[r].x, e, o.x);
    o.y = fmaf(x[r].y, e, o.y);
    o.z = fmaf(x[r].z, e, o.z);
    o.w = fmaf(x[r].w, e, o.w);
  }
  store_column(p, out_at, col, o, ls);
}

// Merge the parts of a split segment.  Few parts: every one of `threads` loads
// all of its column's in one round trip.
__device__ __forceinline__ void merge_few(const Kv8Params& p, const Part8& pt, int tid,
                                          int threads) {
  const int g = p.g;
#pragma unroll 2
  for (int col = tid; col < g * (kD / 4); col += threads) {
    const int h = col / (kD / 4);
    float2 ml[kFewParts];
    float4 x[kFewParts];
#pragma unroll
    for (int r = 0; r < kFewParts; ++r) {
      ml[r] = make_float2(kMInit, 0.f);
      x[r] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < pt.n && slot_ok(p, part_slot(pt, r))) {
        const size_t at = (size_t)part_slot(pt, r) * g;
        ml[r] = __ldcg(reinterpret_cast<const float2*>(p.part_ml + (at + h) * 2));
        x[r] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * kD) + col);
      }
    }
    join_parts(p, pt.out_at, col, ml, x);
  }
}

// More, by the consumer warps once the CTA's tiles are done, with `buf` (the
// ring's memory) in shared memory: the parts' (max, sum) come first, then the
// outputs, a float4 per thread and part, heads x 32 columns, and where those
// leave threads over (g < 8) the parts are dealt out among them as well.
__device__ __forceinline__ void merge_many(const Kv8Params& p, const Part8& pt, float* buf,
                                           ConsumerSync& csync, int warp, int lane) {
  const int g = p.g, tid = warp * 32 + lane;
  // (the slots rise with the part: the last one bounds them all, and `buf`)
  const int n = slot_ok(p, pt.c0) && slot_ok(p, 2 * (pt.c0 + pt.n - 1) + 1) ? pt.n : 0;
  const int cols = g * (kD / 4);
  float* wt = buf;              // [n][g] maxima, then weights
  float* ls = buf + n * g;      // [n][g] sums; row 0 then holds the totals
#pragma unroll 4
  for (int i = tid; i < n * g; i += kConsumers) {
    const int r = i / g, h = i - r * g;
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(
        p.part_ml + ((size_t)part_slot(pt, r) * g + h) * 2));
    wt[i] = ml.x;
    ls[i] = ml.y;
  }
  csync(lane);
  for (int h = warp; h < g; h += kWarps) {
    float M = kMInit, sum = 0.f;
    for (int r = lane; r < n; r += 32) M = fmaxf(M, wt[r * g + h]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    for (int r = lane; r < n; r += 32) {
      const float d = wt[r * g + h] - M;
      wt[r * g + h] = ex2(d);
      sum += moved(ls[r * g + h], d);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    __syncwarp();
    if (lane == 0) ls[h] = sum;  // row 0's own sum has been read
  }
  csync(lane);
  const int deal = max(1, kConsumers / cols);  // threads that share a column
  float4* red = reinterpret_cast<float4*>(buf + ((2 * n * g + 3) & ~3));
  for (int base = 0; base < cols; base += kConsumers) {
    const int who = tid / cols, col = base + (deal > 1 ? tid - who * cols : tid);
    const bool on = deal > 1 ? who < deal : col < cols;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) {
      const int h = col / (kD / 4);
#pragma unroll 16
      for (int r = deal > 1 ? who : 0; r < n; r += deal) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(
                                    p.part_o + (size_t)part_slot(pt, r) * g * kD) + col);
        const float e = wt[r * g + h];
        o.x = fmaf(x.x, e, o.x);
        o.y = fmaf(x.y, e, o.y);
        o.z = fmaf(x.z, e, o.z);
        o.w = fmaf(x.w, e, o.w);
      }
    }
    if (deal > 1) {
      if (on) red[tid] = o;
      csync(lane);
      if (who == 0) {
        for (int k = 1; k < deal; ++k) {
          const float4 x = red[k * cols + tid];
          o.x += x.x;
          o.y += x.y;
          o.z += x.z;
          o.w += x.w;
        }
      }
    }
    if (on && (deal == 1 || who == 0)) store_column(p, pt.out_at, col, o, ls[col / (kD / 4)]);
  }
  csync(lane);  // buf may be written again
}
// This CTA's part of a segment, column by column.
__device__ __forceinline__ void store_part(const Kv8Params& p, int slot, int col, float M,
                                           float ls, const float4& o) {
  if (!slot_ok(p, slot)) return;
  reinterpret_cast<float4*>(p.part_o + (size_t)slot * p.g * kD)[col] = o;
  if (col % (kD / 4) == 0)
    *reinterpret_cast<float2*>(p.part_ml + ((size_t)slot * p.g + col / (kD / 4)) * 2) =
        make_float2(M, ls);
}
// One thread, when all of the CTA's part is written: whether it is the last of
// n to arrive.
__device__ __forceinline__ bool arrive_last(uint32_t* counter, int n) {
  __threadfence();  // (the other threads' stores came before a barrier)
  const bool last = atomicAdd(counter, 1u) + 1 == (uint32_t)n;
  if (last) *counter = 0;
  __threadfence();
  return last;
}
// The statistics of all parts and the dealt-out columns fit two stages.
static_assert((2 * kKv8MaxGrid * 16 + 4 + 4 * kConsumers) * 4 <= 2 * kStageBytes, "merge_many");

template <int NT, bool LIST>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const Kv8Params p) {
  constexpr int E = kEndUnits<NT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int NS = p.stages;
  uint8_t* stages = smem;
  const int B = p.B, Hkv = p.Hkv, L = p.L, g = p.g;
  uint8_t* qbuf = smem + (size_t)NS * kStageBytes;                             // [NS][g][kD] bf16
  SliceMeta* meta = reinterpret_cast<SliceMeta*>(qbuf + NS * g * kD * 2);      // [NS][kSlices]
  // [merge_buffers] of merge_row rows, then (max, sum) [warps][g]
  const int n_buf = merge_buffers(g), buf_floats = merge_floats(g);
  float* merge = reinterpret_cast<float*>(meta + NS * kSlices);
  const int ml_at = kWarps * merge_heads(g) * kMergeRow;
  // full [NS], empty [NS], consumers' sync, merge full [2], empty [2], merged
  float* other = merge + n_buf * buf_floats;  // [g][kD], then (max, sum) [g]
  uint64_t* bars = reinterpret_cast<uint64_t*>(other + other_floats(g));
  uint64_t* m_full = bars + 2 * NS + 1;
  uint64_t* m_empty = m_full + 2;
  uint64_t* merged = m_empty + 2;
  uint64_t* m_sync = merged + 1;  // the merge warps' own barrier
  int* misc = reinterpret_cast<int*>(m_sync + 1);
  int* prefix = misc + kMiscInts;                         // [B+1]
  int* spos = prefix + B + 1;                             // [B]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = misc;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(&bars[s]), 2);  // the copies issued; the scales in place
      mbar_init(smem_u32(&bars[NS + s]), kWarps);
    }
    mbar_init(smem_u32(&bars[2 * NS]), kWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&m_full[i]), kWarps);               // every consumer warp has stashed
      mbar_init(smem_u32(&m_empty[i]), kMergeThreads / 32);  // both merge warps have read
    }
    mbar_init(smem_u32(merged), 1);  // the merge warps have come to the last piece
    mbar_init(smem_u32(m_sync), kMergeThreads / 32);
    misc[0] = 0;
    misc[3] = 0;
    fence_mbar_init();
  }
  grid_dependency_wait();
  grid_dependents_launch();

  // ---- units per sequence and KV head, their exclusive prefix sum (every CTA)
  const int list_tiles = LIST ? (int)((((long long)p.count << p.lb) + kTile - 1) / kTile) : 0;
  int carry = 0;
  for (int base = 0; base < B; base += kConsumers) {
    const int b = base + tid;
    int v = 0;
    if (tid < kConsumers && b < B) {
      const int pos = p.positions[b];
      spos[b] = pos;
      if (rows_in_cache(pos, 0, L)) {
        v = (LIST ? list_tiles : pos / kTile + 1) + E;
      } else if (b % (int)gridDim.x == (int)blockIdx.x) {
        // out-of-range position: flag it and make the sequence's output NaN
        set_status(p.status, ATTN_DEV_BAD_POSITION);
        uint4* row = reinterpret_cast<uint4*>(p.out + (size_t)b * p.Hq * kD);
        for (int i = 0; i < p.Hq * kD / 8; ++i)
          row[i] = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
      }
    }
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    if (lane == 31 && warp < kWarps) misc[8 + warp] = x;
    __syncthreads();
    int before = 0, chunk = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int s = misc[8 + w];
      before += w < warp ? s : 0;
      chunk += s;
    }
    if (tid < kConsumers && b < B) prefix[b] = carry + before + x - v;
    carry += chunk;
    __syncthreads();
  }
  if (tid == 0) prefix[B] = carry;
  __syncthreads();

  const long long T = (long long)Hkv * carry;  // all units
  // As many CTAs as there are units at most; one per segment where segments
  // are short (a split costs a round trip through L2).
  const long long nseg = (long long)B * Hkv;
  long long gw = min((long long)gridDim.x, T);
  if (T <= (long long)(kWholeTiles + E) * nseg) gw = min(gw, nseg);
  const int G = (int)gw;
  if ((int)blockIdx.x >= G) return;
  Range8 rg;
  range8_init<E>(rg, T, blockIdx.x, G, prefix, B, Hkv);
  if (rg.t0 >= rg.t1) return;
  Walk8 w;
  walk8_start<E>(w, rg, prefix, spos, B, Hkv);
  if (w.u >= w.end) return;  // end units alone

  if (warp >= kWarps + 2) {
    // --------------------------------------------------------------- merge --
    // The consumers leave each piece's partials in a buffer and go on; these
    // two warps merge them and write the output, or, for a piece that is only
    // part of its segment, the CTA's partial, and settle who merges the parts.
    // The last piece is for the consumers, which have nothing else to do then;
    // if it is one of two parts and the other has arrived, that one is fetched
    // while they are still at work.
    const int mtid = tid - kConsumers - 64;
    ConsumerSync msync{smem_u32(m_sync), abort_flag, p.status, 0u};
    for (int k = 0; w.u < w.end; ++k) {
      const int len = (int)min((long long)(w.nt - w.k), w.end - w.u);
      const bool whole = w.k == 0 && len == w.nt;
      const int slot = 2 * blockIdx.x + (w.k == 0);  // part_slot
      const long long f0 = w.u - w.k;                // the segment's first unit
      Part8 pt;
      pt.out_at = ((size_t)w.b * p.Hq + (size_t)w.kvh * g) * kD;
      pt.c0 = whole ? 0 : cta_of(f0, T, G);
      pt.n = whole ? 1 : cta_of(f0 + w.nt - 1, T, G) - pt.c0 + 1;
      uint32_t* counter = &p.counters[w.b * Hkv + w.kvh];
      if (len < w.nt - w.k) {  // the part of the range ends inside the segment
        w.u = w.end;
      } else {
        walk8_segment<E>(w, prefix, spos, B, Hkv);
      }
      walk8_turn<E>(w, rg, prefix, spos, B, Hkv);
      if (w.u >= w.end) {  // the last piece
        const int own = (int)blockIdx.x - pt.c0;
        if (mtid == 0) {
          bool have = false;
          if (!whole && pt.n == 2) {
            have = *(volatile uint32_t*)counter == 1u;
            __threadfence();
          }
          Last8* last = reinterpret_cast<Last8*>(misc + 32);
          last->pt = pt;
          last->counter = counter;
          last->whole = whole;
          last->own = own;
          last->have = have;
          misc[1] = have;  // (misc[2] may still be being read for the piece before)
        }
        msync(lane);
        if (misc[1] && slot_ok(p, part_slot(pt, 1 - own))) {
          const size_t at = (size_t)part_slot(pt, 1 - own) * g;
          const float4* o = reinterpret_cast<const float4*>(p.part_o + at * kD);
#pragma unroll 8
          for (int i = mtid; i < g * (kD / 4); i += kMergeThreads)
            reinterpret_cast<float4*>(other)[i] = __ldcg(o + i);
          if (mtid < g)
            reinterpret_cast<float2*>(other + g * kD)[mtid] =
                __ldcg(reinterpret_cast<const float2*>(p.part_ml + at * 2) + mtid);
        }
        msync(lane);
        break;
      }
      const int buf = n_buf == 2 ? k & 1 : 0;
      const uint32_t use = (uint32_t)(n_buf == 2 ? k >> 1 : k);
      if (!consumer_wait(smem_u32(&m_full[buf]), use & 1u, abort_flag, p.status, lane)) break;
      const float* mo = merge + buf * buf_floats;
#pragma unroll 2
      for (int i = mtid; i < g * (kD / 4); i += kMergeThreads) {
        float M, ls;
        float4 os;
        merge_warps8(mo, mo + ml_at, i, g, M, ls, os);
        if (whole) store_column(p, pt.out_at, i, os, ls);
        else store_part(p, slot, i, M, ls, os);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&m_empty[buf]));
      if (!whole) {
        // the segment's last CTA to arrive merges the parts
        msync(lane);
        if (mtid == 0) {
          const bool last = arrive_last(counter, pt.n);
          misc[2] = last;
          if (last && pt.n > kFewParts && range_ok(misc[3] < 2, p.status))  // left to the consumers
            reinterpret_cast<Part8*>(misc + 24)[misc[3]++] = pt;
        }
        msync(lane);
        if (misc[2] && pt.n <= kFewParts && !*abort_flag) merge_few(p, pt, mtid, kMergeThreads);
      }
    }
    if (mtid == 0) mbar_arrive(smem_u32(merged));
  } else if (warp >= kWarps) {
    // ----------------------------------------------------------- producers --
    // Warp kWarps issues the copies, warp kWarps + 1 brings the scales; a tile is full
    // when both have arrived and the copies have landed.
    // Where an address hangs on a load, tiles go in batches of four: lane
    // 8*ti + slice looks after slice `slice` of the batch's tile ti, and what
    // a batch needs is loaded while the one before it is issued, so that the
    // latency is spread over four tiles' time.
    const bool copies = warp == kWarps;
    const int ti = lane >> 3, slice = lane & 7;
    const int entry_rows = 1 << p.lb;
    const int in_block = (slice * 16) & (entry_rows - 1);
    const int entry = (slice * 16) >> p.lb;            // of this slice, within a tile
    const int per_tile = kTile >> p.lb;
    // the block a listed tile's slice lies in (-1: none)
    auto fetch = [&](const Walk8& w) -> int {
      const int e = w.k * per_tile + entry;
      return e < p.count ? p.index[(size_t)(w.b * Hkv + w.kvh) * p.count + e] : -1;
    };
    auto row_of = [&](const Walk8& w, int blk) -> int {
      int row;
      if (LIST) {
        if (blk < -1 || blk >= p.nb) {
          if (copies) set_status(p.status, ATTN_DEV_BAD_BLOCK);
          blk = -1;
        }
        row = blk >= 0 ? (blk << p.lb) + in_block : kNoRow;
      } else {
        row = w.k * kTile + slice * 16;
      }
      return row <= w.pos ? row : kNoRow;
    };
    auto step = [&](Walk8& w, int n) {  // n tiles on, as far as the range goes
      if (w.k + n < w.nt && w.u + n < w.end) {
        w.k += n;
        w.u += n;
        return;
      }
      for (int k = 0; k < n && w.u < w.end; ++k) walk8_next<E>(w, rg, prefix, spos, B, Hkv);
    };
    int s = 0;          // the ring's stage and pass of the tile at hand
    uint32_t pass = 0;
    auto wait_empty = [&]() -> bool {  // by the whole warp
      if (pass == 0) return true;
      if (__all_sync(0xffffffffu,
                     mbar_wait(smem_u32(&bars[NS + s]), (pass & 1u) ^ 1u, abort_flag)))
        return true;
      if (lane == 0) {
        *abort_flag = 1;
        set_status(p.status, ATTN_DEV_TIMEOUT);
      }
      return false;
    };
    auto turn = [&]() {
      if (++s == NS) {
        s = 0;
        ++pass;
      }
    };
    // the tile's arrival, with its bytes; a piece's first tile brings the
    // segment's query rows along
    auto expect = [&](uint32_t full, uint32_t bytes, bool starts, int b, int kvh) {
      const uint32_t q_bytes = starts ? (uint32_t)g * kD * 2u : 0u;
      mbar_arrive_expect_tx(full, q_bytes + bytes);
      if (q_bytes)
        bulk_load(smem_u32(qbuf + s * g * kD * 2),
                  p.q + ((size_t)b * p.Hq + (size_t)kvh * g) * kD, q_bytes, full);
    };
    if (copies && !LIST) {
      for (; w.u < w.end; walk8_next<E>(w, rg, prefix, spos, B, Hkv)) {
        if (!wait_empty()) break;
        const int z = w.b * Hkv + w.kvh, row = w.k * kTile;
        // failure-path tests only: a tile never issued
        const bool skip = p.test_skip >= 0 && z == 0 && w.k == p.test_skip;
        if (lane == 0 && !skip && range_ok(row < L && z < B * Hkv, p.status)) {
          const uint32_t full = smem_u32(&bars[s]);
          const uint32_t sK = smem_u32(stages + (size_t)s * kStageBytes);
          expect(full, kStageBytes, w.k == 0 || w.u == rg.t0, w.b, w.kvh);
          tma_load_3d(sK, &tm_k, 0, row, z, full);
          tma_load_3d(sK + kOpBytes, &tm_v, 0, row, z, full);
        }
        __syncwarp();
        turn();
      }
    } else {
      long long last_end = w.end;  // of the part of the range done last
      if (rg.tA < rg.t1) {
        Walk8 rest;
        walk8_init<E>(rest, rg.t0, prefix, spos, B, Hkv);
        if (rest.u < rg.tA) last_end = rg.tA;
      }
      // What a lane knows of its tile, and of the next batch's.
      struct Mine {
        int row, z, k, flags;
        float ks, vs;
        bool on;
      };
      auto look_up = [&](int blk) -> Mine {
        Mine m;
        m.on = w.u < w.end;
        m.z = w.b * Hkv + w.kvh;
        m.k = w.k;
        m.row = m.on ? row_of(w, blk) : kNoRow;
        m.ks = m.vs = 1.f;
        m.flags = 0;
        if (m.on) {
          if (!copies && m.row != kNoRow &&
              range_ok((m.row >> p.lb) < p.nb && m.z < B * Hkv, p.status)) {
            const size_t at = (size_t)m.z * p.nb + (m.row >> p.lb);
            m.ks = p.k_scale[at];
            m.vs = p.v_scale[at];
            m.flags = min(16, w.pos + 1 - m.row);
          }
          if (w.k == 0 || w.u == rg.t0) m.flags |= kStarts;
          if (w.k == w.nt - 1 || w.u + 1 == w.end) m.flags |= kEnds;
          // the CTA's last tile: none in what is left of this part of the
          // range (the next one would come after the end units), nor a part after it
          if (w.u + 1 + (w.k == w.nt - 1 ? E : 0) >= w.end && w.end == last_end) m.flags |= kLast;
        }
        return m;
      };
      step(w, ti);  // this lane's tile of the first batch
      Mine cur = look_up(LIST && w.u < w.end ? fetch(w) : -1);
      step(w, 4);
      int blk = LIST && w.u < w.end ? fetch(w) : -1;
      bool ok = true, fresh = false;
      while (ok) {
        const int n_q = __popc(__ballot_sync(0xffffffffu, cur.on)) >> 3;  // tiles of the batch
        if (n_q == 0) break;
        const Mine nxt = look_up(blk);
        step(w, 4);
        blk = LIST && w.u < w.end ? fetch(w) : -1;
        SliceMeta mt;
        if (!copies) mt = slice_meta(cur.flags, cur.ks, cur.vs);
        const bool skip = p.test_skip >= 0 && cur.z == 0 && cur.k == p.test_skip;  // tests only
        const bool have = cur.row != kNoRow && in_block == 0 && !skip &&
                          range_ok(cur.row >= 0 && cur.row < L && cur.z < B * Hkv, p.status);
        const uint32_t boxes = __ballot_sync(0xffffffffu, have);
        const uint32_t any = __ballot_sync(0xffffffffu, cur.row != kNoRow);
        const uint32_t first = __ballot_sync(0xffffffffu, (cur.flags & kStarts) != 0);
        const uint32_t ends = __ballot_sync(0xffffffffu, (cur.flags & kEnds) != 0);
        for (int q = 0; q < n_q; ++q) {
          // a listed tile without a row is passed over, but for a piece's last
          fresh = fresh || ((first >> (8 * q)) & 1u);
          if (LIST && !((any >> (8 * q)) & 0xffu) && !((ends >> (8 * q)) & 1u)) continue;
          if (!wait_empty()) {
            ok = false;
            break;
          }
          if (copies) {
            const uint32_t full = smem_u32(&bars[s]);
            if (lane == 8 * q && !skip) {
              const int b = cur.z / Hkv;
              expect(full, __popc((boxes >> (8 * q)) & 0xffu) * (uint32_t)entry_rows * 2u * kD,
                     fresh, b, cur.z - b * Hkv);
            }
            __syncwarp();
            if (ti == q && have) {
              const uint32_t sK = smem_u32(stages + (size_t)s * kStageBytes) + slice * 16 * kD;
              tma_load_3d(sK, &tm_k, 0, cur.row, cur.z, full);
              tma_load_3d(sK + kOpBytes, &tm_v, 0, cur.row, cur.z, full);
            }
          } else {
            if (ti == q) {
              mt.rows = (mt.rows & ~kStarts) | (fresh ? kStarts : 0);
              meta[s * kSlices + slice] = mt;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars[s]));
          }
          fresh = false;
          turn();
        }
        cur = nxt;
      }
    }
  } else {
    // ----------------------------------------------------------- consumers --
    // The flags beside a tile say where pieces start and end, so these warps
    // keep no place in the list.
    Consumer8<NT> cs;
    cs.c = lane >> 2;
    cs.t = lane & 3;
    int s = 0, piece = 0;
    uint32_t ph = 0;
    bool ok = true;
    float* mo = merge;  // the last piece's buffer
    for (int flags = 0; !(flags & kLast);) {
      ok = consumer_wait(smem_u32(&bars[s]), ph, abort_flag, p.status, lane);
      if (!ok) break;
      const SliceMeta mt = meta[s * kSlices + warp];
      flags = mt.rows;
      if (flags & kStarts) {
        cs.load_q(qbuf + s * g * kD * 2, g, p.qscale);
        cs.reset();
      }
      const uint8_t* Ks = stages + (size_t)s * kStageBytes + warp * 16 * kD;
      const int rows = flags & kRowsMask;
      if (rows > 0) cs.slice(Ks, Ks + kOpBytes, rows, mt);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars[NS + s]));
      if (++s == NS) {
        s = 0;
        ph ^= 1u;
      }
      if (flags & kEnds) {  // this piece's partial for the merge warps
        const int buf = n_buf == 2 ? piece & 1 : 0;
        const uint32_t use = (uint32_t)(n_buf == 2 ? piece >> 1 : piece);
        ++piece;
        if (use > 0) {
          ok = consumer_wait(smem_u32(&m_empty[buf]), (use & 1u) ^ 1u, abort_flag, p.status, lane);
          if (!ok) break;
        }
        mo = merge + buf * buf_floats;
        cs.stash(mo, mo + ml_at, warp, g);
        __syncwarp();
        if (lane == 0 && !(flags & kLast)) mbar_arrive(smem_u32(&m_full[buf]));
      }
    }
    // the last piece, and segments of many parts that this CTA was the last to reach
    if (ok && consumer_wait(smem_u32(merged), 0u, abort_flag, p.status, lane) && !*abort_flag) {
      ConsumerSync csync{smem_u32(&bars[2 * NS]), abort_flag, p.status, 0u};
      csync(lane);  // every warp has stashed
      const Last8 last = *reinterpret_cast<const Last8*>(misc + 32);
      const int slot = 2 * blockIdx.x + (last.own == 0);
      for (int i = tid; i < g * (kD / 4); i += kConsumers) {
        float2 ml[kFewParts];
        float4 x[kFewParts];
#pragma unroll
        for (int r = 0; r < kFewParts; ++r) {
          ml[r] = make_float2(kMInit, 0.f);
          x[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float2 me;
        float4 mine;
        merge_warps8(mo, mo + ml_at, i, g, me.x, me.y, mine);
        if (last.whole) {
          store_column(p, last.pt.out_at, i, mine, me.y);
        } else if (last.have) {
          const float4 their = reinterpret_cast<const float4*>(other)[i];
          const float2 tml = reinterpret_cast<const float2*>(other + g * kD)[i / (kD / 4)];
          ml[0] = last.own == 0 ? me : tml;
          x[0] = last.own == 0 ? mine : their;
          ml[1] = last.own == 0 ? tml : me;
          x[1] = last.own == 0 ? their : mine;
          join_parts(p, last.pt.out_at, i, ml, x);
        } else {
          store_part(p, slot, i, me.x, me.y, mine);
        }
      }
      if (!last.whole && last.have) {
        if (tid == 0) *last.counter = 0;
      } else if (!last.whole) {
        csync(lane);
        if (tid == 0) misc[2] = arrive_last(last.counter, last.pt.n);
        csync(lane);
        if (misc[2] && !*abort_flag) {
          if (last.pt.n <= kFewParts)
            merge_few(p, last.pt, tid, kConsumers);
          else
            merge_many(p, last.pt, reinterpret_cast<float*>(stages), csync, warp, lane);
        }
      }
      const int left = *(volatile int*)(misc + 3);
      for (int i = 0; i < left && !*abort_flag; ++i)
        merge_many(p, reinterpret_cast<const Part8*>(misc + 24)[i],
                   reinterpret_cast<float*>(stages), csync, warp, lane);
    }
  }
  if (*abort_flag) {  // copies in flight land before the shared memory goes
    const uint64_t t_start = globaltimer_ns();
    while (globaltimer_ns() - t_start < 2000000ull) {
    }
  }
}

}  // namespace
}  // namespace gqa

#include "kv8_cluster.cuh"

namespace gqa {
namespace {

// ------------------------------------------------------------------ host --

// Per device, found once: its SMs and how many clusters of each size can run
// at once with one CTA to an SM (a cluster stays within one GPC).
struct Device8 {
  int sms;
  int clusters[kMaxCluster + 1];
};

template <int NT, bool LIST>
cudaError_t set_attributes() {
  cudaError_t e = cudaFuncSetAttribute(
      kv8_decode_kernel<NT, LIST>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kv8_cluster_kernel<NT, LIST>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kv8_cluster_kernel<NT, LIST>,
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e;
}

cudaError_t find_device(Device8& d, int dev) {
  cudaError_t e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = set_attributes<1, false>();
  if (e == cudaSuccess) e = set_attributes<1, true>();
  if (e == cudaSuccess) e = set_attributes<2, false>();
  if (e == cudaSuccess) e = set_attributes<2, true>();
  if (e != cudaSuccess) return e;
  for (int c = 1; c <= kMaxCluster; ++c) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c * 64);
    cfg.blockDim = dim3(kClusterThreads);
    cfg.dynamicSmemBytes = kMaxSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&d.clusters[c], kv8_cluster_kernel<1, false>, &cfg) !=
        cudaSuccess) {
      cudaGetLastError();
      d.clusters[c] = 0;
    }
  }
  return cudaSuccess;
}

cudaError_t device8(const Device8** out) {
  static Device8 known[64];
  static std::atomic<bool> ready[64];
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev < 0 || dev >= 64)) e = cudaErrorInvalidDevice;
  if (e != cudaSuccess) return e;
  if (!ready[dev].load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev].load(std::memory_order_relaxed)) {
      e = find_device(known[dev], dev);
      if (e != cudaSuccess) return e;
      ready[dev].store(true, std::memory_order_release);
    }
  }
  *out = &known[dev];
  return cudaSuccess;
}

// CTAs per segment in cluster mode, or 0 for the split over a flat list.  The
// cluster would be the largest that lets every segment have its own resident at
// once, or one CTA; it is taken where it should be faster (us, measured):
//   clusters   a wave: 4.1, and 0.55 for each tile of a CTA (g > 8: 4.6, 0.67)
//   flat list  10, and 0.69 for each tile of a CTA's even share (g > 8: 13),
//              and 0.007 for each head and part of a segment's merge
// The host knows the cache's length only: a position is taken to lie half-way
// on average, and the longest of several, which a cluster waits for, at the
// end; a list is taken as full.  So a young sequence pays for a long cache: at
// row 1000 of one stream (8 KV heads, g = 2) a step takes 4.4 us in caches up to
// about 166000 rows and 9.8 us in longer ones.  (One segment of 131072 rows, g = 2: 37 us in a
// cluster, 17 by the list; of 16384 rows: 8 and 12; 108 segments of up to 10
// tiles: 10 and 17.)
int cluster_size8(const Kv8Params& p, const Device8& d) {
  if (g_decode_test_cluster >= 0)  // schedule tests only
    return min(g_decode_test_cluster, kMaxCluster);
  const long long nseg = (long long)p.B * p.Hkv;
  const long long rows = p.index ? (long long)p.count << p.lb : (long long)p.L;
  const int tiles = (int)((rows + kTile - 1) / kTile);
  int c = min(kMaxCluster, tiles);
  while (c > 1 && nseg > d.clusters[c]) --c;
  const float mean = p.index ? (float)tiles : 0.5f * (float)tiles;
  const float longest = p.B == 1 ? mean : (float)tiles;
  const float waves = c > 1 ? 1.f : (float)((nseg + d.sms - 1) / d.sms);
  const bool wide = p.g > 8;
  const float clusters =
      waves * ((wide ? 4.6f : 4.1f) + (wide ? 0.67f : 0.55f) * ceilf(longest / (float)c));
  const float sms = (float)d.sms, parts = sms / (float)nseg;
  const float flat = (wide ? 13.f : 10.f) + 0.69f * (float)nseg * mean / sms +
                     (parts > 1.f ? 0.007f * (float)p.g * parts : 0.f);
  return clusters <= flat ? c : 0;
}

// A cache [segs, L, 128] of codes as a 3-D tensor map, box 128 codes x rows x
// 1, 128-byte swizzle.  Rows past L read as zeros.
bool codes_map(CUtensorMap* m, const void* ptr, int L, long long segs, int rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)L, (cuuint64_t)segs};
  cuuint64_t strides[2] = {(cuuint64_t)kD, (cuuint64_t)kD * (cuuint64_t)L};
  cuuint32_t box[3] = {(cuuint32_t)kD, (cuuint32_t)rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

template <int NT, bool LIST>
cudaError_t launch8(Kv8Params& p, const CUtensorMap& mk, const CUtensorMap& mv,
                    cudaStream_t stream) {
  const Device8* d = nullptr;
  cudaError_t e = device8(&d);
  if (e != cudaSuccess) return e;
  p.stages = kMaxStages;
  const int C = cluster_size8(p, *d);
  if (C > 0) {
    if (d->clusters[C] == 0) return cudaErrorNotSupported;
    while (p.stages > 2 && cluster_smem_bytes(p.stages, p.g, C) > (size_t)kMaxSmem) --p.stages;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.B * p.Hkv * C));
    cfg.blockDim = dim3(kClusterThreads);
    cfg.dynamicSmemBytes = cluster_smem_bytes(p.stages, p.g, C);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kv8_cluster_kernel<NT, LIST>, mk, mv, p);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  while (p.stages > 2 && smem_bytes(p.stages, p.B, p.g) > (size_t)kMaxSmem) --p.stages;
  return launch_pdl(kv8_decode_kernel<NT, LIST>, dim3(min(kKv8MaxGrid, d->sms)), dim3(kThreads),
                    smem_bytes(p.stages, p.B, p.g), stream, mk, mv, p);
}

}  // namespace

DecodeWorkspace kv8_workspace_layout(int B, int Hq, int Hkv) {
  auto align256 = [](size_t x) { return (x + 255) & ~(size_t)255; };
  DecodeWorkspace w{};
  const int g = Hq / Hkv;
  w.slots = 2 * kKv8MaxGrid;
  w.status_off = 0;
  w.ticket_off = 128;
  w.counters_off = 256;
  w.ml_off = align256(w.counters_off + (size_t)B * Hkv * sizeof(uint32_t));
  w.o_off = align256(w.ml_off + (size_t)w.slots * g * 2 * sizeof(float));
  w.total = align256(w.o_off + (size_t)w.slots * g * kD * sizeof(float));
  return w;
}

cudaError_t launch_kv8_decode(const void* q, const int32_t* positions, const void* k_cache,
                              const void* v_cache, const float* k_scale, const float* v_scale,
                              const int32_t* block_index, int count, int B, int Hq, int Hkv,
                              int L, int block, float scale, void* out, void* workspace,
                              cudaStream_t stream) {
  const DecodeWorkspace ws = kv8_workspace_layout(B, Hq, Hkv);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  Kv8Params p;
  p.q = static_cast<const uint16_t*>(q);
  p.positions = positions;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.index = block_index;
  p.out = static_cast<uint16_t*>(out);
  p.status = reinterpret_cast<uint32_t*>(base + ws.status_off);
  p.counters = reinterpret_cast<uint32_t*>(base + ws.counters_off);
  p.part_ml = reinterpret_cast<float*>(base + ws.ml_off);
  p.part_o = reinterpret_cast<float*>(base + ws.o_off);
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.L = L;
  p.g = Hq / Hkv;
  p.lb = block == 16 ? 4 : block == 32 ? 5 : block == 64 ? 6 : 7;
  p.nb = (L + block - 1) / block;
  p.count = count;
  p.stages = 0;
  p.test_skip = g_decode_test_skip;
  p.qscale = scale * 1.4426950408889634f;
  CUtensorMap mk, mv;
  const int rows = block_index ? block : kTile;
  if (!codes_map(&mk, k_cache, L, (long long)B * Hkv, rows) ||
      !codes_map(&mv, v_cache, L, (long long)B * Hkv, rows))
    return cudaErrorInvalidValue;
  if (block_index)
    return p.g <= 8 ? launch8<1, true>(p, mk, mv, stream)
                    : launch8<2, true>(p, mk, mv, stream);
  return p.g <= 8 ? launch8<1, false>(p, mk, mv, stream)
                  : launch8<2, false>(p, mk, mv, stream);
}

}  // namespace gqa
