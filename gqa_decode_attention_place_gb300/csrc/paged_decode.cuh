// paged_decode.cuh -- split-KV decode attention over a paged bf16 cache, S new
// tokens per sequence: the kernels and their launch, included by one translation
// unit per head dim, and for one token or several (DRAFTS: what several need makes
// a kernel's code longer, which one stream's step pays for: 9.1 and 9.5 us).
//
// For sequence b, new token t, query head h and KV head h/g:
//   out = softmax_j(scale q . K_j) V_j      over rows j = 0 .. positions[b] + t,
// row j in row j % page of page table[b][j / page].  The R = S g <= 32 query
// rows of a KV head share one pass over its keys and values: with x_j the score
// in base 2, M a reference at most kTau below the largest x_j so far and
// w_j = 2^(x_j - M),
//   out = sum_j w_j V_j / sum_j w_j.
//
// Bound by memory: a cache row costs 4 D bytes for K and V.  How:
//  * 128-row tiles stream through a shared-memory ring by tiled TMA copies with
//    the 128-byte swizzle, one copy per page and operand: the pool is a 5-D
//    tensor (dims, rows, dim halves, heads, pages), so any strides will do and
//    a page's rows land where a contiguous tile's would.  Two producer warps,
//    one for keys and one for values, look up table entries four tiles ahead (a
//    lane per 16 rows) and issue.
//  * 8 consumer warps take 16 rows of a tile each, with a maximum and a sum of
//    their own, and never wait for one another inside a piece.  Both products
//    run on warp-level MMAs (m16n8k16, bf16 in, fp32 out) with the query rows
//    as M: the scores' accumulators are then, lane by lane, the A operand of
//    the second product, so the weights stay in registers, and V comes through
//    transposing matrix loads.
//  * The weights enter as two bf16 parts (16 bits): up to 8 query rows for nothing,
//    as rows 8..15 of the MMA's M are free and take the rest; beyond, by a second
//    MMA (32 rows, 1.07 GB: 169 -> 175 us, and nothing for a ragged batch).  Only
//    at D = 64 with more than 16 rows they are rounded to bf16 once (2^-8, of errors
//    that average over the keys; the output's own rounding is the same size):
//    there a tile's transfer is half as long and the MMAs are what it waits for
//    (91 us, 107 with two parts).  The sums are of the weights as they entered.
//    Whatever the parts, an infinite value stays one (split_above_zero, both_parts).
//  * At a piece's end the warps' partials meet in the memory of its last tile,
//    each in the slice that its warp alone has read, so one barrier is enough.
//  * Work is split as in the 8-bit decode (flat_list.cuh): a flat list of all
//    tiles over a persistent grid, or for few segments a thread-block cluster
//    per segment, merged through distributed shared memory.
#pragma once

#include <cooperative_groups.h>

#include <atomic>
#include <mutex>

#include "common.cuh"
#include "decode_params.h"
#include "flat_list.cuh"
#include "paged.h"
#include "tcgen05.cuh"
#include "warp_ops.cuh"

namespace gqa {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8;                   // consumer warps
constexpr int kConsumers = kWarps * 32;
constexpr int kMergeThreads = 64;           // two warps that merge (flat list)
constexpr int kClusterThreads = kConsumers + 64;  // and the producers: of keys, of values
constexpr int kThreads = kClusterThreads + kMergeThreads;
constexpr int kMaxStages = 12;
constexpr int kMaxSmem = 227 * 1024;
// What a segment's end costs, in tiles' time (flat_list.cuh; with 1 for all, 32 ragged
// sequences of up to 16384 rows and 32 query rows: 185 us instead of 173).
template <int NT> constexpr int kEndUnits = NT == 4 ? 4 : NT == 2 ? 3 : 1;
constexpr int kWholeTiles = 4;              // segments this short are not split
// Whole segments, one CTA each (below): a lone CTA's tile takes kWholeNum / kWholeDen of
// its share of a busy GPU, and a merge as long as kMergeCost / kWholeDen tiles.
constexpr int kWholeNum = 5, kWholeDen = 9;
template <int D> constexpr int kMergeCost = 37 * (128 / D);
constexpr int kMaxCluster = 16;
constexpr float kMInit = -3e38f;            // the reference before any row
constexpr float kTau = 8.f;                 // it moves when a score lies more than this above

// TileMeta::flags: bits 0 .. 7, slices (16 rows) that hold rows, and
constexpr int kStarts = 0x100;     // a piece starts with this tile
constexpr int kEnds = 0x200;       // and ends with this one
constexpr int kLast = 0x400;       // the CTA's last tile

// What the producer leaves beside a tile.
struct TileMeta {
  int flags, row0;  // row0: the tile's first row
  int pos, n;       // the sequence's first new row, and how many there are
  int b, kvh;
  int c0, parts;    // the CTAs that share the segment (parts = 1: this one alone)
};

// NT: 8-row groups of query rows (1, 2 or 4).
template <int D, int NT>
struct Shape {
  static constexpr int kTile = 128;               // rows: whole pages, which have 128 at most
  static constexpr int kSlices = kTile / 16;
  static constexpr int kBatch = 32 / kSlices;     // tiles that a producer looks up at a time
  static constexpr int kOp = kTile * D * 2;       // bytes of a tile's keys
  static constexpr int kStage = 2 * kOp;
  static constexpr int kQStride = D * 2 + 16;     // bytes between query rows: no bank conflicts
  static constexpr int kQ = NT * 8 * kQStride;
  static constexpr int kMl = 2 * kWarps * (NT == 1 ? 8 : 16) * 8;  // bytes of (reference, sum)
};

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, int c3, int c4, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The producers' tensor maps, into their cache before they are used.
__device__ __forceinline__ void prefetch_maps(const CUtensorMap& k, const CUtensorMap& v, int warp,
                                              int lane) {
  if (lane == 0 && (warp == kWarps || warp == kWarps + 1))
    asm volatile("prefetch.tensormap [%0];" ::"l"(
                     reinterpret_cast<uint64_t>(warp == kWarps ? &k : &v))
                 : "memory");
}
// Four 8x8 matrices; lane l gives the address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// The token of query row r: r / g, exact for r < 32 and g <= 32.
__device__ __forceinline__ int token_of(const PagedParams& p, int r) {
  return (r * p.g_inverse) >> 16;
}
// Row of q and out that query row r of (b, kvh) is: rows are ordered token, head.
__device__ __forceinline__ size_t query_row(const PagedParams& p, int b, int kvh, int r) {
  const int t = token_of(p, r);
  return ((size_t)b * p.S + t) * p.Hq + (size_t)kvh * p.g + (r - t * p.g);
}

// A consumer warp.  Lane 4c + t.  It serves G 8-row groups of query rows, rows c
// and c + 8 of the MMA's M (G = 1: rows 8..15 are zero queries, and in the second
// product the weights' rest).  Of a tile it takes 16 rows; with more than 16
// query rows (NT = 4) half of the warps take 32 each for query rows 0..15, and the
// other half the same for 16..31.  (Warps with all 32 query rows would hold 128
// registers of outputs, and spill.)
template <int D, int NT, bool DRAFTS>
struct PagedConsumer {
  using Sh = Shape<D, NT>;
  static constexpr int G = NT == 1 ? 1 : 2;       // 8-row groups of a warp
  static constexpr int kTeams = NT == 4 ? 2 : 1;
  static constexpr int kTeam = kWarps / kTeams;   // warps that share query rows
  static constexpr int KS = D / 16;               // MMA steps of a score
  uint32_t qa[KS][2 * G];
  float o[D / 8][4];    // dims 8j + 2t, +1 for rows c, c + 8
  float ref[G];         // the references
  float sums[4];        // of the weights as they entered: rows c, c + 8 (in [0] and [2])
  int lim[G];           // last cache row that the query row sees, -1: none
  int c, t, warp, lane;
  int team, row_base;   // its place; its first query row

  __device__ __forceinline__ void init(int warp_, int lane_) {
    warp = warp_;
    lane = lane_;
    c = lane >> 2;
    t = lane & 3;
    team = warp / kTeam;
    row_base = 16 * team;
  }
  // The queries, negated for a negative score scale.
  __device__ __forceinline__ void load_q(const uint8_t* qs, uint32_t flip) {
    const uint32_t base = smem_u32(qs);
    const int i = lane >> 3, r = lane & 7;
    if (G == 1) {
#pragma unroll
      for (int k = 0; k < KS; k += 2) {
        uint32_t x[4];  // rows 0..7, four 8-dim chunks
        ldmatrix4(x, base + r * Sh::kQStride + (2 * k + i) * 16);
        qa[k][0] = x[0];
        qa[k][1] = x[1];
        qa[k + 1][0] = x[2];
        qa[k + 1][1] = x[3];
      }
    } else {
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t x[4];
        ldmatrix4(x, base + (row_base + r + 8 * (i & 1)) * Sh::kQStride + (2 * k + (i >> 1)) * 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) qa[k][G == 1 ? 0 : e] = x[e];
      }
    }
    if (flip) {
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 2 * G; ++e) qa[k][e] ^= flip;
    }
  }
  __device__ __forceinline__ void start(const PagedParams& p, int pos, int n) {
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int r = row_base + 8 * i + c, tok = DRAFTS ? token_of(p, r) : 0;
      ref[i] = kMInit;
      lim[i] = r < p.R && tok < n ? pos + tok : -1;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sums[e] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
  }
  // Byte offset in a tile of row 16 * slice (its first 64 dims).
  __device__ __forceinline__ static int slice_at(int slice, int lp) {
    const int row = slice * 16, page = row >> lp;
    return ((page << lp) * D * 2) + (row & ((1 << lp) - 1)) * 128;
  }

  // This warp's rows of a tile.  ks: its keys; the values lie behind them.
  __device__ __forceinline__ void tile(const uint8_t* ks, const PagedParams& p,
                                       const TileMeta& mt) {
    const int first = warp & (kTeam - 1);
    const uint32_t base = smem_u32(ks);
    const int half = 128 << p.lp;  // from a page's first 64 dims to the others
    constexpr bool kTwo = Sh::kSlices == 2 * kTeam;
    constexpr int kAll = kTwo ? 1 | (1 << kTeam) : 1;
    // full: every row is there and seen by every query row in use
    if (((mt.flags >> first) & kAll) == kAll &&
        mt.row0 + 16 * (first + (kTwo ? kTeam : 0)) + 15 <= mt.pos) {
      slices<kTwo ? 2 : 1, true>(base + slice_at(first, p.lp),
                                 base + slice_at(first + (kTwo ? kTeam : 0), p.lp), half, Sh::kOp,
                                 mt.row0 + 16 * first, p, mt);
      return;
    }
#pragma unroll 1
    for (int sl = first; sl < Sh::kSlices; sl += kTeam) {
      if (!((mt.flags >> sl) & 1)) continue;  // no rows there
      // (one slice that is full, where two are taken, does without the masks)
      const uint32_t at = base + slice_at(sl, p.lp);
      const int row = mt.row0 + 16 * sl;
      if (kTwo && row + 15 <= mt.pos) slices<1, true>(at, at, half, Sh::kOp, row, p, mt);
      else slices<1, false>(at, at, half, Sh::kOp, row, p, mt);
    }
  }
  // 16 cache rows from row0 on, whose keys lie at at0 (dims from 64 on `half` bytes
  // further, values v_off), and with N = 2 another 16 at at1, which are full too: the
  // two slices' chains of products and exponentials overlap.
  template <int N, bool FULL>
  __device__ __forceinline__ void slices(uint32_t at0, uint32_t at1, int half, int v_off, int row0,
                                         const PagedParams& p, const TileMeta& mt) {
    const int i8 = lane >> 3, r8 = lane & 7;
    const uint32_t at[2] = {at0, at1};
    float s[N][2][2][4];  // of each slice rows 0..7 and 8..15, in two chains each
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][j][h][e] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint32_t a[4];
      if (G == 1) {
        a[0] = qa[k][0];
        a[2] = qa[k][1];
        a[1] = a[3] = 0u;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = qa[k][G == 1 ? 0 : e];
      }
      const int ch = 2 * k + (i8 & 1);
      const int to = (8 * (i8 >> 1) + r8) * 128 + (2 * k >= 8 ? half : 0) + (((ch & 7) ^ r8) << 4);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        uint32_t b[4];
        ldmatrix4(b, at[n] + to);
        mma_bf16(s[n][0][N == 1 ? k & 1 : 0], a, b[0], b[1]);
        mma_bf16(s[n][1][N == 1 ? k & 1 : 0], a, b[2], b[3]);
      }
    }
    auto load_v = [&](uint32_t (&b)[4], int d, int n) {
      const int ch = 2 * d + (i8 >> 1);
      ldmatrix4_trans(b, at[n] + v_off + (8 * (i8 & 1) + r8) * 128 + (2 * d >= 8 ? half : 0) +
                             (((ch & 7) ^ r8) << 4));
    };
    // weights as the second product's A operand: rows 2t, 2t+1 and 8 on of a slice
    uint32_t w[N][4], rest[N][4];
    float x[N][G][4], mine[G];
    bool grow = false;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      mine[i] = -INFINITY;
#pragma unroll
      for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = s[n][e >> 1][0][2 * i + (e & 1)];
          if (N == 1) v += s[n][e >> 1][1][2 * i + (e & 1)];
          const int row = row0 + 8 * (e >> 1) + 2 * t + (e & 1);
          x[n][i][e] = FULL || row <= lim[i] ? v : -INFINITY;
        }
        mine[i] = fmax3(mine[i], x[n][i][0], fmax3(x[n][i][1], x[n][i][2], x[n][i][3]));
      }
      mine[i] *= p.qscale;
      grow = grow || mine[i] > ref[i] + kTau;
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        float mx = mine[i];
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float to = mx > ref[i] + kTau ? mx : ref[i];
        const float alpha = ex2(ref[i] - to);
        ref[i] = to;
        sums[2 * i] *= alpha;
        if (G == 1) sums[2] *= alpha;
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            o[j][2 * i + e] *= alpha;
            if (G == 1) o[j][2 + e] *= alpha;
          }
      }
    }
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
      for (int n = 0; n < N; ++n) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = ex2(fmaf(x[n][i][e], p.qscale, -ref[i]));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (kTwoParts) {
            split_above_zero(y[2 * j], y[2 * j + 1], w[n][2 * j + i], rest[n][2 * j + i]);
            continue;
          }
          const uint32_t hi = pack_bf16x2(y[2 * j], y[2 * j + 1]);
          w[n][2 * j + i] = hi;
          if (G == 1)
            w[n][2 * j + 1] = pack_bf16x2(y[2 * j] - bf16lo(hi), y[2 * j + 1] - bf16hi(hi));
        }
      }
    // their sums, as a product with ones
#pragma unroll
    for (int n = 0; n < N; ++n) {
      mma_bf16(sums, w[n], 0x3f803f80u, 0x3f803f80u);
      if (kTwoParts) mma_bf16(sums, rest[n], 0x3f803f80u, 0x3f803f80u);
    }
    const int seen = mt.pos + mt.n - row0;  // rows that some token may see
    const bool drafts = DRAFTS && !FULL && mt.n > 1;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        uint32_t b[4];  // 16 dims: rows 0..7 and 8..15 of the first 8, then of the others
        load_v(b, d, n);
        if (!FULL) {
          // rows past the last token may be NaN: 0 * NaN would spread
#pragma unroll
          for (int e = 0; e < 4; ++e) b[e] &= keep(seen - 8 * (e & 1) - 2 * t);
          // and so may a drafted token's be, which earlier tokens do not see
          if (drafts) {
            bool odd = false;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              odd = odd || (b[e] & 0x7f80u) == 0x7f80u || (b[e] & 0x7f800000u) == 0x7f800000u;
            if (__any_sync(0xffffffffu, odd)) {
              by_token(o[2 * d], o[2 * d + 1], w[n], b, row0, p, mt);
              if (kTwoParts) by_token(o[2 * d], o[2 * d + 1], rest[n], b, row0, p, mt);
              continue;
            }
          }
        }
        mma_bf16(o[2 * d], w[n], b[0], b[1]);
        mma_bf16(o[2 * d + 1], w[n], b[2], b[3]);
        if (kTwoParts) {
          mma_bf16(o[2 * d], rest[n], b[0], b[1]);
          mma_bf16(o[2 * d + 1], rest[n], b[2], b[3]);
        }
      }
    }
  }
  // a second MMA for the weights' rest
  static constexpr bool kTwoParts = NT == 2 || (NT == 4 && D == 128);
  // Two weights in two parts that go into the same sums.  An infinite value must get the
  // same infinity from both, so the rest has to be above zero: the first part is cut
  // off, not rounded, from a weight whose last bit is set.  (The rest is rounded to 2^-16
  // of the weight.  It is zero for weights below 2^-110, and of a weight of zero.)
  __device__ __forceinline__ static void split_above_zero(float a, float b, uint32_t& hi,
                                                          uint32_t& rest) {
    const uint32_t x = __float_as_uint(a) | 1u, y = __float_as_uint(b) | 1u;
    hi = prmt(x, y, 0x7632u);
    rest = pack_bf16x2(__uint_as_float(x) - __uint_as_float(x & 0xffff0000u),
                       __uint_as_float(y) - __uint_as_float(y & 0xffff0000u));
  }
  // Up to 8 query rows the parts have sums of their own: where the first's is infinite,
  // the rest's (of any sign, or NaN) does not count.
  __device__ __forceinline__ static float both_parts(float hi, float rest) {
    return fabsf(hi) == INFINITY ? hi : hi + rest;
  }
  // Mask of a register with two rows of which the first n (or all) count.
  __device__ __forceinline__ static uint32_t keep(int n) {
    return n >= 2 ? 0xffffffffu : n == 1 ? 0x0000ffffu : 0u;
  }
  // The same products for values b with infinities or NaN among them: token by
  // token, each with the rows that it sees, into its own rows of o0 and o1 only.
  __device__ __forceinline__ void by_token(float (&o0)[4], float (&o1)[4], const uint32_t (&w)[4],
                                           const uint32_t (&b)[4], int row0, const PagedParams& p,
                                           const TileMeta& mt) const {
#pragma unroll 1
    for (int tok = 0; tok < mt.n; ++tok) {
      uint32_t seen[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        seen[e] = b[e] & keep(mt.pos + tok + 1 - row0 - 8 * (e & 1) - 2 * t);
      float y0[4] = {0.f, 0.f, 0.f, 0.f}, y1[4] = {0.f, 0.f, 0.f, 0.f};
      mma_bf16(y0, w, seen[0], seen[1]);
      mma_bf16(y1, w, seen[2], seen[3]);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (token_of(p, G == 1 ? c : row_base + 8 * (e >> 1) + c) == tok) {
          o0[e] += y0[e];
          o1[e] += y1[e];
        }
    }
  }

  // Float index, from a tile's first byte, of dim d of a warp's partial of row c of
  // group i: in the keys (i = 0) or values of the warp's own slice, whose 16 rows
  // of 64 dims are eight of fp32; the dims of rows c turned so that a store's or a
  // load's lanes fall on different banks.
  __device__ __forceinline__ static int partial_at(int w, int i, int row, int d, int lp) {
    return (slice_at(w, lp) + i * Sh::kOp + (d >= 64 ? 128 << lp : 0)) / 4 + row * 64 +
           ((d & 63) ^ ((row & 3) << 3));
  }
  // A piece's end: the warps' partials meet in the memory of its last tile, each in
  // the slice that its warp alone has read (with two teams two warps have: they
  // wait for one another first), their (reference, sum) in ml, [query rows][warps].
  __device__ __forceinline__ void stash(const PagedParams& p, uint8_t* tile, float2* ml,
                                        ConsumerSync& csync) const {
    float* part = reinterpret_cast<float*>(tile);
    if (kTeams > 1) csync(lane);
#pragma unroll
    for (int i = 0; i < G; ++i) {
      if (t == 0)
        ml[(row_base + 8 * i + c) * kTeam + (warp & (kTeam - 1))] =
            make_float2(ref[i], G == 1 ? sums[0] + sums[2] : sums[2 * i]);
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        float2 y = make_float2(o[j][2 * i], o[j][2 * i + 1]);
        if (G == 1) y = make_float2(both_parts(y.x, o[j][2]), both_parts(y.y, o[j][3]));
        *reinterpret_cast<float2*>(part + partial_at(warp, i, c, 8 * j + 2 * t, p.lp)) = y;
      }
    }
  }
  // f(row, dim, reference, sum, four outputs) for each column of a query row,
  // merged in warp order, by `threads` threads, a power of two: as many to a row as
  // there are for R rows, so that a thread makes its row's weights once.
  template <typename F>
  __device__ __forceinline__ static void merge(const PagedParams& p, const uint8_t* tile,
                                               const float2* ml, int tid, int threads, F f) {
    const float* part = reinterpret_cast<const float*>(tile);
    int lt = D == 128 ? 5 : 4;  // log2 of the threads to a row
    while (p.R << lt > threads && lt > 1) --lt;
    for (int r = tid >> lt; r < p.R; r += threads >> lt) {
      const int tm = r / 16 * (kTeams - 1), i = r / 8 % G, row = r % 8;
      float e[kTeam], M = kMInit, L = 0.f;
      {
        float2 x[kTeam];
#pragma unroll
        for (int k = 0; k < kTeam; ++k) {
          x[k] = ml[r * kTeam + k];
          M = fmaxf(M, x[k].x);
        }
#pragma unroll
        for (int k = 0; k < kTeam; ++k) {
          e[k] = ex2(x[k].x - M);
          L = fmaf(x[k].y, e[k], L);
        }
      }
#pragma unroll 2
      for (int d = (tid & ((1 << lt) - 1)) * 4; d < D; d += 4 << lt) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kTeam; ++k) {
          const float4 v = *reinterpret_cast<const float4*>(
              part + partial_at(tm * kTeam + k, i, row, d, p.lp));
          y.x = fmaf(v.x, e[k], y.x);
          y.y = fmaf(v.y, e[k], y.y);
          y.z = fmaf(v.z, e[k], y.z);
          y.w = fmaf(v.w, e[k], y.w);
        }
        f(r, d, M, L, y);
      }
    }
  }
};

// Four dims of a query row's output; a token past the sequence's own (`idle`) gets zeros.
template <int D>
__device__ __forceinline__ void store4(const PagedParams& p, int b, int kvh, int r, int d,
                                       const float4& o, float l, bool idle) {
  const float inv = idle || l == 0.f ? 0.f : 1.f / l;
  const size_t at = query_row(p, b, kvh, r) * D + d;
  if (!range_ok(b < p.B && r < p.R && at + 4 <= (size_t)p.B * p.S * p.Hq * D, p.status)) return;
  uint2 y = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (idle) y = make_uint2(0u, 0u);
  *reinterpret_cast<uint2*>(p.out + at) = y;
}
// Sequence b's first new row and number of them, and what it is: 0 it has no
// new token, 1 its rows do not fit, 2 it takes part.
__device__ __forceinline__ int sequence(const PagedParams& p, int b, int& pos, int& n) {
  n = p.lengths ? p.lengths[b] : p.S;
  pos = p.positions[b];
  if (n == 0) return 0;
  return n > 0 && n <= p.S && n <= p.cap && rows_in_cache(pos, n - 1, p.cap) ? 2 : 1;
}
// The output rows of a sequence that takes no part, by all threads: zeros where it has
// no new token, NaN where its rows do not fit.
template <int D>
__device__ __forceinline__ void fill_rows(const PagedParams& p, int b, int tid) {
  int pos, n;
  const bool bad = sequence(p, b, pos, n) == 1;
  if (bad && tid == 0) set_status(p.status, ATTN_DEV_BAD_POSITION);
  const uint32_t v = bad ? 0x7fff7fffu : 0u;
  uint4* row = reinterpret_cast<uint4*>(p.out + (size_t)b * p.S * p.Hq * D);
  for (int i = tid; i < p.S * p.Hq * D / 8; i += kClusterThreads) row[i] = make_uint4(v, v, v, v);
}

// Where part r of a segment lies: a CTA holds at most one segment's first part
// and at most one later part.
__device__ __forceinline__ int part_slot(int c0, int r) { return 2 * (c0 + r) + (r == 0); }
__device__ __forceinline__ bool slot_ok(const PagedParams& p, int slot) {
  return range_ok(slot >= 0 && slot < 2 * kPagedMaxGrid, p.status);
}

// One column (four dims) of a split segment from N of its parts on, k0 .. k0 + N - 1,
// all loaded in one round trip, onto what the parts before gave.
struct Column {
  float M, l;
  float4 o;
};
template <int D, int N>
__device__ __forceinline__ void join_column(const PagedParams& p, const TileMeta& mt, int parts,
                                            int k0, int r, int d, Column& c) {
  float2 ml[N];
  float4 x[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    ml[k] = make_float2(kMInit, 0.f);
    x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (k0 + k < parts) {
      const size_t slot = part_slot(mt.c0, k0 + k);
      ml[k] = __ldcg(reinterpret_cast<const float2*>(p.part_ml + (slot * p.R + r) * 2));
      x[k] = __ldcg(reinterpret_cast<const float4*>(p.part_o + (slot * p.R + r) * D + d));
    }
  }
  float top = c.M;
#pragma unroll
  for (int k = 0; k < N; ++k) top = fmaxf(top, ml[k].x);
  const float a = ex2(c.M - top);
  c.M = top;
  c.l *= a;
  c.o = make_float4(c.o.x * a, c.o.y * a, c.o.z * a, c.o.w * a);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float e = ex2(ml[k].x - top);
    c.l = fmaf(ml[k].y, e, c.l);
    c.o.x = fmaf(x[k].x, e, c.o.x);
    c.o.y = fmaf(x[k].y, e, c.o.y);
    c.o.z = fmaf(x[k].z, e, c.o.z);
    c.o.w = fmaf(x[k].w, e, c.o.w);
  }
}
// Merge the parts of a split segment, in CTA order.
template <int D>
__device__ __forceinline__ void merge_parts(const PagedParams& p, const TileMeta& mt, int tid,
                                            int threads) {
  const int parts = slot_ok(p, part_slot(mt.c0, mt.parts - 1)) ? mt.parts : 0;
  const int cols = p.R * (D / 4);
  if (parts <= 2) {  // most segments: four columns in one round trip
    for (int c0 = tid; c0 < cols; c0 += 4 * threads) {
      Column c[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int col = c0 + u * threads, r = col / (D / 4), d = col % (D / 4) * 4;
        c[u] = Column{kMInit, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
        if (col < cols) join_column<D, 2>(p, mt, parts, 0, r, d, c[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int col = c0 + u * threads, r = col / (D / 4), d = col % (D / 4) * 4;
        if (col < cols)
          store4<D>(p, mt.b, mt.kvh, r, d, c[u].o, c[u].l, token_of(p, r) >= mt.n);
      }
    }
    return;
  }
  for (int col = tid; col < cols; col += threads) {
    const int r = col / (D / 4), d = col % (D / 4) * 4;
    Column c{kMInit, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int k0 = 0; k0 < parts; k0 += 8) join_column<D, 8>(p, mt, parts, k0, r, d, c);
    store4<D>(p, mt.b, mt.kvh, r, d, c.o, c.l, token_of(p, r) >= mt.n);
  }
}

constexpr int kNoRows = -0x7fffffff - 1;  // a table entry that holds no attended rows
// A table entry that does; -1 where it names no page.
__device__ __forceinline__ int page_ok(const PagedParams& p, int page) {
  if (page >= 0 && page < p.P) return page;
  set_status(p.status, ATTN_DEV_BAD_PAGE);
  return -1;
}

// A piece's output: whole, or this CTA's part of a segment.
template <int D, int NT, bool DRAFTS>
__device__ __forceinline__ void put_piece(const PagedParams& p, const TileMeta& mt,
                                          const uint8_t* tile, const float2* ml, int tid,
                                          int threads) {
  if (mt.parts == 1) {
    auto whole = [&](int r, int d, float, float l, const float4& o) {
      store4<D>(p, mt.b, mt.kvh, r, d, o, l, token_of(p, r) >= mt.n);
    };
    PagedConsumer<D, NT, DRAFTS>::merge(p, tile, ml, tid, threads, whole);
    return;
  }
  const int slot = part_slot(mt.c0, (int)blockIdx.x - mt.c0);
  auto part = [&](int r, int d, float m, float l, const float4& o) {
    if (!slot_ok(p, slot)) return;
    *reinterpret_cast<float4*>(p.part_o + ((size_t)slot * p.R + r) * D + d) = o;
    if (d == 0)
      *reinterpret_cast<float2*>(p.part_ml + ((size_t)slot * p.R + r) * 2) = make_float2(m, l);
  };
  PagedConsumer<D, NT, DRAFTS>::merge(p, tile, ml, tid, threads, part);
}
// The CTA's part is written (by threads that `sync` joins): the last CTA of the
// segment's to come here merges the parts.
template <int D>
__device__ __forceinline__ void join_parts(const PagedParams& p, const TileMeta& mt, int tid,
                                           int threads, ConsumerSync& sync, int* flag, int lane) {
  sync(lane);
  if (tid == 0) {
    uint32_t* counter = p.counters + mt.b * p.Hkv + mt.kvh;
    __threadfence();  // (the other threads' stores came before the barrier)
    const bool last = !*sync.abort_flag && atomicAdd(counter, 1u) + 1 == (uint32_t)mt.parts;
    if (last) *counter = 0;
    __threadfence();
    *flag = last;
  }
  sync(lane);
  if (*(volatile int*)flag && !*sync.abort_flag) merge_parts<D>(p, mt, tid, threads);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Many short segments: a warp takes a whole segment (with more than 16 query rows,
// half of its query rows), 16 cache rows at a time, by copies of its own into
// `room` bytes of shared memory of its own.  A CTA that takes a segment at a time has
// three under way and pays for each one's copy, merge and hand-over in turn; here
// there are eight, and nothing to merge.  (4 query rows: 160 segments of up to 32 rows
// 7.8 -> 4.9 us, of 128 8.2 and 9.6; 912 of 32 rows 12.8 -> 5.4, of 128 15.2 -> 11.3, of
// 256 20.5 -> 19.1.)  Neighbouring units go to different CTAs: 192 segments of 160 rows in
// 24 full CTAs took 12.7 us, a warp in each CTA 11.1.
//
// With several tokens and 128 dims it is a call: inlined, it cost the tiles' loop registers
// (32 sequences up to 16000 rows, 32 query rows a head: 173.5 -> 176.5 us, 16: 147 ->
// 148.5).  The call costs short segments 2 us, the other forms do without.  It takes its
// parameters from shared memory (by reference each use was a load, 5% slower), and all
// warps (8 where it is inlined: with 12, which leave less room for each, 16 query rows
// were 20% slower; with 32 and a call 912 segments of 128 rows went from 36.4 to 22.6 us).
template <int D, bool DRAFTS>
constexpr bool kShortCall = D == 128 && DRAFTS;
template <int D, bool DRAFTS>
constexpr int kShortWarps = kShortCall<D, DRAFTS> ? kThreads / 32 : kWarps;
template <int D, int NT, bool DRAFTS>
__device__ __forceinline__ void short_segments(const PagedParams& p, const int* prefix,
                                               const int* spos, const uint8_t* snew, uint8_t* own,
                                               int room, int warp, int lane) {
  using Sh = Shape<D, NT>;
  using Consumer = PagedConsumer<D, NT, DRAFTS>;
  constexpr int kG = Consumer::G, kTeams = Consumer::kTeams, kRows = 8 * kG;
  // (with all warps the query rows go through the buffer that is filled last)
  constexpr bool kAll = kShortCall<D, DRAFTS>;
  constexpr int kBuf = 16 * D * 4, kQBytes = kRows * Sh::kQStride;
  static_assert(kQBytes <= kBuf, "the query rows' place");
  const int bufs = min(4, (room - (kAll ? 0 : kQBytes)) / kBuf);
  uint8_t* qs = own + (bufs - kAll) * kBuf;
  Consumer cs;
  cs.init(0, lane);
  const long long units = (long long)p.B * p.Hkv * kTeams;
  for (long long u = blockIdx.x + (long long)gridDim.x * warp; u < units;
       u += (long long)gridDim.x * kShortWarps<D, DRAFTS>) {
    const int team = (int)(u % kTeams), seg = (int)(u / kTeams);
    const int b = seg / p.Hkv, kvh = seg - b * p.Hkv;
    if (prefix[b + 1] == prefix[b]) continue;
    TileMeta mt = {};
    mt.pos = spos[b];
    mt.n = snew[b];
    const int rows = mt.pos + mt.n, slices = (rows + 15) >> 4;
    const int mask = (1 << p.lp) - 1;
    // table entries, a lane for each slice
    const int j = (16 * lane) >> p.lp;
    const int entries =
        lane < slices && range_ok(j < p.M, p.status) ? p.table[(size_t)b * p.M + j] : 0;
    cs.row_base = 16 * team;
    // the query rows, zeros behind the last
#pragma unroll
    for (int i = lane; i < kRows * (D / 8); i += 32) {
      const int r = i / (D / 8), ch = i % (D / 8), row = 16 * team + r;
      const uint4 x = row < p.R ? *reinterpret_cast<const uint4*>(
                                      p.q + query_row(p, b, kvh, row) * D + ch * 8)
                                : make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4*>(qs + r * Sh::kQStride + ch * 16) = x;
    }
    // 16 rows of keys and values, as a page of 16 lies in a tile
    uint32_t there = 0;  // of the buffers: which hold rows
    auto load = [&](int i) {
      // (i is a lane.  Without the second limit the kernel for 16 query rows spilled 32 bytes
      // instead of 20: 512 sequences, 8 heads, of up to 32 rows 29.4 us, with it 23.3.)
      if (i < min(slices, 32)) {
        const int pg = page_ok(p, __shfl_sync(0xffffffffu, entries, i));
        const int buf = i % bufs;
        there = pg >= 0 ? there | 1u << buf : there & ~(1u << buf);
        if (pg >= 0) {
          const long long at = pg * p.page_stride + kvh * p.head_stride +
                               (long long)((16 * i) & mask) * p.row_stride;
          const uint32_t dst = smem_u32(own + buf * kBuf);
#pragma unroll
          for (int k = 0; k < 16 * (D / 8) / 32; ++k) {
            const int j = lane + 32 * k, r = j / (D / 8), ch = j % (D / 8);
            if (16 * i + r < rows) {
              const long long e = at + r * p.row_stride + ch * 8;
              const uint32_t to = dst + (ch >> 3) * 2048 + sw128(r, ch & 7);
              cp_async16(to, p.k + e);
              cp_async16(to + 16 * D * 2, p.v + e);
            }
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int i = 0; i < bufs - 1; ++i) load(i);
    __syncwarp();
    cs.load_q(qs - 16 * team * Sh::kQStride, p.flip);
    if (kAll) __syncwarp();
    cs.start(p, mt.pos, mt.n);
    for (int i = 0; i < slices; ++i) {
      load(i + bufs - 1);
      // all but the newest bufs - 1 have landed
      if (bufs == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
      else if (bufs == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
      else if (bufs == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
      else asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncwarp();
      const int buf = i % bufs;
      if (there >> buf & 1) {
        const uint32_t at = smem_u32(own + buf * kBuf);
        if (16 * i + 15 <= mt.pos)
          cs.template slices<1, true>(at, at, 2048, 16 * D * 2, 16 * i, p, mt);
        else
          cs.template slices<1, false>(at, at, 2048, 16 * D * 2, 16 * i, p, mt);
      }
      __syncwarp();  // the buffer may be written again
    }
#pragma unroll
    for (int i = 0; i < kG; ++i) {
      const int r = 16 * team + 8 * i + cs.c;
      const float l = kG == 1 ? cs.sums[0] + cs.sums[2] : cs.sums[2 * i];
      const bool idle = token_of(p, r) >= mt.n;
      const float inv = idle || l == 0.f ? 0.f : 1.f / l;
      if (r >= p.R) continue;
      uint16_t* out = p.out + query_row(p, b, kvh, r) * D + 2 * cs.t;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        float2 y = make_float2(cs.o[j][2 * i], cs.o[j][2 * i + 1]);
        if (kG == 1)
          y = make_float2(cs.both_parts(y.x, cs.o[j][2]), cs.both_parts(y.y, cs.o[j][3]));
        *reinterpret_cast<uint32_t*>(out + 8 * j) =
            idle ? 0u : pack_bf16x2(y.x * inv, y.y * inv);
      }
    }
  }
}

template <int D, int NT, bool DRAFTS>
__device__ __noinline__ void short_segments_call(const PagedParams& p, const int* prefix,
                                                 const int* spos, const uint8_t* snew,
                                                 uint8_t* own, int room, int warp, int lane) {
  short_segments<D, NT, DRAFTS>(p, prefix, spos, snew, own, room, warp, lane);
}

template <int D, int NT, bool DRAFTS>
__global__ void __launch_bounds__(kThreads, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const PagedParams p) {
  using Sh = Shape<D, NT>;
  constexpr int kE = kEndUnits<NT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int NS = p.stages, B = p.B, Hkv = p.Hkv;
  uint8_t* stages = smem;
  uint8_t* qbuf = stages + (size_t)NS * Sh::kStage;            // [NS][NT * 8] query rows
  TileMeta* meta = reinterpret_cast<TileMeta*>(qbuf + NS * Sh::kQ);
  float2* ml = reinterpret_cast<float2*>(meta + NS);             // [query rows][warps]
  // full [NS], empty [NS], the consumers' and the merge warps' sync, merge full [2], empty [2]
  uint64_t* bars = reinterpret_cast<uint64_t*>(ml + Sh::kMl / 8);
  uint64_t* m_full = bars + 2 * NS + 2;
  uint64_t* m_empty = m_full + 2;
  // [0] abort, [1] last to arrive (consumers), [2] longest segment's rows, [3] last to arrive (merge
  // warps), [4..6) stage of the piece's last tile, [8..16) scan
  int* misc = reinterpret_cast<int*>(m_empty + 2);
  int* prefix = misc + 16;                                // [B + 1]
  int* spos = prefix + B + 1;                             // [B]
  uint8_t* snew = reinterpret_cast<uint8_t*>(spos + B);   // [B]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = misc;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(&bars[s]), 2);  // keys, values
      mbar_init(smem_u32(&bars[NS + s]), kWarps);
    }
    mbar_init(smem_u32(&bars[2 * NS]), kWarps);
    mbar_init(smem_u32(&bars[2 * NS + 1]), kMergeThreads / 32);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&m_full[i]), kWarps);
      mbar_init(smem_u32(&m_empty[i]), kMergeThreads / 32);
    }
    misc[0] = misc[2] = 0;
    fence_mbar_init();
  }
  prefetch_maps(tm_k, tm_v, warp, lane);
  for (int i = tid; i < NS * Sh::kQ / 16; i += kThreads)  // rows past R stay zero
    reinterpret_cast<uint4*>(qbuf)[i] = make_uint4(0u, 0u, 0u, 0u);
  // (they come before the query copies that land over them)
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  grid_dependency_wait();
  grid_dependents_launch();

  // ---- units per sequence and KV head, their exclusive prefix sum (every CTA)
  int carry = 0;
  for (int base = 0; base < B; base += kConsumers) {
    const int b = base + tid;
    int v = 0, rows = 0;
    if (tid < kConsumers && b < B) {
      int pos, n;
      const int kind = sequence(p, b, pos, n);
      spos[b] = pos;
      snew[b] = (uint8_t)n;
      if (kind == 2) {
        rows = pos + n;
        v = (rows - 1) / Sh::kTile + 1 + kE;
      }
    }
    const int most = __reduce_max_sync(0xffffffffu, rows);
    if (lane == 0 && warp < kWarps) atomicMax(misc + 2, most);
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

  for (int b = blockIdx.x; b < B; b += gridDim.x)
    if (tid < kClusterThreads && prefix[b + 1] == prefix[b]) fill_rows<D>(p, b, tid);  // no part

  const long long T = (long long)Hkv * carry;  // all units
  const long long nseg = (long long)B * Hkv;
  long long gw = min((long long)gridDim.x, T);
  if (T <= (long long)(kWholeTiles + kE) * nseg) gw = min(gw, nseg);
  // Short segments: the more a CTA has, the longer they may be: 96, 160, 224 and 256 rows
  // for 2, 3, 4 and more of them (128 at most with 32 query rows at 128 dims), where the call
  // below is taken 64, 96 and 128.  Tiles and warps, in us, ragged segments up to so many rows:
  //   4 query rows          304 segments:  96 8.5 and 8.2, 128 8.7 and 9.9; 456: 160 12.2 and
  //                         11.6, 192 12.6 and 13.2; 608: 224 16.1 and 15.6, 256 16.8 and 17.3;
  //                         760: 256 19.3 and 19.3, 320 21.6 and 22.5
  //   16 of several tokens  304: 32 11.0 and 9.9, 64 11.3 and 11.9; 456: 96 13.8 and 14.6; 608: 96
  //                         16.2 and 14.8, 128 16.9 and 17.9; 912: 128 23.3 and 20.3
  // Segments per CTA are rounded up; just above a whole number the warps' limit is too long
  // (312 of up to 160 rows: 9.9 and 11.5).
  constexpr int kWarpRows = D == 128 && (NT == 4 || DRAFTS) ? 128 : 256;
  static_assert(kWarpRows <= 16 * 32, "a lane for each slice's table entry");
  const int per_cta = (int)((nseg + gridDim.x - 1) / gridDim.x);
  if (per_cta > 1 &&
      misc[2] <= min(kWarpRows, kShortCall<D, DRAFTS> ? 32 * per_cta : 64 * per_cta - 32)) {
    constexpr int kShort = kShortWarps<D, DRAFTS>;
    PagedParams* shared = reinterpret_cast<PagedParams*>(qbuf);
    static_assert(sizeof(PagedParams) <= 2 * Sh::kQ);
    if (kShortCall<D, DRAFTS>) {
      if (tid == 0) *shared = p;  // over the query rows, which no copy fills here
      __syncthreads();
    }
    if (warp < kShort) {
      const int room = (NS * Sh::kStage / kShort) & ~1023;
      uint8_t* own = stages + warp * room;
      if constexpr (kShortCall<D, DRAFTS>)
        short_segments_call<D, NT, DRAFTS>(*shared, prefix, spos, snew, own, room, warp, lane);
      else
        short_segments<D, NT, DRAFTS>(p, prefix, spos, snew, own, room, warp, lane);
    }
    return;
  }
  // A CTA for each segment where the longest alone takes no longer than an even
  // share of the tiles and the merge of a split segment would.
  const int longest = ((misc[2] + Sh::kTile - 1) / Sh::kTile) + kE;
  const bool whole =
      nseg <= (long long)gridDim.x &&
      longest * kWholeNum * gw <= T * kWholeDen + kMergeCost<D> * gw;
  const int G = whole ? (int)nseg : (int)gw;
  if ((int)blockIdx.x >= G) return;
  FlatRange rg;
  if (whole) {
    const int b = (int)blockIdx.x / Hkv, n = prefix[b + 1] - prefix[b];
    rg.t0 = (long long)Hkv * prefix[b] + (long long)((int)blockIdx.x - b * Hkv) * n;
    rg.t1 = rg.tA = rg.t0 + n;
  } else {
    flat_range<kE>(rg, T, blockIdx.x, G, prefix, B, Hkv);
  }
  if (rg.t0 >= rg.t1) return;
  FlatWalk w;
  flat_start<kE>(w, rg, prefix, spos, B, Hkv);
  if (w.u >= w.end) return;  // end units alone

  if (warp >= kWarps + 2) {
    // --------------------------------------------------------------- merge --
    // The consumers leave a piece's partials in its last tile and go on; these
    // two warps write its output, or its part of a segment's, give the tile back to
    // the ring, and settle who merges the parts.  (64 sequences of up to 1000 rows, 4
    // query rows: 32.1 -> 30.4 us.)  The last piece is the consumers', who have
    // nothing else to do.
    const int mtid = tid - kClusterThreads;
    ConsumerSync msync{smem_u32(&bars[2 * NS + 1]), abort_flag, p.status, 0u};
    for (int turn = 0;; ++turn) {
      const int buf = turn & 1;
      if (!consumer_wait(smem_u32(&m_full[buf]), (turn >> 1) & 1u, abort_flag, p.status, lane))
        break;
      const int s = *(volatile int*)(misc + 4 + buf);
      if (s < 0) break;
      const TileMeta mt = meta[s];
      put_piece<D, NT, DRAFTS>(p, mt, stages + (size_t)s * Sh::kStage,
                               ml + buf * (Sh::kMl / 16), mtid, kMergeThreads);
      __syncwarp();
      if (lane < kWarps * 32 / kMergeThreads) mbar_arrive(smem_u32(&bars[NS + s]));  // for all
      if (lane == 0) mbar_arrive(smem_u32(&m_empty[buf]));
      if (mt.parts > 1)
        join_parts<D>(p, mt, mtid, kMergeThreads, msync, misc + 3, lane);
    }
  } else if (warp >= kWarps) {
    // ----------------------------------------------------------- producers --
    // Tiles go in batches of kBatch, lane kSlices * ti + slice looks after slice
    // `slice` of the batch's tile ti; a batch's table entries are loaded while
    // the one before it is issued.
    constexpr int kSlices = Sh::kSlices, kBatch = Sh::kBatch;
    const bool keys = warp == kWarps;  // this warp also describes the tile, the other brings the
                                       // queries
    const int ti = lane / kSlices, slice = lane % kSlices;
    const int page_rows = 1 << p.lp, in_page = (slice * 16) & (page_rows - 1);
    // The slice's table entry, kNoRows where it holds none; looked at a batch later.
    auto fetch = [&](const FlatWalk& w) -> int {
      const int row = w.k * Sh::kTile + slice * 16;
      if (w.u >= w.end || row > w.pos + snew[w.b] - 1) return kNoRows;
      if (!range_ok((row >> p.lp) < p.M, p.status)) return kNoRows;
      return p.table[(size_t)w.b * p.M + (row >> p.lp)];
    };
    // This lane's tile of the batch that starts at w, which goes on to the next one
    // (the whole warp walks alike: lanes that walked for themselves took turns).
    auto take = [&](FlatWalk& w) -> FlatWalk {
      FlatWalk mine = w;
      if (w.k + kBatch < w.nt && w.u + kBatch < w.end) {
        mine.k += ti;
        mine.u += ti;
        w.k += kBatch;
        w.u += kBatch;
        return mine;
      }
#pragma unroll 1
      for (int k = 0; k < kBatch; ++k) {
        if (k == ti) mine = w;
        if (w.u < w.end) flat_next<kE>(w, rg, prefix, spos, B, Hkv);
      }
      return mine;
    };
    long long last_end = w.end;  // of the part of the range done last
    if (rg.tA < rg.t1) {
      FlatWalk rest;
      flat_init<kE>(rest, rg.t0, prefix, spos, B, Hkv);
      if (rest.u < rg.tA) last_end = rg.tA;
    }
    auto describe = [&](const FlatWalk& w, TileMeta& m) {
      const long long f0 = w.u - w.k;  // the segment's first unit
      const long long from = w.end == rg.t1 && rg.tA < rg.t1 ? rg.tA : rg.t0;
      m.flags = 0;
      if (w.k == 0 || w.u == rg.t0) m.flags |= kStarts;
      if (w.k == w.nt - 1 || w.u + 1 == w.end) m.flags |= kEnds;
      // the CTA's last tile: none in what is left of this part of the range (the
      // next one would come after the end units), nor a part after it
      if (w.u + 1 + (w.k == w.nt - 1 ? kE : 0) >= w.end && w.end == last_end) m.flags |= kLast;
      m.row0 = w.k * Sh::kTile;
      m.pos = w.pos;
      m.n = snew[w.b];
      m.b = w.b;
      m.kvh = w.kvh;
      m.c0 = 0;
      m.parts = 1;
      if ((m.flags & kEnds) && !(f0 >= from && f0 + w.nt <= w.end)) {
        m.c0 = cta_of(f0, T, G);
        m.parts = cta_of(f0 + w.nt - 1, T, G) - m.c0 + 1;
      }
    };
    int s = 0;
    uint32_t pass = 0;
    FlatWalk cur = take(w);
    int entry = fetch(cur);
    bool ok = true;
    while (ok) {
      const bool on = cur.u < cur.end;
      const int n_q = __popc(__ballot_sync(0xffffffffu, on)) / kSlices;  // tiles of the batch
      if (n_q == 0) break;
      const FlatWalk ahead = take(w);
      const int next = fetch(ahead);
      const int page = entry == kNoRows ? -1 : page_ok(p, entry);
      TileMeta mt = {};
      if (keys && on && slice == 0) describe(cur, mt);
      const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
      const bool lead = page >= 0 && in_page == 0;
      const uint32_t copies = __ballot_sync(0xffffffffu, lead);
      const bool skip = on && p.test_skip >= 0 && cur.b == 0 && cur.kvh == 0 &&
                        cur.k == p.test_skip;  // failure-path tests only
      for (int q = 0; q < n_q; ++q) {
        if (pass > 0 && !__all_sync(0xffffffffu, mbar_wait(smem_u32(&bars[NS + s]),
                                                           (pass & 1u) ^ 1u, abort_flag))) {
          if (lane == 0) {
            *abort_flag = 1;
            set_status(p.status, ATTN_DEV_TIMEOUT);
          }
          ok = false;
          break;
        }
        const uint32_t full = smem_u32(&bars[s]);
        const bool first = __shfl_sync(0xffffffffu, cur.k == 0 || cur.u == rg.t0, kSlices * q);
        if (lane == kSlices * q) {
          mt.flags |= (there >> (kSlices * q)) & ((1u << kSlices) - 1u);
          if (keys) meta[s] = mt;
          if (!skip)
            mbar_arrive_expect_tx(full, __popc((copies >> (kSlices * q)) & ((1u << kSlices) - 1u)) *
                                                ((uint32_t)page_rows * D * 2u) +
                                            (!keys && first ? (uint32_t)p.R * D * 2u : 0u));
        }
        __syncwarp();
        const bool hold = __shfl_sync(0xffffffffu, skip, kSlices * q);
        if (ti == q && lead && !hold) {
          const uint32_t dst = smem_u32(stages + (size_t)s * Sh::kStage) + slice * 16 * D * 2;
          tma_load_5d(dst + (keys ? 0 : Sh::kOp), keys ? &tm_k : &tm_v, 0, 0, 0, cur.kvh, page,
                      full);
        }
        if (first && !hold && !keys) {  // the piece's query rows, one by each lane
          const int b = __shfl_sync(0xffffffffu, cur.b, kSlices * q);
          const int kvh = __shfl_sync(0xffffffffu, cur.kvh, kSlices * q);
          if (lane < p.R)
            bulk_load(smem_u32(qbuf + s * Sh::kQ) + lane * Sh::kQStride,
                      p.q + query_row(p, b, kvh, lane) * D, D * 2, full);
        }
        if (++s == NS) {
          s = 0;
          ++pass;
        }
      }
      cur = ahead;
      entry = next;
    }
  } else {
    // ----------------------------------------------------------- consumers --
    ConsumerSync csync{smem_u32(&bars[2 * NS]), abort_flag, p.status, 0u};
    PagedConsumer<D, NT, DRAFTS> cs;
    cs.init(warp, lane);
    int s = 0, turn = 0;
    uint32_t ph = 0;
    for (;;) {
      if (!consumer_wait(smem_u32(&bars[s]), ph, abort_flag, p.status, lane)) break;
      const int flags = meta[s].flags;
      uint8_t* tile = stages + (size_t)s * Sh::kStage;
      if (flags & kStarts) {
        cs.load_q(qbuf + s * Sh::kQ, p.flip);
        cs.start(p, meta[s].pos, meta[s].n);
      }
      cs.tile(tile, p, meta[s]);
      if (flags & kEnds) {
        const int buf = turn & 1;
        float2* to = ml + buf * (Sh::kMl / 16);
        if (turn > 1 && !consumer_wait(smem_u32(&m_empty[buf]), ((turn >> 1) & 1u) ^ 1u,
                                       abort_flag, p.status, lane))
          break;
        ++turn;
        if (tid == 0) misc[4 + buf] = flags & kLast ? -1 : s;
        cs.stash(p, tile, to, csync);
        // (this memory was written here; copies land in it next)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&m_full[buf]));
        if (flags & kLast) {
          csync(lane);
          if (*abort_flag) break;
          const TileMeta mt = meta[s];
          put_piece<D, NT, DRAFTS>(p, mt, tile, to, tid, kConsumers);
          if (mt.parts > 1) join_parts<D>(p, mt, tid, kConsumers, csync, misc + 1, lane);
          break;
        }
      } else {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars[NS + s]));
      }
      if (++s == NS) {
        s = 0;
        ph ^= 1u;
      }
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

#include "paged_cluster.cuh"

namespace gqa {
namespace {

// ------------------------------------------------------------------ host --

template <int D, int NT>
size_t flat_smem_bytes(int stages, int B) {
  using Sh = Shape<D, NT>;
  return (size_t)stages * (Sh::kStage + Sh::kQ + sizeof(TileMeta) + 16) + Sh::kMl + 48 + 64 +
         (size_t)9 * B + 16;
}

// Per device, found once: its SMs and how many clusters of each size can run
// at once with one CTA to an SM (a cluster stays within one GPC).
struct PagedDevice {
  int sms;
  int clusters[kMaxCluster + 1];
};

template <int D, int NT, bool DRAFTS>
cudaError_t set_attributes() {
  cudaError_t e = cudaFuncSetAttribute(
      paged_decode_kernel<D, NT, DRAFTS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(paged_cluster_kernel<D, NT, DRAFTS>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(paged_cluster_kernel<D, NT, DRAFTS>,
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e;
}

template <int D, bool DRAFTS>
cudaError_t find_device(PagedDevice& d, int dev) {
  cudaError_t e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = set_attributes<D, 1, DRAFTS>();
  if (e == cudaSuccess) e = set_attributes<D, 2, DRAFTS>();
  if (e == cudaSuccess) e = set_attributes<D, 4, DRAFTS>();
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
    if (cudaOccupancyMaxActiveClusters(&d.clusters[c], paged_cluster_kernel<D, 1, DRAFTS>, &cfg) !=
        cudaSuccess) {
      cudaGetLastError();
      d.clusters[c] = 0;
    }
  }
  return cudaSuccess;
}

template <int D, bool DRAFTS>
cudaError_t paged_device(const PagedDevice** out) {
  static PagedDevice known[64];
  static std::atomic<bool> ready[64];
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev < 0 || dev >= 64)) e = cudaErrorInvalidDevice;
  if (e != cudaSuccess) return e;
  if (!ready[dev].load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev].load(std::memory_order_relaxed)) {
      e = find_device<D, DRAFTS>(known[dev], dev);
      if (e != cudaSuccess) return e;
      ready[dev].store(true, std::memory_order_release);
    }
  }
  *out = &known[dev];
  return cudaSuccess;
}

// CTAs per segment in cluster mode, or 0 for the split over a flat list.  The
// cluster would be the largest that lets every segment have its own resident at
// once, or one CTA; it is taken where it should be faster.  The host knows only
// what the table can hold: positions are taken as spread evenly over that.  In
// us, measured (D = 128; a tile at D = 64 takes half):
//   all SMs    1.45 for each tile of an SM's even share
//   clusters   4.3, then the even share and 15% of it, or 0.62 for each tile of the
//              longest segment's CTAs where that is more
//   flat list  12 (scan, lookups, the merge of split segments) and the even share
// With more segments than SMs it is the flat list, which sees on the device how
// long they are.
// (2 sequences up to 8192 rows, 8 heads: 17 in clusters, 21 by the list; 10 up to
// 16000: 74 and 50.)
template <int D, int NT>
int cluster_size(const PagedParams& p, const PagedDevice& d) {
  constexpr int kTile = Shape<D, NT>::kTile;
  if (g_decode_test_cluster >= 0)  // schedule tests only
    return min(g_decode_test_cluster, kMaxCluster);
  const long long nseg = (long long)p.B * p.Hkv;
  if (nseg > d.sms) return 0;
  const int tiles = (p.cap + kTile - 1) / kTile;
  int c = min(kMaxCluster, tiles);
  while (c > 1 && nseg > d.clusters[c]) --c;
  const float longest = (float)tiles * (float)p.B / (float)(p.B + 1);
  const float per_tile = D == 128 ? 1.45f : 0.75f;
  const float share = per_tile * 0.5f * (float)tiles * (float)nseg / (float)d.sms;
  const float clusters =
      4.3f + fmaxf(1.15f * share, 0.43f * per_tile * ceilf(longest / (float)c));
  return clusters <= 12.f + share ? c : 0;
}

template <int D, int NT, bool DRAFTS>
cudaError_t launch_paged(PagedParams& p, const PagedPool& pool, cudaStream_t stream) {
  const PagedDevice* d = nullptr;
  cudaError_t e = paged_device<D, DRAFTS>(&d);
  if (e != cudaSuccess) return e;
  CUtensorMap mk, mv;
  if (!paged_maps(pool, &mk, &mv)) return cudaErrorInvalidValue;
  p.stages = kMaxStages;
  const int C = cluster_size<D, NT>(p, *d);
  if (C > 0) {
    if (d->clusters[C] == 0) return cudaErrorNotSupported;
    while (p.stages > 2 && cluster_smem_bytes<D, NT>(p.stages, p.R, C) > (size_t)kMaxSmem)
      --p.stages;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.B * p.Hkv * C));
    cfg.blockDim = dim3(kClusterThreads);
    cfg.dynamicSmemBytes = cluster_smem_bytes<D, NT>(p.stages, p.R, C);
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
    e = cudaLaunchKernelEx(&cfg, paged_cluster_kernel<D, NT, DRAFTS>, mk, mv, p);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  while (p.stages > 2 && flat_smem_bytes<D, NT>(p.stages, p.B) > (size_t)kMaxSmem) --p.stages;
  return launch_pdl(paged_decode_kernel<D, NT, DRAFTS>, dim3(min(kPagedMaxGrid, d->sms)), dim3(kThreads),
                    flat_smem_bytes<D, NT>(p.stages, p.B), stream, mk, mv, p);
}

template <int D, bool DRAFTS>
cudaError_t launch_paged_rows(PagedParams& p, const PagedPool& pool, cudaStream_t stream) {
  return p.R <= 8    ? launch_paged<D, 1, DRAFTS>(p, pool, stream)
         : p.R <= 16 ? launch_paged<D, 2, DRAFTS>(p, pool, stream)
                     : launch_paged<D, 4, DRAFTS>(p, pool, stream);
}

}  // namespace
}  // namespace gqa
