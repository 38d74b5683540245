// paged_decode.cuh -- split-KV decode attention over a paged bf16 cache, S new
// tokens per sequence: the kernels and their launch, included by one
// translation unit per head dim (paged_decode_d64.cu, paged_decode_d128.cu).
//
// For sequence b, new token t, query head h and KV head h/g:
//   out = softmax_j(scale q . K_j) V_j      over rows j = 0 .. positions[b] + t,
// row j in row j % page of page table[b][j / page].  The R = S g <= 32 query
// rows of a KV head share one pass over its keys and values: with x_j the score
// in base 2, M a reference at most 2^64 below the largest x_j so far and
// w_j = 2^(x_j - M),
//   out = sum_j w_j V_j / sum_j w_j.
//
// Bound by memory: a cache row costs 4 D bytes for K and V.  How:
//  * 128-row tiles stream through a shared-memory ring by tiled TMA copies with
//    the 128-byte swizzle, one copy per page and operand: the pool is a 5-D
//    tensor (dims, rows, dim halves, heads, pages), so any strides will do and
//    a page's rows land where a contiguous tile's would.  One producer warp
//    looks up table entries four tiles ahead (a lane per 16 rows) and issues.
//  * 8 consumer warps.  Scores: each takes 16 rows, S = q K^T with the query
//    rows as M (m16n8k16, bf16 in, fp32 out).  The weights go to shared memory
//    as bf16, and for the second product each warp takes 16 dims of all 128
//    rows (for D = 64: of 64), so a warp holds R x 16 outputs instead of R x D,
//    a segment's end needs no merge among warps, and R can be 32.
//  * One barrier a tile: the weights are relative to a reference that earlier
//    tiles settled, and each tile's maximum, published with them, moves it for
//    the next.  Only where a tile's maximum lies 2^64 above the reference (and
//    in a piece's first tile) are the weights made again.
//  * Up to 8 rows the weights enter as two bf16 parts for nothing: rows 8..15
//    of the MMA's M are free and take the rest (16 bits).  Up to 16 rows they
//    take a second MMA.  Beyond, the weights are rounded to bf16 once (2^-9,
//    of errors that average over the keys; the output's own rounding is the
//    same size).
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

constexpr int kTile = 128;
constexpr int kSlices = kTile / 16;
constexpr int kWarps = 8;                   // consumer warps
constexpr int kConsumers = kWarps * 32;
constexpr int kThreads = kConsumers + 32;   // and the producer
constexpr int kMaxStages = 6;
constexpr int kMaxSmem = 227 * 1024;
constexpr int kE = 1;                       // units of a segment's end (flat_list.cuh)
constexpr int kWholeTiles = 4;              // segments this short are not split
constexpr int kMaxCluster = 16;
constexpr float kMInit = -3e38f;            // the reference before any row
constexpr float kTau = 8.f;                 // it moves when a maximum lies 2^kTau above
constexpr float kFar = 64.f;                // and before the weights, not after, beyond 2^kFar
constexpr int kPStride = kTile * 2 + 16;    // bytes between rows of weights: no bank conflicts

constexpr int kSlicesMask = 0xff;  // TileMeta::flags: slices that hold rows
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
  static constexpr int kOp = kTile * D * 2;       // bytes of a tile's keys
  static constexpr int kStage = 2 * kOp;
  static constexpr int kQStride = D * 2 + 16;     // bytes between query rows: no bank conflicts
  static constexpr int kQ = NT * 8 * kQStride;
  static constexpr int kPRows = NT == 1 ? 16 : 32;  // rows of weights, both parts
  static constexpr int kP = kPRows * kPStride;
  static constexpr int kHalves = 128 / D;         // warps that share 16 dims, half of the rows each
  static constexpr int kO = kHalves > 1 ? NT * 8 * (D + 8) * 4 : 0;
  static constexpr int kFixed = 2 * kP + kO + 3 * NT * 8 * 8 * 4 + 128;
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

// Row of q and out that query row r of (b, kvh) is: rows are ordered token, head.
__device__ __forceinline__ size_t query_row(const PagedParams& p, int b, int kvh, int r) {
  const int t = r / p.g;
  return ((size_t)b * p.S + t) * p.Hq + (size_t)kvh * p.g + (r - t * p.g);
}

// A consumer warp.  Lane 4c + t.  Query rows are r = 8 i + c for group i < NT;
// MMA m-block m holds groups 2m and 2m + 1 as its rows c and c + 8 (NT = 1:
// rows 8..15 are zero queries, and in the second product the weights' rest).
template <int D, int NT>
struct PagedConsumer {
  using Sh = Shape<D, NT>;
  static constexpr int MT = NT == 4 ? 2 : 1;  // m-blocks
  static constexpr int KS = D / 16;           // MMA steps of a score
  uint32_t qa[MT][KS][NT == 1 ? 2 : 4];
  float o[MT][2][4];     // dims 8j + 2t, +1 of this warp's 16 for rows c, c + 8 of m-block m
  float ref[NT], l[NT];  // l: this lane's rows only
  int lim[NT];           // last cache row that the query row sees, -1: none
  int c, t, warp, lane;
  int parity;            // of the weights' double buffer

  uint32_t p_smem;       // weights [2][kPRows][kPStride]
  float* wmax;           // [2][NT * 8][8] maxima of a tile by row and warp
  float* lsum;           // [NT * 8][8]
  float* osum;           // D = 64: the second half's outputs [NT * 8][D + 8]
  ConsumerSync* sync;

  __device__ __forceinline__ void load_q(const uint8_t* qs) {
    const uint32_t base = smem_u32(qs);
    const int i = lane >> 3, r = lane & 7;
    if (NT == 1) {
#pragma unroll
      for (int k = 0; k < KS; k += 2) {
        uint32_t x[4];  // rows 0..7, four 8-dim chunks
        ldmatrix4(x, base + r * Sh::kQStride + (2 * k + i) * 16);
        qa[0][k][0] = x[0];
        qa[0][k][1] = x[1];
        qa[0][k + 1][0] = x[2];
        qa[0][k + 1][1] = x[3];
      }
    } else {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t x[4];
          ldmatrix4(x, base + (16 * m + r + 8 * (i & 1)) * Sh::kQStride + (2 * k + (i >> 1)) * 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) qa[m][k][NT == 1 ? 0 : e] = x[e];
        }
    }
  }
  __device__ __forceinline__ void start(const PagedParams& p, const TileMeta& mt) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int r = 8 * i + c, tok = r / p.g;
      ref[i] = kMInit;
      l[i] = 0.f;
      lim[i] = r < p.R && tok < mt.n ? mt.pos + tok : -1;
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[m][j][e] = 0.f;
  }
  // Group i's rows of an accumulator: elements 2 (i % 2), +1 of m-block i / 2.
  __device__ __forceinline__ void rescale(int i, float alpha) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (NT == 1) {
          o[0][j][e] *= alpha;
          o[0][j][2 + e] *= alpha;
        } else {
          o[i >> 1][j][2 * (i & 1) + e] *= alpha;
        }
      }
    l[i] *= alpha;
  }
  // Byte offset in a tile of row 16 * slice (its first 64 dims).
  __device__ __forceinline__ static int slice_at(int slice, int lp) {
    const int row = slice * 16, pg = row >> lp;
    return ((pg << lp) * D * 2) + (row & ((1 << lp) - 1)) * 128;
  }
  // Four weights of row group i (keys 2t, 2t+1, 8+2t, 9+2t of this warp's 16)
  // and their sum.
  __device__ __forceinline__ float weights(int i, const float (&x)[4]) {
    float w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = ex2(x[e] - ref[i]);
    const uint32_t at = p_smem + parity * Sh::kP + (8 * i + c) * kPStride + (16 * warp + 2 * t) * 2;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t hi = pack_bf16x2(w[2 * j], w[2 * j + 1]);
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 16 * j), "r"(hi) : "memory");
      if (NT <= 2) {
        const uint32_t rest = pack_bf16x2(w[2 * j] - bf16lo(hi), w[2 * j + 1] - bf16hi(hi));
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 8 * NT * kPStride + 16 * j), "r"(rest)
                     : "memory");
      }
    }
    return (w[0] + w[1]) + (w[2] + w[3]);
  }

  // One tile.  ks: its keys; the values lie behind them.
  __device__ __forceinline__ void tile(const uint8_t* ks, const PagedParams& p,
                                       const TileMeta& mt) {
    const bool starts = (mt.flags & kStarts) != 0;
    // every row of the tile is there and seen by every query row in use
    const bool full = mt.row0 + kTile - 1 <= mt.pos && (mt.flags & kSlicesMask) == kSlicesMask;
    const int lp = p.lp;
    float s[MT][2][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[m][j][e] = 0.f;
    {
      const int i = lane >> 3, r = lane & 7;
      const uint32_t at = smem_u32(ks) + slice_at(warp, lp) + (8 * (i >> 1) + r) * 128;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t b[4];
        const int ch = 2 * k + (i & 1);
        ldmatrix4(b, at + (ch >> 3 ? 128 << lp : 0) + (((ch & 7) ^ r) << 4));
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          uint32_t a[4];
          if (NT == 1) {
            a[0] = qa[m][k][0];
            a[2] = qa[m][k][1];
            a[1] = a[3] = 0u;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = qa[m][k][NT == 1 ? 0 : e];
          }
          mma_bf16(s[m][0], a, b[0], b[1]);
          mma_bf16(s[m][1], a, b[2], b[3]);
        }
      }
    }
    float x[NT][4], sum[NT];
    const int buf = parity * NT * 64;
    const bool mine = (mt.flags >> warp) & 1;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float sc = s[i >> 1][e >> 1][2 * (i & 1) + (e & 1)] * p.qscale;
        const int row = mt.row0 + 16 * warp + 8 * (e >> 1) + 2 * t + (e & 1);
        x[i][e] = full || (mine && row <= lim[i]) ? sc : -INFINITY;
      }
      float mx = fmaxf(fmaxf(x[i][0], x[i][1]), fmaxf(x[i][2], x[i][3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if (t == 0) wmax[buf + (8 * i + c) * 8 + warp] = mx;
      sum[i] = starts ? 0.f : weights(i, x[i]);
    }
    (*sync)(lane);
    float top[NT];
    bool far = starts, grow = false;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const float4 u = *reinterpret_cast<const float4*>(wmax + buf + (8 * i + c) * 8);
      const float4 v = *reinterpret_cast<const float4*>(wmax + buf + (8 * i + c) * 8 + 4);
      top[i] = fmaxf(fmax3(u.x, u.y, u.z), fmax3(u.w, v.x, fmax3(v.y, v.z, v.w)));
      far = far || top[i] > ref[i] + kFar;
      grow = grow || top[i] > ref[i] + kTau;
    }
    // every warp sees the same maxima, so all of them decide alike
    far = __any_sync(0xffffffffu, far);
    if (far) {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if (top[i] > ref[i] + kTau) {
          rescale(i, ex2(ref[i] - top[i]));
          ref[i] = top[i];
        }
        sum[i] = weights(i, x[i]);
      }
      grow = false;
      (*sync)(lane);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) l[i] += sum[i];
    if (full) values<true>(ks + Sh::kOp, p, mt);
    else values<false>(ks + Sh::kOp, p, mt);
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
        if (top[i] > ref[i] + kTau) {
          rescale(i, ex2(ref[i] - top[i]));
          ref[i] = top[i];
        }
    }
    parity ^= 1;
  }

  // The A operand of the second product for m-block m, part `rest`, slice s.
  __device__ __forceinline__ void load_p(uint32_t (&a)[4], int m, int rest, int s) const {
    const int i = lane >> 3, r = lane & 7;
    ldmatrix4(a, p_smem + parity * Sh::kP + (16 * m + 8 * NT * rest + r + 8 * (i & 1)) * kPStride +
                     (16 * s + 8 * (i >> 1)) * 2);
  }
  // o += P V for this warp's 16 dims.
  template <bool FULL>
  __device__ __forceinline__ void values(const uint8_t* vs, const PagedParams& p,
                                         const TileMeta& mt) {
    constexpr int kGroups = D / 16;                // warps side by side
    constexpr int kSteps = kSlices / Sh::kHalves;  // slices of a warp
    const int dims = warp % kGroups, s0 = (warp / kGroups) * kSteps;
    const int i = lane >> 3, r = lane & 7;
    const int ch = 2 * dims + (i >> 1);
    const uint32_t at = smem_u32(vs) + (ch >> 3 ? 128 << p.lp : 0) + (8 * (i & 1) + r) * 128 +
                        (((ch & 7) ^ r) << 4);
    const int seen = mt.pos + mt.n - mt.row0;  // rows of the tile that a token may see
#pragma unroll(FULL ? kSteps : 1)
    for (int k = 0; k < kSteps; ++k) {
      const int s = s0 + k;
      if (!FULL && !((mt.flags >> s) & 1)) continue;  // nothing was loaded there
      uint32_t b[4];
      ldmatrix4_trans(b, at + slice_at(s, p.lp));
      if (!FULL) {
        // rows past the last token may be NaN: 0 * NaN would spread
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] &= keep(seen - (16 * s + 8 * (e & 1) + 2 * t));
        // and so may a drafted token's be, which earlier tokens do not see
        if (mt.n > 1 && 16 * s + 15 > mt.pos - mt.row0) {
          bool odd = false;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            odd = odd || (b[e] & 0x7f80u) == 0x7f80u || (b[e] & 0x7f800000u) == 0x7f800000u;
          if (__any_sync(0xffffffffu, odd)) {
            values_by_token(b, s, p, mt);
            continue;
          }
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint32_t a[4];
        load_p(a, m, 0, s);
        mma_bf16(o[m][0], a, b[0], b[1]);
        mma_bf16(o[m][1], a, b[2], b[3]);
        if (NT == 2) {
          load_p(a, m, 1, s);
          mma_bf16(o[m][0], a, b[0], b[1]);
          mma_bf16(o[m][1], a, b[2], b[3]);
        }
      }
    }
  }
  // Mask of a register with two rows of which the first n (or all) count.
  __device__ __forceinline__ static uint32_t keep(int n) {
    return n >= 2 ? 0xffffffffu : n == 1 ? 0x0000ffffu : 0u;
  }
  // The same for one slice with infinities or NaN among the values: token by
  // token, each with the rows that it sees, into its own rows of o only.
  __device__ __forceinline__ void values_by_token(const uint32_t (&b)[4], int s, const PagedParams& p,
                                               const TileMeta& mt) {
    for (int tok = 0; tok < mt.n; ++tok) {
      uint32_t seen[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        seen[e] = b[e] & keep(mt.pos + tok + 1 - mt.row0 - (16 * s + 8 * (e & 1) + 2 * t));
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float y[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) y[j][e] = 0.f;
#pragma unroll
        for (int rest = 0; rest < (NT == 2 ? 2 : 1); ++rest) {
          uint32_t a[4];
          load_p(a, m, rest, s);
          mma_bf16(y[0], a, seen[0], seen[1]);
          mma_bf16(y[1], a, seen[2], seen[3]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = NT == 1 ? c : 16 * m + 8 * (e >> 1) + c;
            if (r / p.g == tok) o[m][j][e] += y[j][e];
          }
      }
    }
  }

  // The piece's sums over all lanes and warps; for D = 64 also the outputs of
  // both halves, in the first four warps.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      float sum = l[i];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (t == 0) lsum[(8 * i + c) * 8 + warp] = sum;
    }
    if (NT == 1) {  // the weights' two parts
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) o[0][j][e] += o[0][j][2 + e];
    }
    if (Sh::kHalves > 1 && warp >= kWarps / 2) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          *reinterpret_cast<float2*>(osum + (8 * i + c) * (D + 8) + 16 * (warp - kWarps / 2) +
                                     8 * j + 2 * t) =
              make_float2(o[i >> 1][j][2 * (i & 1)], o[i >> 1][j][2 * (i & 1) + 1]);
    }
    (*sync)(lane);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const float4 u = *reinterpret_cast<const float4*>(lsum + (8 * i + c) * 8);
      const float4 v = *reinterpret_cast<const float4*>(lsum + (8 * i + c) * 8 + 4);
      l[i] = ((u.x + u.y) + (u.z + u.w)) + ((v.x + v.y) + (v.z + v.w));
    }
    if (Sh::kHalves > 1 && warp < kWarps / 2) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 y = *reinterpret_cast<const float2*>(osum + (8 * i + c) * (D + 8) +
                                                            16 * warp + 8 * j + 2 * t);
          o[i >> 1][j][2 * (i & 1)] += y.x;
          o[i >> 1][j][2 * (i & 1) + 1] += y.y;
        }
    }
  }
  __device__ __forceinline__ bool holds_output() const {
    return Sh::kHalves == 1 || warp < kWarps / 2;
  }
  // f(row, first of two dims, values) for this lane's outputs.
  template <typename F>
  __device__ __forceinline__ void each_output(F f) const {
    if (!holds_output()) return;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        f(i, 8 * i + c, 16 * warp + 8 * j + 2 * t,
          make_float2(o[i >> 1][j][2 * (i & 1)], o[i >> 1][j][2 * (i & 1) + 1]));
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
  for (int i = tid; i < p.S * p.Hq * D / 8; i += kThreads) row[i] = make_uint4(v, v, v, v);
}

// Where part r of a segment lies: a CTA holds at most one segment's first part
// and at most one later part.
__device__ __forceinline__ int part_slot(int c0, int r) { return 2 * (c0 + r) + (r == 0); }
__device__ __forceinline__ bool slot_ok(const PagedParams& p, int slot) {
  return range_ok(slot >= 0 && slot < 2 * kPagedMaxGrid, p.status);
}

// Merge the parts of a split segment, in CTA order, eight in one round trip.
template <int D>
__device__ __forceinline__ void merge_parts(const PagedParams& p, const TileMeta& mt, int tid) {
  const int R = p.R;
  const int parts = slot_ok(p, part_slot(mt.c0, mt.parts - 1)) ? mt.parts : 0;
  for (int col = tid; col < R * (D / 4); col += kConsumers) {
    const int r = col / (D / 4), d = (col % (D / 4)) * 4;
    float M = kMInit, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < parts; k0 += 8) {
      float2 ml[8];
      float4 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        ml[k] = make_float2(kMInit, 0.f);
        x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + k < parts) {
          const size_t slot = part_slot(mt.c0, k0 + k);
          ml[k] = __ldcg(reinterpret_cast<const float2*>(p.part_ml + (slot * R + r) * 2));
          x[k] = __ldcg(reinterpret_cast<const float4*>(p.part_o + (slot * R + r) * D + d));
        }
      }
      float top = M;
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, ml[k].x);
      const float a = ex2(M - top);
      M = top;
      l *= a;
      o = make_float4(o.x * a, o.y * a, o.z * a, o.w * a);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float e = ex2(ml[k].x - M);
        l = fmaf(ml[k].y, e, l);
        o.x = fmaf(x[k].x, e, o.x);
        o.y = fmaf(x[k].y, e, o.y);
        o.z = fmaf(x[k].z, e, o.z);
        o.w = fmaf(x[k].w, e, o.w);
      }
    }
    store4<D>(p, mt.b, mt.kvh, r, d, o, l, r / p.g >= mt.n);
  }
}

// A table entry that is in use; -1 where it names no page.
__device__ __forceinline__ int page_ok(const PagedParams& p, int page) {
  if (page >= 0 && page < p.P) return page;
  set_status(p.status, ATTN_DEV_BAD_PAGE);
  return -1;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const PagedParams p) {
  using Sh = Shape<D, NT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int NS = p.stages, B = p.B, Hkv = p.Hkv;
  uint8_t* stages = smem;
  uint8_t* qbuf = stages + (size_t)NS * Sh::kStage;            // [NS][NT * 8] query rows
  TileMeta* meta = reinterpret_cast<TileMeta*>(qbuf + NS * Sh::kQ);
  uint8_t* weights = reinterpret_cast<uint8_t*>(meta + NS);
  float* osum = reinterpret_cast<float*>(weights + 2 * Sh::kP);
  float* wmax = osum + Sh::kO / 4;
  float* lsum = wmax + 2 * NT * 64;
  uint64_t* bars = reinterpret_cast<uint64_t*>(lsum + NT * 64);  // full [NS], empty [NS], sync
  int* misc = reinterpret_cast<int*>(bars + 2 * NS + 1);  // [0] abort, [1] last to arrive, [8..16) scan
  int* prefix = misc + 16;                                // [B + 1]
  int* spos = prefix + B + 1;                             // [B]
  uint8_t* snew = reinterpret_cast<uint8_t*>(spos + B);   // [B]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = misc;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(&bars[s]), 1);
      mbar_init(smem_u32(&bars[NS + s]), kWarps);
    }
    mbar_init(smem_u32(&bars[2 * NS]), kWarps);
    misc[0] = 0;
    fence_mbar_init();
  }
  for (int i = tid; i < NS * Sh::kQ / 16; i += kThreads)  // rows past R stay zero
    reinterpret_cast<uint4*>(qbuf)[i] = make_uint4(0u, 0u, 0u, 0u);
  grid_dependency_wait();
  grid_dependents_launch();

  // ---- units per sequence and KV head, their exclusive prefix sum (every CTA)
  int carry = 0;
  for (int base = 0; base < B; base += kConsumers) {
    const int b = base + tid;
    int v = 0;
    if (tid < kConsumers && b < B) {
      int pos, n;
      const int kind = sequence(p, b, pos, n);
      spos[b] = pos;
      snew[b] = (uint8_t)n;
      if (kind == 2) v = (pos + n - 1) / kTile + 1 + kE;
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
  // (the zeros written above come before the query copies that land over them)
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();

  for (int b = blockIdx.x; b < B; b += gridDim.x)
    if (prefix[b + 1] == prefix[b]) fill_rows<D>(p, b, tid);  // it takes no part

  const long long T = (long long)Hkv * carry;  // all units
  const long long nseg = (long long)B * Hkv;
  long long gw = min((long long)gridDim.x, T);
  if (T <= (long long)(kWholeTiles + kE) * nseg) gw = min(gw, nseg);
  const int G = (int)gw;
  if ((int)blockIdx.x >= G) return;
  FlatRange rg;
  flat_range<kE>(rg, T, blockIdx.x, G, prefix, B, Hkv);
  if (rg.t0 >= rg.t1) return;
  FlatWalk w;
  flat_start<kE>(w, rg, prefix, spos, B, Hkv);
  if (w.u >= w.end) return;  // end units alone

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer --
    // Tiles go in batches of four, lane 8*ti + slice looks after slice
    // `slice` of the batch's tile ti; a batch's table entries are loaded while
    // the one before it is issued.
    const int ti = lane >> 3, slice = lane & 7;
    const int page_rows = 1 << p.lp, in_page = (slice * 16) & (page_rows - 1);
    auto fetch = [&](const FlatWalk& w) -> int {  // -1: no rows there
      const int row = w.k * kTile + slice * 16;
      if (w.u >= w.end || row > w.pos + snew[w.b] - 1) return -1;
      if (!range_ok((row >> p.lp) < p.M, p.status)) return -1;
      return page_ok(p, p.table[(size_t)w.b * p.M + (row >> p.lp)]);
    };
    auto step = [&](FlatWalk& w, int n) {  // n tiles on, as far as the range goes
      if (w.k + n < w.nt && w.u + n < w.end) {
        w.k += n;
        w.u += n;
        return;
      }
      for (int k = 0; k < n && w.u < w.end; ++k) flat_next<kE>(w, rg, prefix, spos, B, Hkv);
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
      m.row0 = w.k * kTile;
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
    step(w, ti);
    FlatWalk cur = w;
    int page = fetch(w);
    bool ok = true;
    while (ok) {
      const bool on = cur.u < cur.end;
      const int n_q = __popc(__ballot_sync(0xffffffffu, on)) >> 3;  // tiles of the batch
      if (n_q == 0) break;
      step(w, 4);
      const int next_page = fetch(w);
      TileMeta mt;
      if (on && slice == 0) describe(cur, mt);
      const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
      const bool lead = page >= 0 && in_page == 0;
      const uint32_t boxes = __ballot_sync(0xffffffffu, lead);
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
        uint32_t first = 0;
        int b = 0, kvh = 0;
        if (lane == 8 * q) {
          mt.flags |= (there >> (8 * q)) & 0xffu;
          meta[s] = mt;
          first = (mt.flags & kStarts) != 0;
          b = mt.b;
          kvh = mt.kvh;
          if (!skip)
            mbar_arrive_expect_tx(full, __popc((boxes >> (8 * q)) & 0xffu) *
                                                ((uint32_t)page_rows * D * 4u) +
                                            (first ? (uint32_t)p.R * D * 2u : 0u));
        }
        __syncwarp();
        first = __shfl_sync(0xffffffffu, first, 8 * q);
        const bool hold = __shfl_sync(0xffffffffu, skip, 8 * q);
        if (ti == q && lead && !hold) {
          const uint32_t dst =
              smem_u32(stages + (size_t)s * Sh::kStage) + slice * 16 * D * 2;
          tma_load_5d(dst, &tm_k, 0, 0, 0, cur.kvh, page, full);
          tma_load_5d(dst + Sh::kOp, &tm_v, 0, 0, 0, cur.kvh, page, full);
        }
        if (first && !hold) {  // the piece's query rows, one by each lane
          b = __shfl_sync(0xffffffffu, b, 8 * q);
          kvh = __shfl_sync(0xffffffffu, kvh, 8 * q);
          if (lane < p.R)
            bulk_load(smem_u32(qbuf + s * Sh::kQ) + lane * Sh::kQStride,
                      p.q + query_row(p, b, kvh, lane) * D, D * 2, full);
        }
        if (++s == NS) {
          s = 0;
          ++pass;
        }
      }
      cur = w;
      page = next_page;
    }
  } else {
    // ----------------------------------------------------------- consumers --
    ConsumerSync csync{smem_u32(&bars[2 * NS]), abort_flag, p.status, 0u};
    PagedConsumer<D, NT> cs;
    cs.c = lane >> 2;
    cs.t = lane & 3;
    cs.warp = warp;
    cs.lane = lane;
    cs.parity = 0;
    cs.p_smem = smem_u32(weights);
    cs.wmax = wmax;
    cs.lsum = lsum;
    cs.osum = osum;
    cs.sync = &csync;
    int s = 0;
    uint32_t ph = 0;
    for (;;) {
      if (!consumer_wait(smem_u32(&bars[s]), ph, abort_flag, p.status, lane)) break;
      const TileMeta mt = meta[s];
      if (mt.flags & kStarts) {
        cs.load_q(qbuf + s * Sh::kQ);
        cs.start(p, mt);
      }
      cs.tile(stages + (size_t)s * Sh::kStage, p, mt);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars[NS + s]));
      if (++s == NS) {
        s = 0;
        ph ^= 1u;
      }
      if (mt.flags & kEnds) {
        cs.finish();
        if (*abort_flag) break;
        if (mt.parts == 1) {
          cs.each_output([&](int i, int r, int d, float2 y) {
            if (r >= p.R) return;
            const bool idle = r / p.g >= mt.n;
            const float inv = idle || cs.l[i] == 0.f ? 0.f : 1.f / cs.l[i];
            const size_t at = query_row(p, mt.b, mt.kvh, r) * D + d;
            if (range_ok(at + 2 <= (size_t)p.B * p.S * p.Hq * D, p.status))
              *reinterpret_cast<uint32_t*>(p.out + at) =
                  idle ? 0u : pack_bf16x2(y.x * inv, y.y * inv);
          });
        } else {
          const int slot = part_slot(mt.c0, (int)blockIdx.x - mt.c0);
          if (slot_ok(p, slot)) {
            cs.each_output([&](int i, int r, int d, float2 y) {
              if (r >= p.R) return;
              *reinterpret_cast<float2*>(p.part_o + ((size_t)slot * p.R + r) * D + d) = y;
              if (d == 0)
                *reinterpret_cast<float2*>(p.part_ml + ((size_t)slot * p.R + r) * 2) =
                    make_float2(cs.ref[i], cs.l[i]);
            });
          }
          csync(lane);
          if (tid == 0) {
            uint32_t* counter = p.counters + mt.b * Hkv + mt.kvh;
            __threadfence();  // (the other threads' stores came before the barrier)
            const bool last = atomicAdd(counter, 1u) + 1 == (uint32_t)mt.parts;
            if (last) *counter = 0;
            __threadfence();
            misc[1] = last;
          }
          csync(lane);
          if (misc[1] && !*abort_flag) merge_parts<D>(p, mt, tid);
        }
      }
      if (mt.flags & kLast) break;
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
  return (size_t)stages * (Sh::kStage + Sh::kQ + sizeof(TileMeta) + 16) + Sh::kFixed + 8 + 64 +
         (size_t)9 * B + 16;
}

// Per device, found once: its SMs and how many clusters of each size can run
// at once with one CTA to an SM (a cluster stays within one GPC).
struct PagedDevice {
  int sms;
  int clusters[kMaxCluster + 1];
};

template <int D, int NT>
cudaError_t set_attributes() {
  cudaError_t e = cudaFuncSetAttribute(
      paged_decode_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(paged_cluster_kernel<D, NT>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(paged_cluster_kernel<D, NT>,
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e;
}

template <int D>
cudaError_t find_device(PagedDevice& d, int dev) {
  cudaError_t e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = set_attributes<D, 1>();
  if (e == cudaSuccess) e = set_attributes<D, 2>();
  if (e == cudaSuccess) e = set_attributes<D, 4>();
  if (e != cudaSuccess) return e;
  for (int c = 1; c <= kMaxCluster; ++c) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c * 64);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kMaxSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&d.clusters[c], paged_cluster_kernel<D, 1>, &cfg) !=
        cudaSuccess) {
      cudaGetLastError();
      d.clusters[c] = 0;
    }
  }
  return cudaSuccess;
}

template <int D>
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
      e = find_device<D>(known[dev], dev);
      if (e != cudaSuccess) return e;
      ready[dev].store(true, std::memory_order_release);
    }
  }
  *out = &known[dev];
  return cudaSuccess;
}

// CTAs per segment in cluster mode, or 0 for the split over a flat list.  The
// cluster would be the largest that lets every segment have its own resident at
// once; it is taken where its estimate is lower (us).  The host knows only what
// the table can hold: a position is taken to lie half-way on average, and the
// longest of several, which a cluster waits for, at the end.
template <int D>
int cluster_size(const PagedParams& p, const PagedDevice& d) {
  if (g_decode_test_cluster >= 0)  // schedule tests only
    return min(g_decode_test_cluster, kMaxCluster);
  const long long nseg = (long long)p.B * p.Hkv;
  const int tiles = (p.cap + kTile - 1) / kTile;
  int c = min(kMaxCluster, tiles);
  while (c > 1 && nseg > d.clusters[c]) --c;
  const float mean = 0.5f * (float)tiles;
  const float longest = p.B == 1 ? mean : (float)tiles;
  const float waves = c > 1 ? 1.f : (float)((nseg + d.sms - 1) / d.sms);
  const float per_tile = D == 128 ? 1.4f : 0.8f;
  const float clusters = waves * (4.f + per_tile * ceilf(longest / (float)c));
  const float flat = 9.f + per_tile * (float)nseg * mean / (float)d.sms;
  return clusters <= flat ? c : 0;
}

template <int D, int NT>
cudaError_t launch_paged(PagedParams& p, const CUtensorMap& mk, const CUtensorMap& mv,
                         cudaStream_t stream) {
  const PagedDevice* d = nullptr;
  cudaError_t e = paged_device<D>(&d);
  if (e != cudaSuccess) return e;
  p.stages = kMaxStages;
  const int C = cluster_size<D>(p, *d);
  if (C > 0) {
    if (d->clusters[C] == 0) return cudaErrorNotSupported;
    while (p.stages > 2 && cluster_smem_bytes<D, NT>(p.stages, p.R, C) > (size_t)kMaxSmem)
      --p.stages;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.B * p.Hkv * C));
    cfg.blockDim = dim3(kThreads);
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
    e = cudaLaunchKernelEx(&cfg, paged_cluster_kernel<D, NT>, mk, mv, p);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  while (p.stages > 2 && flat_smem_bytes<D, NT>(p.stages, p.B) > (size_t)kMaxSmem) --p.stages;
  return launch_pdl(paged_decode_kernel<D, NT>, dim3(min(kPagedMaxGrid, d->sms)), dim3(kThreads),
                    flat_smem_bytes<D, NT>(p.stages, p.B), stream, mk, mv, p);
}

template <int D>
cudaError_t launch_paged_rows(PagedParams& p, const CUtensorMap& mk, const CUtensorMap& mv,
                              cudaStream_t stream) {
  return p.R <= 8    ? launch_paged<D, 1>(p, mk, mv, stream)
         : p.R <= 16 ? launch_paged<D, 2>(p, mk, mv, stream)
                     : launch_paged<D, 4>(p, mk, mv, stream);
}

}  // namespace
}  // namespace gqa
