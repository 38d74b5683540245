// block_select.cu -- which blocks of a cache a decode step attends.
//
// Scores.  Block j of a KV head has, per channel d, the largest and smallest
// key value max_jd and min_jd, so no key of the block, as it was appended,
// scores above sum_d max(q_d max_jd, q_d min_jd) with query q (its code may, by
// the code's rounding: the scores rank blocks).  Summed over the g query
// heads of the KV head (q+ = max(q, 0), q- = min(q, 0)):
//   s_j = sum_d (sum_h q+_hd) max_jd + (sum_h q-_hd) min_jd,
// one vector of 256 against the block's 512 bytes of bounds.  Bound by
// memory: the bounds are read once.
//
// Selection.  Of the blocks 0..last a position has (last = pos / block): all
// of them if there are no more than `count`; else the first `first`, the
// `recent` last ones, and of the others the best-scored, ties to the lowest
// index.  A row that fits the block's registers (8192 scores) has its range cut
// into 4095 equal parts: a histogram in shared memory over them and a scan give
// the part that the need-th largest lies in, and its few scores are ranked
// among themselves.  Longer rows, and rows of another shape (infinities,
// outliers, hundreds alike), go by order-preserving integer keys, digit by digit
// from the top (12, 12 and 8 bits, a histogram and a scan each, scores read
// again in every pass where they do not fit).  The first digit holds sign,
// exponent and three bits of the mantissa.  Each thread holds items in a row, so
// one scan over the threads' counts places the chosen indices in ascending
// order.  Bound by its instructions (512 rows of up to 8192 scores: 36 us with
// one bit a round, 20 with three digits, 15 with one digit and up to 256 keys
// ranked, 10.6 with equal parts and four blocks to an SM; the 32 registers that
// leaves a thread of the 8192 form spill 88 bytes).  A longer row, and one of
// 8190 or 8191 scores that does not start on 16 bytes, is one CTA's with up to
// four reads: 512 rows of 8192 11.4 us, of 8190 18.5, of 16384 28, of 65536 100.
#include "common.cuh"
#include "decode_params.h"
#include "internal.h"

namespace gqa {
namespace {

__device__ unsigned int g_block_skips;  // debug builds: accesses a range check skipped

constexpr int kScoreWarps = 4;  // (8: 26.6 us for 142 MB, 4: 23.7)
constexpr int kScoreThreads = kScoreWarps * 32;
constexpr int kScoreBlocksPerWarp = 16;
constexpr int kScoreBlocksPerCta = kScoreWarps * kScoreBlocksPerWarp;

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A warp scores 16 blocks: their bounds are the 16 rows of MMA operand A,
// loaded from memory in the operand's own layout (lane 4c + t takes 16-byte
// pieces 4i + t of rows c and c + 8; the order of the 256 products is free),
// and the vector is operand B as three bf16 columns (value, remainder,
// remainder of that: 24 bits), so every product is exact and nothing is
// unpacked.  (With fp32 multiply-adds on unpacked values the kernel was bound
// by its instructions: 30.5 against 24 us for 142 MB.)
__global__ void __launch_bounds__(kScoreThreads) block_scores_kernel(
    const uint16_t* __restrict__ q, const int32_t* __restrict__ positions,
    const uint4* __restrict__ bounds, float* __restrict__ scores, int Hkv, int g, int L,
    int block, int nb) {
  __shared__ __align__(16) uint16_t parts[3][2 * kDecodeD];
  grid_dependency_wait();
  grid_dependents_launch();
  const int seg = blockIdx.x, b = seg / Hkv, tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31, c = lane >> 2, t = lane & 3;
  const int pos = positions[b];
  const int n = rows_in_cache(pos, 0, L) ? pos / block + 1 : 0;
  const int j0 = blockIdx.y * kScoreBlocksPerCta + warp * kScoreBlocksPerWarp;
  const int cta0 = blockIdx.y * kScoreBlocksPerCta;
  float* out = scores + (size_t)seg * nb;
  if (!range_ok_count(n <= nb, &g_block_skips)) return;  // so j < n is inside bounds and scores
  if (cta0 >= n) {  // nothing here up to the position
    for (int j = cta0 + tid; j < min(nb, cta0 + kScoreBlocksPerCta); j += kScoreThreads)
      out[j] = -INFINITY;
    return;
  }
  uint4 ua[8], ub[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint4* row = bounds + ((size_t)seg * nb + j0) * 32 + 4 * i + t;
    ua[i] = j0 + c < n ? row[c * 32] : make_uint4(0u, 0u, 0u, 0u);
    ub[i] = j0 + c + 8 < n ? row[(c + 8) * 32] : make_uint4(0u, 0u, 0u, 0u);
  }
  // the vector: dims of q+ summed over the heads, then of q-
  for (int e = tid; e < 2 * kDecodeD; e += kScoreThreads) {
    const uint16_t* src = q + (size_t)seg * g * kDecodeD + (e & (kDecodeD - 1));
    float w = 0.f;
#pragma unroll 4
    for (int h = 0; h < g; ++h) {
      const float x = __uint_as_float((uint32_t)src[h * kDecodeD] << 16);
      w += e < kDecodeD ? fmaxf(x, 0.f) : fminf(x, 0.f);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint32_t r = pack_bf16x2(w, 0.f);
      parts[k][e] = (uint16_t)r;
      w -= bf16lo(r);
    }
  }
  __syncthreads();
  float d[2][4] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint4 v = c < 3 ? *reinterpret_cast<const uint4*>(&parts[c < 3 ? c : 0][8 * (4 * i + t)])
                          : make_uint4(0u, 0u, 0u, 0u);
    mma_bf16(d[0], ua[i].x, ub[i].x, ua[i].y, ub[i].y, v.x, v.y);
    mma_bf16(d[1], ua[i].z, ub[i].z, ua[i].w, ub[i].w, v.z, v.w);
  }
  // columns 0 and 1 are in the lanes t = 0, column 2 in t = 1
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float c0 = d[0][2 * r] + d[1][2 * r], c1 = d[0][2 * r + 1] + d[1][2 * r + 1];
    const float s = c0 + (c1 + __shfl_down_sync(0xffffffffu, c0, 1));
    const int j = j0 + c + 8 * r;
    if (t == 0 && j < nb) out[j] = j < n ? s : -INFINITY;
  }
}

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 4096;
constexpr int kListed = 256;  // a bin of keys this small is ranked directly
constexpr int kFew = 64;      // a part of the scores' range this small is
static_assert(kSelectThreads == 2 * kListed, "two threads to a listed key");

// Order-preserving key of a score: larger score, larger key, never 0; -0 is
// +0, NaN is taken as -inf (fmaxf drops it).
__device__ __forceinline__ uint32_t score_key(float x) {
  const uint32_t u = __float_as_uint(fmaxf(x, -INFINITY) + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_score(uint32_t k) {
  return __uint_as_float(k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}

// Exclusive prefix sum of v over the block's threads; *all = the total.  One
// barrier; calls in a row use the two sets of `slots` in turn.
__device__ __forceinline__ int block_scan(int v, uint32_t (*slots)[32], int& phase, int* all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) slots[phase][warp] = x;
  __syncthreads();
  const uint32_t w = lane < kSelectWarps ? slots[phase][lane] : 0u;
  phase ^= 1;
  *all = (int)__reduce_add_sync(0xffffffffu, w);
  return (int)__reduce_add_sync(0xffffffffu, lane < warp ? w : 0u) + x - v;
}

// Thread t holds I items in a row of each chunk of I * kSelectThreads; LOOP:
// more than one chunk, whose scores are read again in every pass; else the
// keys stay in registers.
template <int I, bool LOOP>
__global__ void __launch_bounds__(kSelectThreads, I == 16 && !LOOP ? 4 : 3) block_select_kernel(
    const float* __restrict__ scores, const int32_t* __restrict__ positions, int32_t* out,
    int Hkv, int L, int block, int nb, int count, int first, int recent) {
  static_assert(I % 4 == 0, "scores come in fours");
  constexpr int kChunk = I * kSelectThreads;
  __shared__ __align__(16) int hist[kBins];
  __shared__ uint32_t slots[2][32];
  __shared__ int found[4];
  grid_dependency_wait();
  grid_dependents_launch();
  const int seg = blockIdx.x, b = seg / Hkv, tid = threadIdx.x;
  auto clear = [&]() {
    for (int i = tid; i < kBins / 4; i += kSelectThreads)
      reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
  };
  clear();
  const int pos = positions[b];
  const int n = rows_in_cache(pos, 0, L) ? pos / block + 1 : 0;
  int32_t* o = out + (size_t)seg * count;
  if (!range_ok_count(n <= nb, &g_block_skips)) return;  // so the items below hi are in the row
  if (n <= count) {
    for (int i = tid; i < count; i += kSelectThreads) o[i] = i < n ? i : -1;
    return;
  }
  const float* sc = scores + (size_t)seg * nb;
  const int need = count - first - recent;  // of the blocks lo .. hi-1
  const int lo = first, hi = n - recent;
  // items are shifted so that their groups of four start on 16 bytes
  const int shift4 = (int)((reinterpret_cast<uintptr_t>(sc) >> 2) & 3);
  const int j0 = tid * I - shift4;  // this thread's first item of chunk 0
  const int end = LOOP ? n + shift4 : 1;  // chunks: at 0, kChunk, .. below this
  uint32_t key[I];
  auto load = [&](int at) {  // the keys of the chunk at item `at`; 0 (below every key): no candidate
#pragma unroll
    for (int g = 0; g < I; g += 4) {
      const int j = at + j0 + g;
      if (j >= lo && j + 4 <= hi) {
        const float4 x = *reinterpret_cast<const float4*>(sc + j);
        key[g] = score_key(x.x);
        key[g + 1] = score_key(x.y);
        key[g + 2] = score_key(x.z);
        key[g + 3] = score_key(x.w);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          key[g + k] = j + k >= lo && j + k < hi ? score_key(sc[j + k]) : 0u;
      }
    }
  };
  int phase = 0;
  uint32_t th = 0, mask = 0;  // keys above every key with (key & mask) == th are chosen,
  int left = need;            // and `left` of those in that bin: the largest, the lowest indices
  bool whole = true;          // ... which are all of them
  bool listed = false;        // ... which are ranked in a list
  // In the histogram, the bin of the left-th largest: thread t holds 8 bins
  // from the top.
  auto find = [&]() {
    __syncthreads();
    constexpr int kPer = kBins / kSelectThreads;
    static_assert(kPer == 8, "two int4 per thread");
    int c[kPer], sum = 0, all;
    const int top = kBins - 1 - tid * kPer;
    *reinterpret_cast<int4*>(c) = *reinterpret_cast<const int4*>(&hist[top - 7]);
    *reinterpret_cast<int4*>(c + 4) = *reinterpret_cast<const int4*>(&hist[top - 3]);
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += c[i];
    int before = block_scan(sum, slots, phase, &all);
    if (before < left && before + sum >= left) {  // one thread
#pragma unroll
      for (int i = kPer - 1; i >= 0; --i) {
        if (before < left && before + c[i] >= left) {
          found[0] = top - 7 + i;
          found[1] = left - before;
          found[2] = c[i];
          found[3] = 0;  // the list's length
        }
        before += c[i];
      }
    }
    __syncthreads();
    whole = found[2] == found[1];
  };
  unsigned long long* list = reinterpret_cast<unsigned long long*>(hist);  // [kListed]
  // A score and its index as one number: a larger score first, then a lower index.
  auto entry = [&](uint32_t k, int j) { return ((unsigned long long)k << 32) | (uint32_t)~j; };
  bool done = need == 0;
  uint32_t sure = 0;  // bit i: item i is chosen (done)
  if (!LOOP && !done) {
    // One row in registers: its range in 4095 equal parts (part 0: no
    // candidate), which rise with the score; scores of any common shape spread
    // over them so well that the last part to be chosen from holds only few.
    float x[I];
    float low = INFINITY, high = -INFINITY;
    const bool some = j0 < hi && j0 + I > lo;  // (few threads of a short row have candidates)
#pragma unroll
    for (int g = 0; g < I; g += 4) {
      if (!some) break;
      const int j = j0 + g;
      if (j >= lo && j + 4 <= hi) {
        const float4 f = *reinterpret_cast<const float4*>(sc + j);
        x[g] = fmaxf(f.x, -INFINITY);  // NaN is taken as -inf
        x[g + 1] = fmaxf(f.y, -INFINITY);
        x[g + 2] = fmaxf(f.z, -INFINITY);
        x[g + 3] = fmaxf(f.w, -INFINITY);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          x[g + k] = j + k >= lo && j + k < hi ? fmaxf(sc[j + k], -INFINITY)
                                               : __uint_as_float(0x7fffffffu);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // (a NaN is passed over)
        low = fminf(low, x[g + k]);
        high = fmaxf(high, x[g + k]);
      }
    }
    uint32_t k_low = __reduce_min_sync(0xffffffffu, score_key(low));
    uint32_t k_high = __reduce_max_sync(0xffffffffu, score_key(high));
    const int lane = tid & 31;
    if (lane == 0) {
      slots[0][tid >> 5] = k_low;
      slots[1][tid >> 5] = k_high;
    }
    __syncthreads();  // and the histogram is clear
    k_low = __reduce_min_sync(0xffffffffu, slots[0][lane & (kSelectWarps - 1)]);
    k_high = __reduce_max_sync(0xffffffffu, slots[1][lane & (kSelectWarps - 1)]);
    low = key_score(k_low);
    const float span = key_score(k_high) - low;
    if (span > 1e-30f && span < 1e30f) {  // (neither infinities nor scores all alike)
      const float per_unit = (float)(kBins - 2) / span;
      uint32_t part[I / 2];
#pragma unroll
      for (int i = 0; i < I; ++i) {
        if (!some) break;
        const uint32_t d =
            x[i] == x[i] ? (uint32_t)min((int)((x[i] - low) * per_unit), kBins - 2) + 1u : 0u;
        if (d != 0u) atomicAdd(&hist[d], 1);
        if (i & 1) part[i >> 1] |= d << 16;
        else part[i >> 1] = d;
      }
      find();
      if (whole || found[2] <= kFew) {
        done = true;
        const uint32_t d = (uint32_t)found[0], from = whole ? d : d + 1;
        uint32_t mine = 0;  // the items in part d
#pragma unroll
        for (int i = 0; i < I; ++i) {
          if (!some) break;
          const uint32_t e = i & 1 ? part[i >> 1] >> 16 : part[i >> 1] & 0xffffu;
          if (e >= from) sure |= 1u << i;
          if (e == d) mine |= 1u << i;
        }
        if (!whole) {
          left = found[1];
          for (uint32_t r = mine; r; r &= r - 1u) {
            const int j = j0 + __ffs((int)r) - 1, k = atomicAdd(&found[3], 1);
            if (range_ok_count(k < kListed && j >= lo && j < hi, &g_block_skips))
              list[k] = entry(score_key(sc[j]), j);
          }
          __syncthreads();
          const int m = kDebugChecks ? min(found[3], kListed) : found[3];
          for (uint32_t r = mine; r; r &= r - 1u) {
            const int i = __ffs((int)r) - 1;
            const unsigned long long me = entry(score_key(sc[j0 + i]), j0 + i);
            int above = 0;
            for (int k = 0; k < m; ++k) above += list[k] > me;
            if (above < left) sure |= 1u << i;
          }
        }
      } else {
        clear();
      }
    }
  }
  if (!done) {
    if (!LOOP) load(0);
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 20 : pass == 1 ? 8 : 0;
      const uint32_t digits = pass == 2 ? 0xffu : 0xfffu;
      if (pass > 0) clear();
      __syncthreads();
      for (int at = 0; at < end; at += kChunk) {
        if (LOOP) load(at);
#pragma unroll
        for (int i = 0; i < I; ++i)
          if (key[i] != 0u && (key[i] & mask) == th) atomicAdd(&hist[(key[i] >> shift) & digits], 1);
      }
      find();
      th |= (uint32_t)found[0] << shift;
      mask |= digits << shift;
      left = found[1];
      listed = !LOOP && !whole && found[2] <= kListed;  // few: rank them among themselves
      if (whole || listed) break;
    }
  }
  const uint32_t bin_top = th | ~mask;  // the bin's largest possible key
  // The bin's entries, in any order, and each one's rank among them: chosen if
  // below `left`.  The list takes the histogram's place; a thread keeps its
  // item's place in it where the key was.
  int* rank_of = hist + 2 * kListed;  // [kListed]
  uint32_t in_list = 0;  // bit i: key[i] is a place
  if (listed) {
#pragma unroll
    for (int i = 0; i < I; ++i)
      if (key[i] >= th && key[i] <= bin_top) {
        const int k = atomicAdd(&found[3], 1);
        if (!range_ok_count(k < kListed, &g_block_skips)) continue;
        list[k] = entry(key[i], j0 + i);
        key[i] = (uint32_t)k;
        in_list |= 1u << i;
      }
    if (tid < kListed) rank_of[tid] = 0;
    __syncthreads();
    const int m = kDebugChecks ? min(found[3], kListed) : found[3];
    // two threads to a key, or four if that covers the list
    const int parts = m <= kSelectThreads / 4 ? 4 : 2;
    const int k = tid & (kSelectThreads / parts - 1), part = tid / (kSelectThreads / parts);
    if (k < m) {
      const unsigned long long me = list[k];
      int rank = 0;
#pragma unroll 4
      for (int x = part; x < m; x += parts) rank += list[x] > me;
      atomicAdd(&rank_of[k], rank);
    }
    __syncthreads();
  }
  // Place the chosen indices in ascending order: a count per thread, a scan.
  int base = 0, tie_base = 0;
  for (int at = 0; at < end; at += kChunk) {
    if (LOOP && !done) load(at);
    uint32_t take = sure;  // bit i: item i of this thread
    if (!done) {
      // keys that are chosen for sure: above the bin, or all of it too (th > 0)
      const uint32_t above = whole ? th - 1u : bin_top;
#pragma unroll
      for (int i = 0; i < I; ++i)
        if (key[i] > above) take |= 1u << i;
      if (listed) {
        take &= ~in_list;
#pragma unroll
        for (int i = 0; i < I; ++i)
          if ((in_list >> i) & 1u && rank_of[key[i]] < left) take |= 1u << i;
      } else if (!whole) {
        // the bin is one key alone (all three digits): its lowest indices
        uint32_t ties = 0;
#pragma unroll
        for (int i = 0; i < I; ++i)
          if (key[i] == th) ties |= 1u << i;
        int all;
        int room = left - tie_base - block_scan(__popc(ties), slots, phase, &all);
        tie_base += all;
        for (; ties && room > 0; --room) {
          take |= ties & (0u - ties);
          ties &= ties - 1u;
        }
      }
    }
    const int j = at + j0;
    if (j < lo || j + I > hi) {  // the first and the last blocks
#pragma unroll
      for (int i = 0; i < I; ++i)
        if ((j + i >= 0 && j + i < lo) || (j + i >= hi && j + i < n)) take |= 1u << i;
    }
    int all;
    int32_t* to = o + base + block_scan(__popc(take), slots, phase, &all);
    base += all;
    for (; take; take &= take - 1u, ++to)
      if (range_ok_count(to - o < count, &g_block_skips)) *to = j + __ffs((int)take) - 1;
  }
}

}  // namespace

cudaError_t block_read_skips(uint32_t* count) { return read_and_clear(g_block_skips, count); }

cudaError_t launch_block_scores(const void* q, const int32_t* positions, const void* k_bounds,
                                int B, int Hq, int Hkv, int L, int block, float* scores,
                                cudaStream_t stream) {
  const int nb = (L + block - 1) / block;
  const int ctas = (nb + kScoreBlocksPerCta - 1) / kScoreBlocksPerCta;
  return launch_pdl(block_scores_kernel, dim3(B * Hkv, ctas), dim3(kScoreThreads), 0, stream,
                    static_cast<const uint16_t*>(q), positions, static_cast<const uint4*>(k_bounds),
                    scores, Hkv, Hq / Hkv, L, block, nb);
}

cudaError_t launch_block_select(const float* scores, const int32_t* positions, int B, int Hkv,
                                int L, int block, int count, int first, int recent, int32_t* out,
                                cudaStream_t stream) {
  const int nb = (L + block - 1) / block;
  // rows that do not all start on 16 bytes shift their items by up to three
  const int shifts = nb % 4 != 0 || (reinterpret_cast<uintptr_t>(scores) & 15u) != 0 ? 3 : 0;
  const int per = (nb + shifts + kSelectThreads - 1) / kSelectThreads;
  auto kernel = per <= 4    ? block_select_kernel<4, false>
                : per <= 16 ? block_select_kernel<16, false>
                            : block_select_kernel<16, true>;
  return launch_pdl(kernel, dim3(B * Hkv), dim3(kSelectThreads), 0, stream, scores, positions,
                    out, Hkv, L, block, nb, count, first, recent);
}

}  // namespace gqa
