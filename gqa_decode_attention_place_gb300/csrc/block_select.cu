// block_select.cu -- which blocks of a cache a decode step attends.
//
// Scores.  Block j of a KV head has, per channel d, the largest and smallest
// key value max_jd and min_jd, so no key of the block scores above
// sum_d max(q_d max_jd, q_d min_jd) with query q.  Summed over the g query
// heads of the KV head (q+ = max(q, 0), q- = min(q, 0)):
//   s_j = sum_d (sum_h q+_hd) max_jd + (sum_h q-_hd) min_jd,
// one vector of 256 against the block's 512 bytes of bounds.  Bound by
// memory: the bounds are read once.
//
// Selection.  Of the blocks 0..last a position has (last = pos / block): all
// of them if there are no more than `count`; else the first `first`, the
// `recent` last ones, and of the others the best-scored, ties to the lowest
// index.  The threshold is the need-th largest score: found bit by bit from
// the top over order-preserving integer keys (32 block-wide counts, the keys
// in registers), then one block scan places the chosen indices in ascending
// order.
#include "common.cuh"
#include "internal.h"

namespace gqa {
namespace {

constexpr int kScoreWarps = 8;
constexpr int kScoreBlocksPerWarp = 8;
constexpr int kScoreBlocksPerCta = kScoreWarps * kScoreBlocksPerWarp;

__global__ void __launch_bounds__(kScoreWarps * 32) block_scores_kernel(
    const uint4* __restrict__ q, const int32_t* __restrict__ positions,
    const uint4* __restrict__ bounds, float* __restrict__ scores, int Hkv, int g, int L,
    int block, int nb) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int seg = blockIdx.x, b = seg / Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pos = positions[b];
  const int n = rows_in_cache(pos, 0, L) ? pos / block + 1 : 0;
  const int j0 = blockIdx.y * kScoreBlocksPerCta + warp * kScoreBlocksPerWarp;
  float w[8];  // lanes 0-15: sum of q+ for dims 8l.., lanes 16-31: sum of q-
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 0.f;
  if (j0 < n)
    for (int h = 0; h < g; ++h) {
      const uint4 u = q[((size_t)seg * g + h) * 16 + (lane & 15)];
      const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = bf16lo(x[i]), hi = bf16hi(x[i]);
        w[2 * i] += lane < 16 ? fmaxf(lo, 0.f) : fminf(lo, 0.f);
        w[2 * i + 1] += lane < 16 ? fmaxf(hi, 0.f) : fminf(hi, 0.f);
      }
    }
  // the bounds of the warp's 8 blocks, all in flight together
  uint4 u[kScoreBlocksPerWarp];
#pragma unroll
  for (int i = 0; i < kScoreBlocksPerWarp; ++i)
    u[i] = j0 + i < n ? bounds[((size_t)seg * nb + j0 + i) * 32 + lane] : make_uint4(0u, 0u, 0u, 0u);
  float s[kScoreBlocksPerWarp];
#pragma unroll
  for (int i = 0; i < kScoreBlocksPerWarp; ++i) {
    const uint32_t x[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
    s[i] = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      s[i] = fmaf(bf16lo(x[k]), w[2 * k], fmaf(bf16hi(x[k]), w[2 * k + 1], s[i]));
  }
  // 8 sums over 32 lanes: each of the first three exchanges halves the number
  // of sums a lane still carries, so 9 shuffles do the work of 40
#pragma unroll
  for (int half = 4; half > 0; half >>= 1) {
    const bool up = lane & (4 * half);
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float give = up ? s[i] : s[i + half], keep = up ? s[i + half] : s[i];
      s[i] = keep + __shfl_xor_sync(0xffffffffu, give, 4 * half);
    }
  }
  s[0] += __shfl_xor_sync(0xffffffffu, s[0], 2);
  s[0] += __shfl_xor_sync(0xffffffffu, s[0], 1);
  const int j = j0 + (lane >> 2);  // lanes 4i .. 4i+3 hold block i's sum
  if ((lane & 3) == 0 && j < nb) scores[(size_t)seg * nb + j] = j < n ? s[0] : -INFINITY;
}

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;

// Order-preserving key of a score: larger score, larger key; -0 = +0; NaN is
// taken as -inf.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) x = -INFINITY;
  x += 0.f;  // -0 -> +0
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum of v over the block; every thread gets it.  `slots` holds two sets of
// counters so that one barrier per call suffices.
__device__ __forceinline__ uint32_t block_sum(uint32_t v, uint32_t (*slots)[32], int phase) {
  v = __reduce_add_sync(0xffffffffu, v);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) slots[phase][warp] = v;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, lane < kSelectWarps ? slots[phase][lane] : 0u);
}
// Exclusive prefix sum of v over the block's threads.
__device__ __forceinline__ int block_scan(int v, uint32_t (*slots)[32], int phase) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) slots[phase][warp] = x;
  __syncthreads();
  const uint32_t w = lane < warp ? slots[phase][lane] : 0u;
  return (int)__reduce_add_sync(0xffffffffu, w) + x - v;
}

// I items per thread, thread t holding items t*I .. t*I + I-1 (I = 0: any
// number of items, read again from memory in every pass).
template <int I>
__global__ void __launch_bounds__(kSelectThreads) block_select_kernel(
    const float* __restrict__ scores, const int32_t* __restrict__ positions, int32_t* out,
    int Hkv, int L, int block, int nb, int count, int first, int recent) {
  __shared__ uint32_t slots[2][32];
  grid_dependency_wait();
  grid_dependents_launch();
  const int seg = blockIdx.x, b = seg / Hkv, tid = threadIdx.x;
  const int pos = positions[b];
  const int n = rows_in_cache(pos, 0, L) ? pos / block + 1 : 0;
  int32_t* o = out + (size_t)seg * count;
  if (n <= count) {
    for (int i = tid; i < count; i += kSelectThreads) o[i] = i < n ? i : -1;
    return;
  }
  const float* s = scores + (size_t)seg * nb;
  const int items = I > 0 ? I : (n + kSelectThreads - 1) / kSelectThreads;
  const long long i0 = (long long)tid * items;
  const int need = count - first - recent;  // of the blocks first .. n-recent-1
  uint32_t key[I > 0 ? I : 1];
  if (I > 0) {
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const long long j = i0 + i;
      key[i] = j >= first && j < n - recent ? score_key(s[j]) : 0u;  // 0: below every key
    }
  }
  auto get = [&](int i) -> uint32_t {
    if (I > 0) return key[i];
    const long long j = i0 + i;
    return j >= first && j < n - recent ? score_key(s[j]) : 0u;
  };
  int phase = 0;
  // the need-th largest key: the largest th with count(key >= th) >= need
  uint32_t th = 0;
  if (need > 0) {
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t cand = th | (1u << bit);
      int c = 0;
#pragma unroll
      for (int i = 0; i < items; ++i) c += get(i) >= cand;
      const int all = (int)block_sum(c, slots, phase);
      phase ^= 1;
      if (all >= need) th = cand;
      if (all == need) break;  // exactly the keys >= th: the lower bits do not matter
    }
  }
  int above = 0, ties = 0;
#pragma unroll
  for (int i = 0; i < items; ++i) {
    const uint32_t k = get(i);
    above += need > 0 && k > th;
    ties += need > 0 && k == th;
  }
  const int all_above = (int)block_sum(above, slots, phase);
  phase ^= 1;
  const int ties_before = block_scan(ties, slots, phase);
  phase ^= 1;
  const int tie_room = need - all_above;  // ties taken, lowest indices first
  const int forced = (int)(min(i0 + items, (long long)n) - min(i0, (long long)n)) -
                     (int)max(0ll, min(i0 + items, (long long)(n - recent)) -
                                       max(i0, (long long)first));
  const int mine = above + min(ties, max(0, tie_room - ties_before)) + max(0, forced);
  int at = block_scan(mine, slots, phase);
  int tie = ties_before;
#pragma unroll
  for (int i = 0; i < items; ++i) {
    const long long j = i0 + i;
    if (j >= n) break;
    bool take = j < first || j >= n - recent;
    if (!take && need > 0) {
      const uint32_t k = get(i);
      take = k > th || (k == th && tie < tie_room);
      tie += k == th;
    }
    if (take) o[at++] = (int)j;
  }
}

}  // namespace

cudaError_t launch_block_scores(const void* q, const int32_t* positions, const void* k_bounds,
                                int B, int Hq, int Hkv, int L, int block, float* scores,
                                cudaStream_t stream) {
  const int nb = (L + block - 1) / block;
  const int ctas = (nb + kScoreBlocksPerCta - 1) / kScoreBlocksPerCta;
  return launch_pdl(block_scores_kernel, dim3(B * Hkv, ctas), dim3(kScoreWarps * 32), 0, stream,
                    static_cast<const uint4*>(q), positions, static_cast<const uint4*>(k_bounds),
                    scores, Hkv, Hq / Hkv, L, block, nb);
}

cudaError_t launch_block_select(const float* scores, const int32_t* positions, int B, int Hkv,
                                int L, int block, int count, int first, int recent, int32_t* out,
                                cudaStream_t stream) {
  const int nb = (L + block - 1) / block;
  const int per = (nb + kSelectThreads - 1) / kSelectThreads;
  auto kernel = per <= 1    ? block_select_kernel<1>
                : per <= 2  ? block_select_kernel<2>
                : per <= 4  ? block_select_kernel<4>
                : per <= 8  ? block_select_kernel<8>
                : per <= 16 ? block_select_kernel<16>
                : per <= 32 ? block_select_kernel<32>
                            : block_select_kernel<0>;
  return launch_pdl(kernel, dim3(B * Hkv), dim3(kSelectThreads), 0, stream, scores, positions,
                    out, Hkv, L, block, nb, count, first, recent);
}

}  // namespace gqa
