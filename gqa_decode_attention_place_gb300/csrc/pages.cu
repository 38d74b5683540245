// pages.cu -- the pages of a paged cache: given out to new rows (with the copy
// of a page that several sequences share), passed on to forked sequences,
// freed, and moved to the front of the pool.
//
// The whole state is the table [B, M] (the page of rows j*page .. of sequence
// b, -1 none) and one count per page, how many entries name it; a page whose
// count is 0 is free.  There is no free list to keep: the lowest free pages
// are taken, in the order of the sequences, so results depend on the state
// alone.  Counts change by integer atomics, whose order does not matter.
//
// Latency bounds the bookkeeping (a few hundred KB at most).  Reserve and compact
// are one launch for a small pool: every CTA scans all counts for itself and copies
// its part of the rows.  For a larger one a cluster scans them, its CTAs' sums meet
// through distributed shared memory, and a second launch over the whole GPU copies
// rows with the list ready.
#include <cooperative_groups.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "paged.h"

namespace gqa {
namespace {

namespace cg = cooperative_groups;

constexpr int kScanThreads = 1024;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kManyCtas = 8;     // of the cluster that scans a large pool
constexpr int kCopyThreads = 256;
// Up to these sizes a call is one launch: every CTA scans the counts for itself.
constexpr int kSoloPages = 16384;     // reserve
constexpr int kSoloItems = 1024;
constexpr int kSoloPool = 8192;       // compact
// and so many 16-row copies (4096 pages of 64 KB: 30 us in one launch, 32 in two; 2048
// of 512 KB: 92 and 85)
constexpr int kSoloUnits = 49152;

__device__ __forceinline__ uint32_t lanes_below(int lane) { return (1u << lane) - 1u; }

// A warp's contiguous part of [0, n), split over the warps of C CTAs.
struct Span {
  int lo, hi;
};
template <int C>
__device__ __forceinline__ Span span_of(int n, int rank, int warp) {
  const long long w = (long long)rank * kScanWarps + warp, all = C * kScanWarps;
  return Span{(int)((long long)n * w / all), (int)((long long)n * (w + 1) / all)};
}

// Exclusive sums over all warps, in order, of N counts each; total[] over all.
// C > 1: the kernel arrived at the cluster's barrier when it started.
template <int C, int N>
struct Prefix {
  int warps[N][kScanWarps], ctas[N][C];
  __device__ __forceinline__ void operator()(const int (&count)[N], int (&before)[N],
                                             int (&total)[N]) {
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (lane == 0) warps[i][warp] = count[i];
    __syncthreads();
    // every CTA has started before another writes into its shared memory
    if (C > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) {
      int x = warps[i][lane];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
      }
      before[i] = __shfl_sync(0xffffffffu, x, warp) - count[i];
      total[i] = __shfl_sync(0xffffffffu, x, 31);
      if (C > 1 && warp == i && lane < C) cluster.map_shared_rank(ctas[i], lane)[rank] = total[i];
    }
    if (C == 1) return;
    cluster.sync();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      total[i] = 0;
#pragma unroll
      for (int r = 0; r < C; ++r) {
        const int c = ctas[i][r];
        total[i] += c;
        before[i] += r < rank ? c : 0;
      }
    }
  }
};

// The counts of a warp's span of pages as bits, one word of 32 pages at a time;
// the first kWords stay in registers for a second look.
struct PageBits {
  static constexpr int kWords = 16;
  uint32_t kept[kWords];
  const int32_t* refs;
  Span s;
  int lane;
  // The first words' loads, to be under way beside others; their values become
  // bits in settle().
  __device__ __forceinline__ PageBits(const int32_t* refs_, Span s_, int lane_)
      : refs(refs_), s(s_), lane(lane_) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const int i = s.lo + 32 * k + lane;
      kept[k] = i < s.hi ? (uint32_t)refs[i] : 0u;
    }
  }
  __device__ __forceinline__ void settle() {
#pragma unroll
    for (int k = 0; k < kWords; ++k) kept[k] = __ballot_sync(0xffffffffu, (int)kept[k] > 0);
  }
  __device__ __forceinline__ uint32_t look(int k) const {  // pages in use, of word k
    const int i = s.lo + 32 * k + lane;
    return __ballot_sync(0xffffffffu, i < s.hi && refs[i] > 0);
  }
  __device__ __forceinline__ uint32_t valid(int k) const {
    const int n = s.hi - s.lo - 32 * k;
    return n >= 32 ? 0xffffffffu : (1u << n) - 1u;
  }
  // f(k, bits) for every word, until it says false.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int n = (s.hi - s.lo + 31) >> 5;
    bool on = true;
#pragma unroll
    for (int k = 0; k < kWords; ++k)
      if (on && k < n) on = f(k, kept[k]);
#pragma unroll 4
    for (int k = kWords; k < n && on; ++k) on = f(k, look(k));
  }
};

// Rows r0 .. r1 - 1 (16 at most) of one operand and head of page `from` to page
// `to`, by a warp: all of a lane's loads (four or eight) are under way at once.
__device__ __forceinline__ void copy_rows(uint8_t* base, const PagedPool& pool, int h, int from,
                                          int to, int r0, int r1, int lane, uint32_t* status) {
  if (!range_ok(from >= 0 && from < pool.P && to >= 0 && to < pool.P && h < pool.Hkv && r0 < r1 &&
                    r1 <= pool.page && r1 - r0 <= 16,
                status))
    return;
  const int lv = pool.D == 128 ? 4 : 3;
  const int vecs = (r1 - r0) << lv;
  const long long rs = pool.row_stride >> 3, step = rs << (5 - lv);  // of 32 vectors
  const long long in = (h * pool.head_stride >> 3) + (r0 + (lane >> lv)) * rs +
                       (lane & ((1 << lv) - 1));
  const uint4* src = reinterpret_cast<const uint4*>(base) + (from * pool.page_stride >> 3) + in;
  uint4* dst = reinterpret_cast<uint4*>(base) + (to * pool.page_stride >> 3) + in;
  uint4 x[8];
#pragma unroll
  for (int u = 0; u < 8; ++u)
    if (lane + 32 * u < vecs) x[u] = src[u * step];
#pragma unroll
  for (int u = 0; u < 8; ++u)
    if (lane + 32 * u < vecs) dst[u * step] = x[u];
}

// Unit u of copied pages: page `c`, operand and head `oh`, first row.
struct Unit {
  int c, oh, r0;
  // lp: log2 of the page's rows; heads: operands and heads of a page
  __device__ __forceinline__ Unit(uint32_t u, int lp, int heads) {
    const uint32_t x = u >> (lp - 4);
    c = (int)(x / (uint32_t)heads);
    oh = (int)(x - (uint32_t)c * heads);
    r0 = (int)(u & ((1u << (lp - 4)) - 1u)) * 16;
  }
};

// Thread 0 of a CTA that has read all it will: whether it is the last of the
// grid's, and may write what others read.
__device__ __forceinline__ bool last_to_read(uint32_t* ticket) {
  __threadfence();  // (the other threads' reads came before a barrier)
  const bool last = atomicAdd(ticket, 1u) + 1 == gridDim.x;
  if (last) *ticket = 0;
  __threadfence();
  return last;
}

// ---------------------------------------------------------------- reserve --

struct ReserveParams {
  int32_t* table;
  int32_t* refs;
  const int32_t* positions;
  const int32_t* lengths;
  int32_t* taken;
  uint32_t* status;
  uint32_t* ticket;
  int* n_copies;
  int4* copies;    // (from, to, rows) in any order
  int2* reach;     // [B] needed pages before and up to a sequence
  int32_t* info;   // [B * per] what an item's entry names, or kNothing
  int32_t* list;   // free pages, in order
  int B, S, M, P, lp, cap, per;
};
constexpr int kNothing = -2;  // an item that needs no page

// An item is one of the `per` pages that a sequence's new rows can touch.
struct Item {
  int was;  // its entry if it needs a page: -1 (it has none) or the page that others share
  int pos;
  __device__ __forceinline__ Item(const ReserveParams& p, int b, int jj) {
    const int n = p.lengths ? p.lengths[b] : p.S;
    pos = p.positions[b];
    was = kNothing;
    if (n <= 0 || n > p.S || n > p.cap || !rows_in_cache(pos, n - 1, p.cap)) return;
    const int j = (pos >> p.lp) + jj;
    if (j > (pos + n - 1) >> p.lp) return;
    const int page = p.table[(size_t)b * p.M + j];
    if (page < 0 || page >= p.P) was = -1;
    else if (p.refs[page] > 1) was = page;
  }
};

// The item's page changes hands.
__device__ __forceinline__ void give(const ReserveParams& p, int b, int jj, int was, int pos,
                                     int page) {
  if (!range_ok(page >= 0 && page < p.P && b < p.B && (pos >> p.lp) + jj < p.M, p.status)) return;
  p.table[(size_t)b * p.M + (pos >> p.lp) + jj] = page;
  p.refs[page] = 1;
  if (was >= 0) atomicSub(&p.refs[was], 1);
}
// Rows to copy from the page `was` that item jj leaves: those before the new ones.
__device__ __forceinline__ int copied(const ReserveParams& p, int jj, int was, int pos) {
  return jj == 0 && was >= 0 ? pos & ((1 << p.lp) - 1) : 0;
}
// What a sequence took, of its needed pages' reach; sets the status of one that does not fit.
__device__ __forceinline__ int taken_by(const ReserveParams& p, int n, int pos, int2 reach,
                                        int n_free) {
  if (n == 0) return 0;
  if (n < 0 || n > p.S || n > p.cap || !rows_in_cache(pos, n - 1, p.cap)) {
    set_status(p.status, ATTN_DEV_BAD_POSITION);
    return -1;
  }
  return reach.y == reach.x ? 0 : reach.y <= n_free ? reach.y - reach.x : -1;
}

// A small pool: every CTA works out who gets what from the state as it was, an
// item a thread, and copies its part of the rows; the last one to have read the
// state changes it.  No CTA waits for another.  (One CTA's scan, then a launch of
// copies: 8.4 us on the device for 256 sequences' step instead of 6.3, and 2 more
// of the host's time.)
__global__ void __launch_bounds__(kScanThreads, 1)
    pages_reserve_solo_kernel(const ReserveParams p, const PagedPool pool) {
  __shared__ Prefix<1, 2> prefix;
  __shared__ int list[kSoloItems];
  __shared__ int2 reach[kSoloItems];
  __shared__ int4 copies[kSoloItems];  // by sequence: (from, to, rows)
  __shared__ bool last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dependency_wait();
  grid_dependents_launch();
  const int items = p.B * p.per, b = tid / p.per, jj = tid - b * p.per;
  int was = kNothing, pos = 0, n_b = 0, pos_b = 0;
  PageBits bits(p.refs, span_of<1>(p.P, 0, warp), lane);
  if (tid < p.B) {
    n_b = p.lengths ? p.lengths[tid] : p.S;
    pos_b = p.positions[tid];
  }
  if (tid < items) {
    const Item x(p, b, jj);
    was = x.was;
    pos = x.pos;
  }
  bits.settle();
  int count[2] = {0, 0}, before[2], total[2];
  bits.each([&](int k, uint32_t used) {
    count[0] += __popc(~used & bits.valid(k));
    return true;
  });
  const uint32_t need = __ballot_sync(0xffffffffu, was != kNothing);
  count[1] = __popc(need);
  prefix(count, before, total);
  if (tid == 0) last = last_to_read(p.ticket);  // (this CTA has read all of the state)
  bits.each([&](int k, uint32_t used) {
    if (before[0] >= total[1]) return false;  // no more are wanted
    const uint32_t m = ~used & bits.valid(k);
    const int to = before[0] + __popc(m & lanes_below(lane));
    if ((m >> lane & 1) && to < total[1] && range_ok(to < kSoloItems, p.status))
      list[to] = bits.s.lo + 32 * k + lane;
    before[0] += __popc(m);
    return true;
  });
  const int k = before[1] + __popc(need & lanes_below(lane));
  if (tid < items) {
    if (jj == 0) reach[b].x = k;
    if (jj == p.per - 1) reach[b].y = k + (was != kNothing);
  }
  __syncthreads();
  // a sequence gets its pages if there are enough for it and those before it
  const bool given = was != kNothing && reach[b].y <= total[0];
  const int page = given ? list[k] : -1;
  const int rows = given ? copied(p, jj, was, pos) : 0;
  if (tid < items && jj == 0) copies[b] = make_int4(was, page, rows, 0);
  const bool some = __syncthreads_or(rows > 0);
  const int heads = 2 * pool.Hkv;
  const uint32_t units = (uint32_t)(p.B * heads) << (p.lp - 4);
  for (uint32_t u = blockIdx.x * kScanWarps + warp; some && u < units;
       u += gridDim.x * kScanWarps) {
    const Unit v(u, p.lp, heads);
    const int4 x = copies[v.c];
    if (v.r0 < x.z)
      copy_rows(v.oh & 1 ? pool.v : pool.k, pool, v.oh >> 1, x.x, x.y, v.r0,
                min(v.r0 + 16, x.z), lane, p.status);
  }
  if (!last) return;
  if (given) give(p, b, jj, was, pos, page);
  if (tid < p.B) p.taken[tid] = taken_by(p, n_b, pos_b, reach[tid], total[0]);
}

// A larger one: a cluster.  Three steps, a barrier between them: count the free pages
// and the needed ones; list the free pages that are wanted and how far the
// sequences reach; give the pages out.
__global__ void __launch_bounds__(kScanThreads, 1) pages_reserve_kernel(const ReserveParams p) {
  constexpr int C = kManyCtas;
  __shared__ Prefix<C, 2> prefix;
  const int rank = (int)cg::this_cluster().block_rank(), tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  grid_dependency_wait();
  grid_dependents_launch();
  const Span is = span_of<C>(p.B * p.per, rank, warp);
  if (rank == 0 && tid == 0) *p.n_copies = 0;

  // the first 32 items of a warp stay in registers, the others in `info`
  PageBits bits(p.refs, span_of<C>(p.P, rank, warp), lane);
  int first = kNothing, pos0 = 0, count[2] = {0, 0};
  if (is.lo + lane < is.hi) {
    const int b = (is.lo + lane) / p.per;
    const Item x(p, b, is.lo + lane - b * p.per);
    first = x.was;
    pos0 = x.pos;
  }
  bits.settle();
  bits.each([&](int k, uint32_t used) {
    count[0] += __popc(~used & bits.valid(k));
    return true;
  });
  count[1] = __popc(__ballot_sync(0xffffffffu, first != kNothing));
  for (int i0 = is.lo + 32; i0 < is.hi; i0 += 32) {
    const int i = i0 + lane;
    int was = kNothing;
    if (i < is.hi) {
      const int b = i / p.per;
      was = Item(p, b, i - b * p.per).was;
      p.info[i] = was;
    }
    count[1] += __popc(__ballot_sync(0xffffffffu, was != kNothing));
  }
  int before[2], total[2];
  prefix(count, before, total);
  const int n_free = total[0], n_need = total[1];

  int at = before[0];
  bits.each([&](int k, uint32_t used) {
    if (at >= n_need) return false;  // no more are wanted
    const uint32_t m = ~used & bits.valid(k);
    const int to = at + __popc(m & lanes_below(lane));
    if ((m >> lane & 1) && to < n_need && range_ok(to < p.B * p.per, p.status))
      p.list[to] = bits.s.lo + 32 * k + lane;
    at += __popc(m);
    return true;
  });
  at = before[1];
  int k0 = 0;  // of the first item
  for (int i0 = is.lo; i0 < is.hi; i0 += 32) {
    const int i = i0 + lane;
    const bool need = (i0 == is.lo ? first : i < is.hi ? p.info[i] : kNothing) != kNothing;
    const uint32_t m = __ballot_sync(0xffffffffu, need);
    const int k = at + __popc(m & lanes_below(lane));
    if (i0 == is.lo) k0 = k;
    if (i < is.hi) {
      const int b = i / p.per, jj = i - b * p.per;
      if (jj == 0) p.reach[b].x = k;
      if (jj == p.per - 1) p.reach[b].y = k + need;
    }
    at += __popc(m);
  }
  cg::this_cluster().sync();

  auto hand_over = [&](int b, int jj, int was, int pos, int page) {
    give(p, b, jj, was, pos, page);
    const int rows = copied(p, jj, was, pos);
    if (rows == 0) return;
    const int at = atomicAdd(p.n_copies, 1);
    if (range_ok(at < p.B, p.status)) p.copies[at] = make_int4(was, page, rows, 0);
  };
  if (first != kNothing) {
    const int b = (is.lo + lane) / p.per, jj = is.lo + lane - b * p.per;
    if (p.reach[b].y <= n_free) hand_over(b, jj, first, pos0, p.list[k0]);
  }
  at = before[1] + __popc(__ballot_sync(0xffffffffu, first != kNothing));
  for (int i0 = is.lo + 32; i0 < is.hi; i0 += 32) {
    const int i = i0 + lane;
    const int was = i < is.hi ? p.info[i] : kNothing;
    const uint32_t m = __ballot_sync(0xffffffffu, was != kNothing);
    const int k = at + __popc(m & lanes_below(lane));
    at += __popc(m);
    if (was == kNothing) continue;
    const int b = i / p.per, jj = i - b * p.per;
    if (p.reach[b].y <= n_free) hand_over(b, jj, was, p.positions[b], p.list[k]);
  }
  for (int b = rank * kScanThreads + tid; b < p.B; b += C * kScanThreads)
    p.taken[b] = taken_by(p, p.lengths ? p.lengths[b] : p.S, p.positions[b], p.reach[b], n_free);
}

// ------------------------------------------------------------------ copies --

// A warp for each (copy, operand, head, 16 rows).  (A warp for all rows of a
// head: 64 copies of up to 127 rows, 8 heads: 10.5 us instead of 4.4.)
__global__ void __launch_bounds__(kCopyThreads) pages_copy_rows_kernel(
    PagedPool pool, const int* __restrict__ n_copies, const int4* __restrict__ copies,
    uint32_t* status) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int lane = threadIdx.x & 31, parts = pool.page >> 4, per = 2 * pool.Hkv * parts;
  const long long units = (long long)*n_copies * per;
  for (long long u = ((long long)blockIdx.x * kCopyThreads + threadIdx.x) >> 5; u < units;
       u += (long long)gridDim.x * (kCopyThreads / 32)) {
    const int c = (int)(u / per);
    int rest = (int)(u - (long long)c * per);
    const int r0 = rest % parts * 16;
    rest /= parts;
    const int4 x = copies[c];
    if (r0 < x.z)
      copy_rows(rest & 1 ? pool.v : pool.k, pool, rest >> 1, x.x, x.y, r0, min(r0 + 16, x.z),
                lane, status);
  }
}

// -------------------------------------------------------------------- fork --

// Row b becomes what row parents[b] was, cut to the pages of its first
// lengths[b] rows.  A CTA takes 8 or 32 columns of all rows, so that it has read
// what it will write over: a column's entries depend on that column alone.  A
// thread's first kForkRows rows stay in registers: all its loads are one round trip.
constexpr int kForkThreads = 1024;
constexpr int kForkRows = 4;
__global__ void __launch_bounds__(kForkThreads) pages_fork_kernel(
    int32_t* __restrict__ table, int32_t* __restrict__ refs, const int32_t* __restrict__ parents,
    const int32_t* __restrict__ lengths, int B, int M, int P, int lp, int lc, uint32_t* status) {
  extern __shared__ int32_t old[];  // [B][columns]
  grid_dependency_wait();
  grid_dependents_launch();
  const int col = threadIdx.x & ((1 << lc) - 1), j = (blockIdx.x << lc) + col;
  const int b0 = threadIdx.x >> lc, step = kForkThreads >> lc;
  int was[kForkRows], from[kForkRows], kept[kForkRows];
#pragma unroll
  for (int k = 0; k < kForkRows; ++k) {
    const int b = b0 + k * step;
    was[k] = b < B && j < M ? table[(size_t)b * M + j] : -1;
    from[k] = b < B ? parents[b] : -1;
    kept[k] = lengths && b < B ? lengths[b] : 0x7fffffff;
  }
#pragma unroll
  for (int k = 0; k < kForkRows; ++k)
    if (b0 + k * step < B) old[((b0 + k * step) << lc) + col] = was[k];
#pragma unroll 4
  for (int b = b0 + kForkRows * step; b < B; b += step)
    old[(b << lc) + col] = j < M ? table[(size_t)b * M + j] : -1;
  __syncthreads();
  if (j >= M) return;
  auto pass_on = [&](int b, int was, int from, int kept) {
    if (from < -1 || from >= B) {  // no such row: this one stays
      set_status(status, ATTN_DEV_BAD_PARENT);
      from = b;
    }
    int now = from < 0 ? -1 : old[(from << lc) + col];
    if ((long long)j << lp >= kept) now = -1;
    if (now == was) return;
    table[(size_t)b * M + j] = now;
    if (now >= 0 && now < P) atomicAdd(&refs[now], 1);
    if (was >= 0 && was < P) atomicSub(&refs[was], 1);
  };
#pragma unroll
  for (int k = 0; k < kForkRows; ++k)
    if (b0 + k * step < B) pass_on(b0 + k * step, was[k], from[k], kept[k]);
  for (int b = b0 + kForkRows * step; b < B; b += step)
    pass_on(b, old[(b << lc) + col], parents[b], lengths ? lengths[b] : 0x7fffffff);
}
// Without parents: only entries past the kept rows are looked at.  A warp for
// 256 columns of a row, all of a lane's eight loads under way at once.
__global__ void __launch_bounds__(256) pages_cut_kernel(int32_t* __restrict__ table,
                                                        int32_t* __restrict__ refs,
                                                        const int32_t* __restrict__ lengths, int B,
                                                        int M, int P, int lp) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int lane = threadIdx.x & 31, b = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (b >= B) return;
  const int first = (int)(((long long)max(lengths[b], 0) + (1 << lp) - 1) >> lp);
  const int j0 = blockIdx.x * 256 + lane;
  int32_t* row = table + (size_t)b * M;
  int was[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int j = j0 + 32 * k;
    was[k] = j >= first && j < M ? row[j] : -1;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (was[k] == -1) continue;
    row[j0 + 32 * k] = -1;
    if (was[k] >= 0 && was[k] < P) atomicSub(&refs[was[k]], 1);
  }
}

// ----------------------------------------------------------------- compact --

struct CompactParams {
  int32_t* table;
  int32_t* refs;
  int32_t* map;
  uint32_t* status;
  uint32_t* ticket;
  int* n_moves;
  int32_t* from;  // [P] used pages by how many come before them
  int32_t* to;    // [P] free pages by how many come before them
  int B, M, P, lp;
};

// A small pool in one launch: every CTA works the moves out for itself, and does
// its part of the rows and of the table; the last one to have read the counts
// changes them.
__global__ void __launch_bounds__(kScanThreads, 1)
    pages_compact_solo_kernel(const CompactParams p, const PagedPool pool) {
  __shared__ Prefix<1, 1> prefix;
  // from: the high pages from the last on; to: the free pages below n
  __shared__ uint16_t from[kSoloPool / 2], to[kSoloPool / 2], where[kSoloPool];
  __shared__ int holes;  // free pages below n
  __shared__ bool last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dependency_wait();
  grid_dependents_launch();
  PageBits bits(p.refs, span_of<1>(p.P, 0, warp), lane);
  int count[1] = {0}, at[1], total[1];
  bits.settle();
  bits.each([&](int, uint32_t used) {
    count[0] += __popc(used);
    return true;
  });
  if (tid == 0) holes = 0;
  prefix(count, at, total);
  const int n = total[0];
  if (tid == 0) last = last_to_read(p.ticket);  // (this CTA has read all of the counts)
  bits.each([&](int k, uint32_t m) {
    const int i = bits.s.lo + 32 * k + lane;
    const int before = at[0] + __popc(m & lanes_below(lane));  // used pages before i
    at[0] += __popc(m);
    if (i >= bits.s.hi) return true;
    if (i == n) holes = n - before;
    const bool used = m >> lane & 1;
    if (used && i >= n && range_ok(n - 1 - before < kSoloPool / 2, p.status))
      from[n - 1 - before] = (uint16_t)i;
    if (!used && i < n && range_ok(i - before < kSoloPool / 2, p.status))
      to[i - before] = (uint16_t)i;
    where[i] = used ? (uint16_t)i : 0xffff;
    return true;
  });
  __syncthreads();
  const int moves = holes;
  for (int k = tid; k < moves; k += kScanThreads) where[from[moves - 1 - k]] = to[k];
  __syncthreads();
  const int thread = blockIdx.x * kScanThreads + tid, threads = gridDim.x * kScanThreads;
  for (int i = thread; i < p.P; i += threads) p.map[i] = where[i] == 0xffff ? -1 : where[i];
  if (moves == 0) return;
  for (long long i = thread; i < (long long)p.B * p.M; i += threads) {
    const int e = p.table[i];
    if (e >= n && e < p.P) p.table[i] = where[e] == 0xffff ? -1 : where[e];
  }
  const int heads = 2 * pool.Hkv;
  const uint32_t units = (uint32_t)(moves * heads) << (p.lp - 4);
  for (uint32_t u = thread >> 5; u < units; u += threads >> 5) {
    const Unit v(u, p.lp, heads);
    copy_rows(v.oh & 1 ? pool.v : pool.k, pool, v.oh >> 1, from[moves - 1 - v.c], to[v.c], v.r0,
              v.r0 + 16, lane, p.status);
  }
  if (!last) return;
  for (int k = tid; k < moves; k += kScanThreads) {
    const int src = from[moves - 1 - k], dst = to[k];
    p.refs[dst] = p.refs[src];
    p.refs[src] = 0;
  }
}

// n pages are in use: the k-th of those at n or above goes to the k-th free
// page below n.  A cluster.
__global__ void __launch_bounds__(kScanThreads, 1) pages_plan_kernel(const CompactParams p) {
  constexpr int C = kManyCtas;
  __shared__ Prefix<C, 1> prefix;
  const int rank = (int)cg::this_cluster().block_rank(), tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  grid_dependency_wait();
  grid_dependents_launch();
  PageBits bits(p.refs, span_of<C>(p.P, rank, warp), lane);
  int count[1] = {0}, at[1], total[1];
  bits.settle();
  bits.each([&](int, uint32_t used) {
    count[0] += __popc(used);
    return true;
  });
  prefix(count, at, total);
  const int n = total[0];
  bits.each([&](int k, uint32_t m) {
    const int i = bits.s.lo + 32 * k + lane;
    const int before = at[0] + __popc(m & lanes_below(lane));  // used pages before i
    at[0] += __popc(m);
    if (i >= bits.s.hi) return true;
    if (i == n) {
      p.n_moves[0] = n - before;  // as many high pages as low holes
      p.n_moves[1] = n;
    }
    if (m >> lane & 1) {
      if (!range_ok(before >= 0 && before < p.P, p.status)) return true;
      if (i >= n) p.from[before] = i;
      else p.map[i] = i;
    } else {
      if (i < n && range_ok(i - before >= 0 && i - before < p.P, p.status)) p.to[i - before] = i;
      p.map[i] = -1;
    }
    return true;
  });
  if (n == p.P && rank == 0 && tid == 0) p.n_moves[0] = 0;  // no page is free
  cg::this_cluster().sync();
  const int moves = *(volatile int*)p.n_moves;
  for (int k = rank * kScanThreads + tid; k < moves; k += C * kScanThreads) {
    const int src = p.from[n - moves + k], dst = p.to[k];
    p.map[src] = dst;
    p.refs[dst] = p.refs[src];
    p.refs[src] = 0;
  }
}

// The moved pages' rows, a warp for each (move, operand, head, 16 rows), and the table.
__global__ void __launch_bounds__(kCopyThreads) pages_move_kernel(CompactParams p, PagedPool pool) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int moves = p.n_moves[0], n = p.n_moves[1];
  if (moves == 0) return;  // (nothing in the table changes either)
  const int lane = threadIdx.x & 31, parts = pool.page >> 4, per = 2 * pool.Hkv * parts;
  const long long thread = (long long)blockIdx.x * kCopyThreads + threadIdx.x;
  const long long threads = (long long)gridDim.x * kCopyThreads;
  for (long long i = thread; i < (long long)p.B * p.M; i += threads) {
    const int e = p.table[i];
    if (e < n || e >= p.P) continue;  // pages below n stay
    p.table[i] = p.map[e];
  }
  const long long units = (long long)moves * per;
  for (long long u = thread >> 5; u < units; u += threads >> 5) {
    const int c = (int)(u / per);
    int rest = (int)(u - (long long)c * per);
    const int r0 = rest % parts * 16;
    rest /= parts;
    copy_rows(rest & 1 ? pool.v : pool.k, pool, rest >> 1, p.from[n - moves + c], p.to[c], r0,
              r0 + 16, lane, p.status);
  }
}

// A scanning kernel on a cluster of kManyCtas.
template <typename P>
cudaError_t launch_scan(void (*kernel)(P), cudaStream_t stream, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kManyCtas);
  cfg.blockDim = dim3(kScanThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kManyCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// The current device's SMs; found once per device, with what its kernels need.
cudaError_t sm_count(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if ((*sms = known[dev].load(std::memory_order_acquire)) > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(pages_fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             128 * 1024);
  if (e == cudaSuccess) known[dev].store(*sms, std::memory_order_release);
  return e;
}
// CTAs for `warps` warps' work, one to an SM.
dim3 solo_grid(long long warps, int sms) {
  return dim3((unsigned)max(1ll, min((warps + kScanWarps - 1) / kScanWarps, (long long)sms)));
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

// [B] copies, [B] reaches, then info and list [B * per] each.
PagesWorkspace pages_reserve_layout(int B, int S, int page) {
  const size_t per = (size_t)pages_touched(S, page);
  PagesWorkspace w;
  w.copies_off = 256;
  w.list_off = align256(w.copies_off + (size_t)B * 24);
  w.total = align256(w.list_off + (size_t)B * per * 8);
  return w;
}
PagesWorkspace pages_compact_layout(int P) {
  PagesWorkspace w;
  w.copies_off = w.list_off = 256;
  w.total = align256(w.list_off + (size_t)P * 8);
  return w;
}

cudaError_t launch_pages_reserve(int32_t* table, int32_t* refs, const int32_t* positions,
                                 const int32_t* lengths, const PagedPool& pool, int B, int S, int M,
                                 int32_t* taken, void* workspace, cudaStream_t stream) {
  const PagesWorkspace ws = pages_reserve_layout(B, S, pool.page);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  ReserveParams p;
  p.table = table;
  p.refs = refs;
  p.positions = positions;
  p.lengths = lengths;
  p.taken = taken;
  p.status = reinterpret_cast<uint32_t*>(base);
  p.ticket = reinterpret_cast<uint32_t*>(base + 64);
  p.n_copies = reinterpret_cast<int*>(base + 128);
  p.copies = reinterpret_cast<int4*>(base + ws.copies_off);
  p.reach = reinterpret_cast<int2*>(base + ws.copies_off + (size_t)B * 16);
  p.B = B;
  p.S = S;
  p.M = M;
  p.P = pool.P;
  p.lp = log2_of(pool.page);
  p.cap = M * pool.page;
  p.per = (int)pages_touched(S, pool.page);
  p.info = reinterpret_cast<int32_t*>(base + ws.list_off);
  p.list = p.info + (size_t)B * p.per;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const long long warps = (long long)B * 2 * pool.Hkv * (pool.page >> 4);  // of copies, at most
  if (pool.P <= kSoloPages && (long long)B * p.per <= kSoloItems)
    return launch_pdl(pages_reserve_solo_kernel, solo_grid(warps, sms), dim3(kScanThreads), 0,
                      stream, p, pool);
  e = launch_scan(pages_reserve_kernel, stream, p);
  if (e != cudaSuccess) return e;
  const long long blocks = (warps * 32 + kCopyThreads - 1) / kCopyThreads;
  return launch_pdl(pages_copy_rows_kernel, dim3((unsigned)min(blocks, (long long)sms * 8)),
                    dim3(kCopyThreads), 0, stream, pool, (const int*)p.n_copies,
                    (const int4*)p.copies, p.status);
}

cudaError_t launch_pages_fork(int32_t* table, int32_t* refs, const int32_t* parents,
                              const int32_t* lengths, int B, int M, int P, int page,
                              void* workspace, cudaStream_t stream) {
  if (!parents) {
    if (!lengths) return cudaSuccess;
    return launch_pdl(pages_cut_kernel, dim3((M + 255) / 256, (B + 7) / 8), dim3(256), 0, stream,
                      table, refs, lengths, B, M, P, log2_of(page));
  }
  // 128-byte pieces of rows; 32-byte ones where that many rows would not fit, or
  // where that makes CTAs for SMs that would have none
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int lc = B > 1024 || M <= 8 * sms ? 3 : 5;
  const size_t smem = ((size_t)B << lc) * 4;
  return launch_pdl(pages_fork_kernel, dim3((M + (1 << lc) - 1) >> lc), dim3(kForkThreads), smem,
                    stream, table, refs, parents, lengths, B, M, P, log2_of(page), lc,
                    reinterpret_cast<uint32_t*>(workspace));
}

cudaError_t launch_pages_compact(int32_t* table, int32_t* refs, const PagedPool& pool, int B,
                                 int M, int32_t* page_map, void* workspace, cudaStream_t stream) {
  const PagesWorkspace ws = pages_compact_layout(pool.P);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  CompactParams p;
  p.table = table;
  p.refs = refs;
  p.map = page_map;
  p.status = reinterpret_cast<uint32_t*>(base);
  p.ticket = reinterpret_cast<uint32_t*>(base + 64);
  p.n_moves = reinterpret_cast<int*>(base + 128);
  p.from = reinterpret_cast<int32_t*>(base + ws.list_off);
  p.to = p.from + pool.P;
  p.B = B;
  p.M = M;
  p.P = pool.P;
  p.lp = log2_of(pool.page);
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  // 16-row copies, as many as there can be, and CTAs' worth of table entries
  const long long units = (long long)(pool.P / 2) * 2 * pool.Hkv * (pool.page >> 4);
  if (pool.P <= kSoloPool && units <= kSoloUnits)
    return launch_pdl(pages_compact_solo_kernel,
                      solo_grid(max(units, ((long long)B * M + 31) / 32), sms), dim3(kScanThreads),
                      0, stream, p, pool);
  e = launch_scan(pages_plan_kernel, stream, p);
  if (e != cudaSuccess) return e;
  // About one unit a warp: CTAs that come and go keep reads and writes of DRAM better
  // apart than a few that stay (8192 pages of 64 KB: 168 us by 64 to an SM, 177 by 8
  // and 206 by 2).
  const long long ctas = max(((long long)B * M + kCopyThreads - 1) / kCopyThreads,
                             units / (kCopyThreads / 32));
  return launch_pdl(pages_move_kernel, dim3((unsigned)max(1ll, min(ctas, (long long)sms * 64))),
                    dim3(kCopyThreads), 0, stream, p, pool);
}

}  // namespace gqa
