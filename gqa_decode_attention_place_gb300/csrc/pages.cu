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
// Latency bounds the bookkeeping (a few hundred KB at most): reserve and
// compact scan the counts with one cluster of 8 CTAs, whose sums meet through
// distributed shared memory, and the pages' rows are copied by a second launch
// over the whole GPU that starts with the list ready.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"
#include "paged.h"

namespace gqa {
namespace {

namespace cg = cooperative_groups;

constexpr int kCtas = 8;         // CTAs of the scanning cluster
constexpr int kScanThreads = 1024;
constexpr int kScanWarps = kScanThreads / 32;

int log2_of(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

__device__ __forceinline__ uint32_t lanes_below(int lane) { return (1u << lane) - 1u; }

// A warp's contiguous part of [0, n), split over the cluster's warps.
struct Span {
  int lo, hi;
};
__device__ __forceinline__ Span span_of(int n, int rank, int warp) {
  const long long w = (long long)rank * kScanWarps + warp, all = kCtas * kScanWarps;
  return Span{(int)((long long)n * w / all), (int)((long long)n * (w + 1) / all)};
}

// Exclusive sum over the cluster's warps, in order, of one count each; *total
// over all.  `mine` is [kScanWarps] of shared memory, `ctas` [kCtas] that every
// CTA of the cluster writes its own sum into.  begun: the cluster barrier that the
// kernel arrived at when it started is still to be waited for.
__device__ __forceinline__ int cluster_prefix(cg::cluster_group& cluster, bool begun, int count,
                                              int* mine, int* ctas, int* total) {
  const int rank = (int)cluster.block_rank(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) mine[warp] = count;
  __syncthreads();
  int x = mine[lane];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  const int before = __shfl_sync(0xffffffffu, x, warp) - count;
  const int sum = __shfl_sync(0xffffffffu, x, 31);
  // every CTA has started before another writes into its shared memory
  if (begun) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (warp == 0 && lane < kCtas) cluster.map_shared_rank(ctas, lane)[rank] = sum;
  cluster.sync();
  int all = 0, ahead = 0;
#pragma unroll
  for (int r = 0; r < kCtas; ++r) {
    const int c = ctas[r];
    all += c;
    ahead += r < rank ? c : 0;
  }
  *total = all;
  return ahead + before;
}

// ---------------------------------------------------------------- reserve --

struct ReserveParams {
  int32_t* table;
  int32_t* refs;
  const int32_t* positions;
  const int32_t* lengths;
  int32_t* taken;
  uint32_t* status;
  int* n_copies;
  int4* copies;    // (from, to, rows) in any order
  int2* reach;     // [B] needed pages before and up to a sequence
  int32_t* info;   // [B * per] what an item's entry names, or kNothing
  int32_t* list;   // free pages, in order
  int B, S, M, P, lp, cap, per;
};
constexpr int kNothing = -2;  // an item that needs no page

// The item's entry if it needs a page: -1 (it has none) or the page that others
// share; kNothing if it needs none.
__device__ __forceinline__ int item_info(const ReserveParams& p, int b, int jj) {
  const int n = p.lengths ? p.lengths[b] : p.S, pos = p.positions[b];
  if (n <= 0 || n > p.S || n > p.cap || !rows_in_cache(pos, n - 1, p.cap)) return kNothing;
  const int j = (pos >> p.lp) + jj;
  if (j > (pos + n - 1) >> p.lp) return kNothing;
  const int page = p.table[(size_t)b * p.M + j];
  if (page < 0 || page >= p.P) return -1;
  return p.refs[page] > 1 ? page : kNothing;
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kScanThreads, 1)
    pages_reserve_kernel(const ReserveParams p) {
  __shared__ int warps[2][kScanWarps], ctas[2][kCtas];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  grid_dependency_wait();
  grid_dependents_launch();
  const int items = p.B * p.per;
  const Span fs = span_of(p.P, rank, warp), is = span_of(items, rank, warp);
  if (rank == 0 && tid == 0) *p.n_copies = 0;

  // how many pages are free, and how many are needed
  int n_free = 0, n_need = 0;
  for (int i0 = is.lo; i0 < is.hi; i0 += 32) {
    const int i = i0 + lane;
    int x = kNothing;
    if (i < is.hi) {
      const int b = i / p.per;
      x = item_info(p, b, i - b * p.per);
      p.info[i] = x;
    }
    n_need += __popc(__ballot_sync(0xffffffffu, x != kNothing));
  }
#pragma unroll 4
  for (int i0 = fs.lo; i0 < fs.hi; i0 += 32) {
    const int i = i0 + lane;
    n_free += __popc(__ballot_sync(0xffffffffu, i < fs.hi && p.refs[i] <= 0));
  }
  int free_all, need_all;
  int at_free = cluster_prefix(cluster, true, n_free, warps[0], ctas[0], &free_all);
  int at_need = cluster_prefix(cluster, false, n_need, warps[1], ctas[1], &need_all);

  // the free pages that are wanted, and how far the sequences reach
#pragma unroll 4
  for (int i0 = fs.lo; i0 < fs.hi && at_free < need_all; i0 += 32) {
    const int i = i0 + lane;
    const bool is_free = i < fs.hi && p.refs[i] <= 0;
    const uint32_t m = __ballot_sync(0xffffffffu, is_free);
    const int k = at_free + __popc(m & lanes_below(lane));
    if (is_free && k < need_all) p.list[k] = i;
    at_free += __popc(m);
  }
  {
    int at = at_need;
    for (int i0 = is.lo; i0 < is.hi; i0 += 32) {
      const int i = i0 + lane;
      const bool need = i < is.hi && p.info[i] != kNothing;
      const uint32_t m = __ballot_sync(0xffffffffu, need);
      const int k = at + __popc(m & lanes_below(lane));
      if (i < is.hi) {
        const int b = i / p.per, jj = i - b * p.per;
        if (jj == 0) p.reach[b].x = k;
        if (jj == p.per - 1) p.reach[b].y = k + need;
      }
      at += __popc(m);
    }
  }
  cluster.sync();

  // the pages change hands
  for (int i0 = is.lo; i0 < is.hi; i0 += 32) {
    const int i = i0 + lane;
    const int was = i < is.hi ? p.info[i] : kNothing;
    const uint32_t m = __ballot_sync(0xffffffffu, was != kNothing);
    const int k = at_need + __popc(m & lanes_below(lane));
    at_need += __popc(m);
    if (was == kNothing) continue;
    const int b = i / p.per, jj = i - b * p.per;
    if (p.reach[b].y > free_all) continue;  // the pool is too small for this sequence
    const int page = p.list[k], pos = p.positions[b];
    p.table[(size_t)b * p.M + (pos >> p.lp) + jj] = page;
    p.refs[page] = 1;
    if (was >= 0) {
      atomicSub(&p.refs[was], 1);
      const int rows = pos & ((1 << p.lp) - 1);
      if (jj == 0 && rows > 0)
        p.copies[atomicAdd(p.n_copies, 1)] = make_int4(was, page, rows, 0);
    }
  }
  for (int b = rank * kScanThreads + tid; b < p.B; b += kCtas * kScanThreads) {
    const int n = p.lengths ? p.lengths[b] : p.S, pos = p.positions[b];
    int t = 0;
    if (n != 0) {
      if (n < 0 || n > p.S || n > p.cap || !rows_in_cache(pos, n - 1, p.cap)) {
        set_status(p.status, ATTN_DEV_BAD_POSITION);
        t = -1;
      } else {
        const int2 r = p.reach[b];
        t = r.y == r.x ? 0 : r.y <= free_all ? r.y - r.x : -1;
      }
    }
    p.taken[b] = t;
  }
}

// ------------------------------------------------------------------ copies --

// `rows` rows of one operand and head of page `from` to page `to`, by a warp.
__device__ __forceinline__ void copy_rows(uint8_t* base, const PagedPool& pool, int h, int from,
                                          int to, int rows, int lane) {
  const int lv = pool.D == 128 ? 4 : 3;
  const int vecs = rows << lv;
  const long long rs = pool.row_stride >> 3;
  const uint4* src = reinterpret_cast<const uint4*>(base) +
                     ((from * pool.page_stride + h * pool.head_stride) >> 3);
  uint4* dst = reinterpret_cast<uint4*>(base) +
               ((to * pool.page_stride + h * pool.head_stride) >> 3);
  for (int j0 = lane; j0 < vecs; j0 += 256) {
    uint4 x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = j0 + 32 * u;
      if (j < vecs) x[u] = src[(j >> lv) * rs + (j & ((1 << lv) - 1))];
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = j0 + 32 * u;
      if (j < vecs) dst[(j >> lv) * rs + (j & ((1 << lv) - 1))] = x[u];
    }
  }
}

constexpr int kCopyThreads = 256;
// A warp for each (copy, operand, head).
__global__ void __launch_bounds__(kCopyThreads) pages_copy_rows_kernel(
    PagedPool pool, const int* __restrict__ n_copies, const int4* __restrict__ copies) {
  grid_dependency_wait();
  grid_dependents_launch();
  const long long units = (long long)*n_copies * 2 * pool.Hkv;
  const int lane = threadIdx.x & 31;
  for (long long u = ((long long)blockIdx.x * kCopyThreads + threadIdx.x) >> 5; u < units;
       u += (long long)gridDim.x * (kCopyThreads / 32)) {
    const int c = (int)(u / (2 * pool.Hkv)), oh = (int)(u - (long long)c * 2 * pool.Hkv);
    const int4 x = copies[c];
    copy_rows(oh & 1 ? pool.v : pool.k, pool, oh >> 1, x.x, x.y, x.z, lane);
  }
}

// -------------------------------------------------------------------- fork --

// Row b becomes what row parents[b] was, cut to the pages of its first
// lengths[b] rows.  A CTA takes `cols` columns of all rows, so that it has read
// what it will write over: a column's entries depend on that column alone.
constexpr int kForkThreads = 1024;
__global__ void __launch_bounds__(kForkThreads) pages_fork_kernel(
    int32_t* __restrict__ table, int32_t* __restrict__ refs, const int32_t* __restrict__ parents,
    const int32_t* __restrict__ lengths, int B, int M, int P, int lp, int lc, uint32_t* status) {
  extern __shared__ int32_t old[];  // [B][cols]
  grid_dependency_wait();
  grid_dependents_launch();
  const int cols = 1 << lc, j0 = blockIdx.x << lc;
  const int col = threadIdx.x & (cols - 1), j = j0 + col;
  const int b0 = threadIdx.x >> lc, step = kForkThreads >> lc;
#pragma unroll 4
  for (int b = b0; b < B; b += step)
    old[(b << lc) + col] = j < M ? table[(size_t)b * M + j] : -1;
  __syncthreads();
  if (j >= M) return;
  for (int b = b0; b < B; b += step) {
    int from = parents[b];
    if (from < -1 || from >= B) {  // no such row: this one stays
      set_status(status, ATTN_DEV_BAD_PARENT);
      from = b;
    }
    const int was = old[(b << lc) + col];
    int now = from < 0 ? -1 : old[(from << lc) + col];
    if (lengths && (long long)j << lp >= lengths[b]) now = -1;
    if (now == was) continue;
    table[(size_t)b * M + j] = now;
    if (now >= 0 && now < P) atomicAdd(&refs[now], 1);
    if (was >= 0 && was < P) atomicSub(&refs[was], 1);
  }
}
// Without parents: only entries past the kept rows are looked at.  A warp for
// each row and 1024 columns.
__global__ void __launch_bounds__(256) pages_cut_kernel(int32_t* __restrict__ table,
                                                        int32_t* __restrict__ refs,
                                                        const int32_t* __restrict__ lengths, int B,
                                                        int M, int P, int lp) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int lane = threadIdx.x & 31, b = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (b >= B) return;
  const int first = (int)(((long long)max(lengths[b], 0) + (1 << lp) - 1) >> lp);
  const int j0 = blockIdx.x * 1024, j1 = min(j0 + 1024, M);
#pragma unroll 8
  for (int j = max(first, j0) + lane; j < j1; j += 32) {
    const int was = table[(size_t)b * M + j];
    if (was == -1) continue;
    table[(size_t)b * M + j] = -1;
    if (was >= 0 && was < P) atomicSub(&refs[was], 1);
  }
}

// ----------------------------------------------------------------- compact --

struct CompactParams {
  int32_t* table;
  int32_t* refs;
  int32_t* map;
  int* n_moves;
  int32_t* from;  // [P] used pages by how many come before them
  int32_t* to;    // [P] free pages by how many come before them
  int B, M, P;
};

// n pages are in use: the k-th of those at n or above goes to the k-th free
// page below n.
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kScanThreads, 1)
    pages_plan_kernel(const CompactParams p) {
  __shared__ int warps[kScanWarps], ctas[kCtas];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  grid_dependency_wait();
  grid_dependents_launch();
  const Span s = span_of(p.P, rank, warp);
  int count = 0;
#pragma unroll 4
  for (int i0 = s.lo; i0 < s.hi; i0 += 32) {
    const int i = i0 + lane;
    count += __popc(__ballot_sync(0xffffffffu, i < s.hi && p.refs[i] > 0));
  }
  int n;
  int at = cluster_prefix(cluster, true, count, warps, ctas, &n);
  for (int i0 = s.lo; i0 < s.hi; i0 += 32) {
    const int i = i0 + lane;
    const bool in = i < s.hi, used = in && p.refs[i] > 0;
    const uint32_t m = __ballot_sync(0xffffffffu, used);
    const int before = at + __popc(m & lanes_below(lane));  // used pages before i
    at += __popc(m);
    if (!in) continue;
    if (i == n) *p.n_moves = n - before;  // as many high pages as low holes
    if (used) {
      if (i >= n) p.from[before] = i;
      else p.map[i] = i;
    } else {
      if (i < n) p.to[i - before] = i;
      p.map[i] = -1;
    }
  }
  if (n == p.P && rank == 0 && tid == 0) *p.n_moves = 0;  // no page is free
  cluster.sync();
  const int moves = *(volatile int*)p.n_moves;
  for (int k = rank * kScanThreads + tid; k < moves; k += kCtas * kScanThreads) {
    const int src = p.from[n - moves + k], dst = p.to[k];
    p.map[src] = dst;
    p.refs[dst] = p.refs[src];
    p.refs[src] = 0;
    if (k == 0) p.n_moves[1] = n;
  }
}

// The moved pages' rows, a warp for each (move, operand, head), and the table.
__global__ void __launch_bounds__(kCopyThreads) pages_move_kernel(CompactParams p, PagedPool pool) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int moves = p.n_moves[0], n = p.n_moves[1];
  const int lane = threadIdx.x & 31;
  const long long thread = (long long)blockIdx.x * kCopyThreads + threadIdx.x;
  const long long threads = (long long)gridDim.x * kCopyThreads;
  const long long units = (long long)moves * 2 * pool.Hkv;
  for (long long u = thread >> 5; u < units; u += threads >> 5) {
    const int c = (int)(u / (2 * pool.Hkv)), oh = (int)(u - (long long)c * 2 * pool.Hkv);
    copy_rows(oh & 1 ? pool.v : pool.k, pool, oh >> 1, p.from[n - moves + c], p.to[c], pool.page,
              lane);
  }
  for (long long i = thread; i < (long long)p.B * p.M; i += threads) {
    const int e = p.table[i];
    if (e < 0 || e >= p.P) continue;
    const int now = p.map[e];
    if (now != e) p.table[i] = now;
  }
}

cudaError_t sm_count(int* sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

// [B] copies, [B] reaches, then info and list [B * per] each.
PagesWorkspace pages_reserve_layout(int B, int S, int page) {
  const size_t per = (size_t)(S - 1 + page - 1) / page + 1;
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
  p.n_copies = reinterpret_cast<int*>(base + 128);
  p.copies = reinterpret_cast<int4*>(base + ws.copies_off);
  p.reach = reinterpret_cast<int2*>(base + ws.copies_off + (size_t)B * 16);
  p.B = B;
  p.S = S;
  p.M = M;
  p.P = pool.P;
  p.lp = log2_of(pool.page);
  p.cap = M * pool.page;
  p.per = (S - 1 + pool.page - 1) / pool.page + 1;
  p.info = reinterpret_cast<int32_t*>(base + ws.list_off);
  p.list = p.info + (size_t)B * p.per;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e == cudaSuccess)
    e = launch_pdl(pages_reserve_kernel, dim3(kCtas), dim3(kScanThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  const long long warps = (long long)B * 2 * pool.Hkv;
  const long long blocks = (warps * 32 + kCopyThreads - 1) / kCopyThreads;
  return launch_pdl(pages_copy_rows_kernel, dim3((unsigned)min(blocks, (long long)sms * 8)),
                    dim3(kCopyThreads), 0, stream, pool, (const int*)p.n_copies,
                    (const int4*)p.copies);
}

cudaError_t launch_pages_fork(int32_t* table, int32_t* refs, const int32_t* parents,
                              const int32_t* lengths, int B, int M, int P, int page,
                              void* workspace, cudaStream_t stream) {
  if (!parents) {
    if (!lengths) return cudaSuccess;
    return launch_pdl(pages_cut_kernel, dim3((M + 1023) / 1024, (B + 7) / 8), dim3(256), 0, stream,
                      table, refs, lengths, B, M, P, log2_of(page));
  }
  // 128-byte pieces of rows; 32-byte ones where that many rows would not fit
  const int lc = B <= 1024 ? 5 : 3;
  const size_t smem = ((size_t)B << lc) * 4;
  cudaError_t e = cudaFuncSetAttribute(pages_fork_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
  if (e != cudaSuccess) return e;
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
  p.n_moves = reinterpret_cast<int*>(base + 128);
  p.from = reinterpret_cast<int32_t*>(base + ws.list_off);
  p.to = p.from + pool.P;
  p.B = B;
  p.M = M;
  p.P = pool.P;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e == cudaSuccess)
    e = launch_pdl(pages_plan_kernel, dim3(kCtas), dim3(kScanThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(pages_move_kernel, dim3(sms * 8), dim3(kCopyThreads), 0, stream, p, pool);
}

}  // namespace gqa
