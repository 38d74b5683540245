// paged_cluster.cuh -- the paged decode for few segments: one thread-block
// cluster of C CTAs per (sequence, KV head), merged through distributed shared
// memory.  Included by paged_decode.cuh, whose consumers and tiles it shares.
//
// Rank r takes tiles r, r + C, r + 2C, ...  Its first tile is then tile r
// whatever the position, so the tile's table entries are fetched beside the
// position, and its copies go out one round trip after the launch's start.  No
// scan, no global scratch, no atomics: each CTA's merged column goes straight
// into the shared memory of the rank that owns it, and after one cluster barrier
// each rank merges its columns, in rank order, and writes them.
#pragma once

namespace gqa {
namespace {

struct Landing {  // one column of 4 dims of a query row, from one rank
  float4 o;
  float m, l;
  float pad[2];
};
__host__ __device__ constexpr int landing_cols(int R, int D, int C) {
  return (R * (D / 4) + C - 1) / C;
}
template <int D, int NT>
size_t cluster_smem_bytes(int stages, int R, int C) {
  using Sh = Shape<D, NT>;
  return (size_t)stages * (Sh::kStage + sizeof(TileMeta) + 16) + Sh::kQ + Sh::kMl + 8 + 64 +
         (size_t)C * landing_cols(R, D, C) * sizeof(Landing) + 16;
}

template <int D, int NT, bool DRAFTS>
__global__ void __launch_bounds__(kClusterThreads, 1)
    paged_cluster_kernel(const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const PagedParams p) {
  using Sh = Shape<D, NT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int NS = p.stages, R = p.R, cols = landing_cols(R, D, C);
  uint8_t* stages = smem;
  uint8_t* qbuf = stages + (size_t)NS * Sh::kStage;               // [NT * 8] query rows
  TileMeta* meta = reinterpret_cast<TileMeta*>(qbuf + Sh::kQ);
  Landing* land = reinterpret_cast<Landing*>(meta + NS);          // [C][cols]
  float2* ml = reinterpret_cast<float2*>(land + C * cols);        // [query rows][warps]
  uint64_t* bars = reinterpret_cast<uint64_t*>(ml + Sh::kMl / 8);  // full [NS], empty [NS], sync
  int* misc = reinterpret_cast<int*>(bars + 2 * NS + 1);          // [0] abort

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seg = blockIdx.x / C, b = seg / p.Hkv, kvh = seg % p.Hkv;
  volatile int* abort_flag = misc;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(&bars[s]), 2);  // keys, values
      mbar_init(smem_u32(&bars[NS + s]), kWarps);
    }
    mbar_init(smem_u32(&bars[2 * NS]), kWarps);
    misc[0] = 0;
    fence_mbar_init();
  }
  prefetch_maps(tm_k, tm_v, warp, lane);
  for (int i = tid; i < Sh::kQ / 16; i += kClusterThreads)  // rows past R stay zero
    reinterpret_cast<uint4*>(qbuf)[i] = make_uint4(0u, 0u, 0u, 0u);
  // (they come before the query copies that land over them)
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  grid_dependency_wait();
  grid_dependents_launch();

  // the producer's first table entries, beside the position
  constexpr int kTile = Sh::kTile, kSlices = Sh::kSlices, kBatch = Sh::kBatch;
  constexpr uint32_t kAll = (1u << kSlices) - 1u;
  const int ti = lane / kSlices, slice = lane % kSlices;
  auto entry = [&](int i) -> int {  // of slice `slice` of my tile i, whatever is in use
    const long long e = ((long long)(rank + (long long)i * C) * kTile + slice * 16) >> p.lp;
    return e < p.M ? p.table[(size_t)b * p.M + e] : -1;
  };
  int page = warp >= kWarps ? entry(ti) : -1;
  int pos, n;
  const int kind = sequence(p, b, pos, n);
  if (kind != 2) {  // the same for the whole cluster, and for the sequence's other heads
    if (rank == 0 && kvh == 0) fill_rows<D>(p, b, tid);
    return;
  }
  // this CTA runs: the matching wait comes before any write into another's
  // shared memory, so that one is known to have started by then
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int nt = (pos + n - 1) / kTile + 1;
  const int mine = rank < nt ? (nt - rank + C - 1) / C : 0;  // tiles rank + i*C

  if (warp >= kWarps) {
    // ----------------------------------------------------------- producers --
    const bool keys = warp == kWarps;
    const int page_rows = 1 << p.lp, in_page = (slice * 16) & (page_rows - 1);
    auto in_use = [&](int i, int page) -> int {
      if (i >= mine || (rank + i * C) * kTile + slice * 16 > pos + n - 1) return -1;
      return page_ok(p, page);
    };
    int s = 0;
    uint32_t pass = 0;
    bool ok = true;
    for (int base = 0; ok && base < mine; base += kBatch) {
      const int i = base + ti;
      const int cur = in_use(i, page);
      if (i + kBatch < mine) page = entry(i + kBatch);
      const uint32_t there = __ballot_sync(0xffffffffu, cur >= 0);
      const bool lead = cur >= 0 && in_page == 0;
      const uint32_t copies = __ballot_sync(0xffffffffu, lead);
      for (int q = 0; q < kBatch && base + q < mine; ++q) {
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
        const int k = rank + (base + q) * C;
        const bool first = base + q == 0;
        const bool skip = p.test_skip >= 0 && seg == 0 && k == p.test_skip;  // tests only
        if (lane == 0) {
          if (keys)
            meta[s] = TileMeta{(int)((there >> (kSlices * q)) & kAll), k * kTile, pos, n, b, kvh, 0, 1};
          if (!skip)
            mbar_arrive_expect_tx(full, __popc((copies >> (kSlices * q)) & kAll) *
                                                ((uint32_t)page_rows * D * 2u) +
                                            (keys && first ? (uint32_t)R * D * 2u : 0u));
        }
        __syncwarp();
        if (ti == q && lead && !skip) {
          const uint32_t dst = smem_u32(stages + (size_t)s * Sh::kStage) + slice * 16 * D * 2;
          tma_load_5d(dst + (keys ? 0 : Sh::kOp), keys ? &tm_k : &tm_v, 0, 0, 0, kvh, cur,
                      full);
        }
        if (first && !skip && keys && lane < R)
          bulk_load(smem_u32(qbuf) + lane * Sh::kQStride,
                    p.q + query_row(p, b, kvh, lane) * D, D * 2, full);
        if (++s == NS) {
          s = 0;
          ++pass;
        }
      }
    }
    __syncwarp();
  } else {
    // ----------------------------------------------------------- consumers --
    ConsumerSync csync{smem_u32(&bars[2 * NS]), abort_flag, p.status, 0u};
    PagedConsumer<D, NT, DRAFTS> cs;
    cs.init(warp, lane);
    cs.start(p, pos, n);
    int s = 0, last = 0;  // last: the stage of the last tile
    uint32_t ph = 0;
    for (int i = 0; i < mine; ++i) {
      last = s;
      if (!consumer_wait(smem_u32(&bars[s]), ph, abort_flag, p.status, lane)) break;
      if (i == 0) cs.load_q(qbuf, p.flip);
      cs.tile(stages + (size_t)s * Sh::kStage, p, meta[s]);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars[NS + s]));
      if (++s == NS) {
        s = 0;
        ph ^= 1u;
      }
    }
    // every other CTA of the cluster has started; each column goes to its owner
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    uint8_t* tile = stages + (size_t)last * Sh::kStage;
    cs.stash(p, tile, ml, csync);
    csync(lane);
    cs.merge(p, tile, ml, tid, kConsumers, [&](int r, int d, float m, float l, const float4& o) {
      const int at = r * (D / 4) + d / 4, owner = at / cols;
      if (!range_ok(owner < C && rank < C, p.status)) return;
      Landing* to = cluster.map_shared_rank(land, owner) + rank * cols + (at - owner * cols);
      to->o = o;
      *reinterpret_cast<float2*>(&to->m) = make_float2(m, l);
    });
  }
  if (warp >= kWarps) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  cluster.sync();
  for (int j = tid; j < cols; j += kClusterThreads) {
    const int at = rank * cols + j;
    if (at >= R * (D / 4)) break;
    float M = kMInit;
#pragma unroll 4
    for (int k = 0; k < C; ++k) M = fmaxf(M, land[k * cols + j].m);
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < C; ++k) {
      const Landing& x = land[k * cols + j];
      const float e = ex2(x.m - M);
      l = fmaf(x.l, e, l);
      o.x = fmaf(x.o.x, e, o.x);
      o.y = fmaf(x.o.y, e, o.y);
      o.z = fmaf(x.o.z, e, o.z);
      o.w = fmaf(x.o.w, e, o.w);
    }
    const int r = at / (D / 4);
    store4<D>(p, b, kvh, r, (at - r * (D / 4)) * 4, o, l, token_of(p, r) >= n);
  }
  if (*abort_flag) {  // copies in flight land before the shared memory goes
    const uint64_t t_start = globaltimer_ns();
    while (globaltimer_ns() - t_start < 2000000ull) {
    }
  }
}

}  // namespace
}  // namespace gqa
