// paged_cluster.cuh -- the paged decode for few segments: one thread-block
// cluster of C CTAs per (sequence, KV head), merged through distributed shared
// memory.  Included by paged_decode.cuh, whose consumers and tiles it shares.
//
// Rank r takes tiles r, r + C, r + 2C, ...  Its first tile is then tile r
// whatever the position, so the tile's table entries are fetched beside the
// position, and its copies go out one round trip after the launch's start.  No
// scan, no global scratch, no atomics: each CTA's maxima and sums go to all
// ranks, its outputs to the rank that owns their columns, and after one cluster
// barrier each rank merges its columns, in rank order, and writes them.
#pragma once

namespace gqa {
namespace {

// Floats of the outputs that a rank owns.
__host__ __device__ constexpr int owned(int R, int D, int C) {
  return (R * (D / 4) + C - 1) / C * 4;
}
template <int D, int NT>
size_t cluster_smem_bytes(int stages, int R, int C) {
  using Sh = Shape<D, NT>;
  return (size_t)stages * (Sh::kStage + sizeof(TileMeta) + 16) + Sh::kQ + Sh::kFixed + 8 + 64 +
         (size_t)C * (owned(R, D, C) * 4 + R * 8) + 16;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    paged_cluster_kernel(const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const PagedParams p) {
  using Sh = Shape<D, NT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int NS = p.stages, R = p.R, own = owned(R, D, C);
  uint8_t* stages = smem;
  uint8_t* qbuf = stages + (size_t)NS * Sh::kStage;               // [NT * 8] query rows
  TileMeta* meta = reinterpret_cast<TileMeta*>(qbuf + Sh::kQ);
  uint8_t* weights = reinterpret_cast<uint8_t*>(meta + NS);
  float* osum = reinterpret_cast<float*>(weights + 2 * Sh::kP);
  float* wmax = osum + Sh::kO / 4;
  float* lsum = wmax + 2 * NT * 64;
  float* land = lsum + NT * 64;                                   // [C][own]
  float2* land_ml = reinterpret_cast<float2*>(land + C * own);    // [C][R]
  uint64_t* bars = reinterpret_cast<uint64_t*>(land_ml + C * R);  // full [NS], empty [NS], sync
  int* misc = reinterpret_cast<int*>(bars + 2 * NS + 1);          // [0] abort

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seg = blockIdx.x / C, b = seg / p.Hkv, kvh = seg % p.Hkv;
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
  for (int i = tid; i < Sh::kQ / 16; i += kThreads)  // rows past R stay zero
    reinterpret_cast<uint4*>(qbuf)[i] = make_uint4(0u, 0u, 0u, 0u);
  // (they come before the query copies that land over them)
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  grid_dependency_wait();
  grid_dependents_launch();

  // the producer's first table entries, beside the position
  const int ti = lane >> 3, slice = lane & 7;
  auto entry = [&](int i) -> int {  // of slice `slice` of my tile i, whatever is in use
    const long long e = ((long long)(rank + (long long)i * C) * kTile + slice * 16) >> p.lp;
    return e < p.M ? p.table[(size_t)b * p.M + e] : -1;
  };
  int page = warp == kWarps ? entry(ti) : -1;
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

  ConsumerSync csync{smem_u32(&bars[2 * NS]), abort_flag, p.status, 0u};
  PagedConsumer<D, NT> cs;
  if (warp == kWarps) {
    // ------------------------------------------------------------ producer --
    const int page_rows = 1 << p.lp, in_page = (slice * 16) & (page_rows - 1);
    auto in_use = [&](int i, int page) -> int {
      if (i >= mine || (rank + i * C) * kTile + slice * 16 > pos + n - 1) return -1;
      return page_ok(p, page);
    };
    int s = 0;
    uint32_t pass = 0;
    bool ok = true;
    for (int base = 0; ok && base < mine; base += 4) {
      const int i = base + ti;
      const int cur = in_use(i, page);
      if (i + 4 < mine) page = entry(i + 4);
      const uint32_t there = __ballot_sync(0xffffffffu, cur >= 0);
      const bool lead = cur >= 0 && in_page == 0;
      const uint32_t boxes = __ballot_sync(0xffffffffu, lead);
      for (int q = 0; q < 4 && base + q < mine; ++q) {
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
          meta[s] = TileMeta{(int)((there >> (8 * q)) & 0xffu) | (first ? kStarts : 0), k * kTile,
                             pos, n, b, kvh, 0, 1};
          if (!skip)
            mbar_arrive_expect_tx(full, __popc((boxes >> (8 * q)) & 0xffu) *
                                                ((uint32_t)page_rows * D * 4u) +
                                            (first ? (uint32_t)R * D * 2u : 0u));
        }
        __syncwarp();
        if (ti == q && lead && !skip) {
          const uint32_t dst = smem_u32(stages + (size_t)s * Sh::kStage) + slice * 16 * D * 2;
          tma_load_5d(dst, &tm_k, 0, 0, 0, kvh, cur, full);
          tma_load_5d(dst + Sh::kOp, &tm_v, 0, 0, 0, kvh, cur, full);
        }
        if (first && !skip && lane < R)
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
    const TileMeta none{0, 0, pos, n, b, kvh, 0, 1};
    cs.start(p, none);
    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < mine; ++i) {
      if (!consumer_wait(smem_u32(&bars[s]), ph, abort_flag, p.status, lane)) break;
      const TileMeta mt = meta[s];
      if (i == 0) cs.load_q(qbuf);
      cs.tile(stages + (size_t)s * Sh::kStage, p, mt);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars[NS + s]));
      if (++s == NS) {
        s = 0;
        ph ^= 1u;
      }
    }
    cs.finish();
  }
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (warp < kWarps) {
    cs.each_output([&](int, int r, int d, float2 y) {
      if (r >= R) return;
      const int at = r * D + d, owner = at / own;
      if (!range_ok(owner < C && rank < C, p.status)) return;
      *reinterpret_cast<float2*>(cluster.map_shared_rank(land, owner) + rank * own +
                                 (at - owner * own)) = y;
    });
    // maxima and sums: warp w tells ranks w, w + 8; lane (c, t = i) row 8i + c
    for (int to = warp; to < C; to += kWarps) {
      float2* ml = cluster.map_shared_rank(land_ml, to) + rank * R;
#pragma unroll
      for (int i = 0; i < NT; ++i)
        if (cs.t == i && 8 * i + cs.c < R) ml[8 * i + cs.c] = make_float2(cs.ref[i], cs.l[i]);
    }
  }
  cluster.sync();
  for (int j = tid * 4; j < own; j += kThreads * 4) {
    const int at = rank * own + j;
    if (at >= R * D) break;
    const int r = at / D;
    float M = kMInit;
#pragma unroll 4
    for (int k = 0; k < C; ++k) M = fmaxf(M, land_ml[k * R + r].x);
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < C; ++k) {
      const float2 ml = land_ml[k * R + r];
      const float4 x = *reinterpret_cast<const float4*>(land + k * own + j);
      const float e = ex2(ml.x - M);
      l = fmaf(ml.y, e, l);
      o.x = fmaf(x.x, e, o.x);
      o.y = fmaf(x.y, e, o.y);
      o.z = fmaf(x.z, e, o.z);
      o.w = fmaf(x.w, e, o.w);
    }
    store4<D>(p, b, kvh, r, at - r * D, o, l, r / p.g >= n);
  }
  if (*abort_flag) {  // copies in flight land before the shared memory goes
    const uint64_t t_start = globaltimer_ns();
    while (globaltimer_ns() - t_start < 2000000ull) {
    }
  }
}

}  // namespace
}  // namespace gqa
