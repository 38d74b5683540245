// kv8_cluster.cuh -- the 8-bit decode for few segments: one thread-block
// cluster of C CTAs per (sequence, KV head), merged through distributed shared
// memory.  Included by kv8_decode.cu, whose consumers, slices and pipeline it
// shares.
//
// Rank r takes tiles r, r + C, r + 2C, ...  Without a list its first tile is
// then tile r whatever the position, so its copy (and the query rows') goes
// out before the position has been read.  No scan, no global scratch, no
// atomics: the CTA's partial (max, sum, unnormalised o) of output column i
// goes straight into the shared memory of the rank that owns column i; after
// one cluster barrier each rank merges its columns from its own memory, in
// rank order, and writes them.  Against the split over a flat list this saves
// the merge's three round trips through L2 and the scan: B=1, 8 KV heads,
// 8001 rows, g=2: 10.5 -> 6.6 us (7.0 with probabilities in two parts).  (When
// it is taken: cluster_size8.)
#pragma once

namespace gqa {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxCluster = 16;

struct Landing {  // one column of 4 dims of one head, from one rank
  float4 o;
  float m, l;
  float pad[2];
};

__host__ __device__ constexpr int landing_cols(int g, int C) { return (g * (kD / 4) + C - 1) / C; }
inline size_t cluster_smem_bytes(int stages, int g, int C) {
  return (size_t)stages * (kStageBytes + kSlices * sizeof(SliceMeta) + 16) + 16 +
         (size_t)g * kD * 2 + (size_t)merge_floats(g) * 4 +
         (size_t)C * landing_cols(g, C) * sizeof(Landing) + kMiscInts * 4;
}

template <int NT, bool LIST>
__global__ void __launch_bounds__(kClusterThreads, 1)
    kv8_cluster_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const Kv8Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int NS = p.stages, g = p.g, L = p.L;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int cols = landing_cols(g, C);
  uint8_t* stages = smem;
  uint8_t* qbuf = smem + (size_t)NS * kStageBytes;                          // [g][kD] bf16
  SliceMeta* meta = reinterpret_cast<SliceMeta*>(qbuf + g * kD * 2);        // [NS][kSlices]
  Landing* land = reinterpret_cast<Landing*>(meta + NS * kSlices);          // [C][cols]
  float* merge_o = reinterpret_cast<float*>(land + C * cols);               // merge_row
  float* merge_ml = merge_o + kWarps * merge_heads(g) * kMergeRow;          // [warps][g][2]
  uint64_t* bars = reinterpret_cast<uint64_t*>(merge_ml + kWarps * g * 2);  // full, empty, sync
  int* misc = reinterpret_cast<int*>(bars + 2 * NS + 2);                    // [0] abort

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seg = blockIdx.x / C, b = seg / p.Hkv, kvh = seg % p.Hkv;
  volatile int* abort_flag = misc;
  const size_t out_at = ((size_t)b * p.Hq + (size_t)kvh * g) * kD;

  if (tid == kWarps * 32) {  // the thread that issues the copies
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(&bars[s]), 2);  // the copies issued; the scales in place
      mbar_init(smem_u32(&bars[NS + s]), kWarps);
    }
    mbar_init(smem_u32(&bars[2 * NS]), kWarps);
    misc[0] = 0;
    fence_mbar_init();
  }
  grid_dependency_wait();
  grid_dependents_launch();

  auto issue = [&](int s, int row) {  // one thread: both operands' whole tile
    const uint32_t full = smem_u32(&bars[s]);
    const uint32_t sK = smem_u32(stages + (size_t)s * kStageBytes);
    tma_load_3d(sK, &tm_k, 0, row, seg, full);
    tma_load_3d(sK + kOpBytes, &tm_v, 0, row, seg, full);
  };
  const uint32_t q_bytes = (uint32_t)g * kD * 2u;
  auto expect_first = [&](uint32_t bytes) {  // stage 0's arrival, with the query rows
    mbar_arrive_expect_tx(smem_u32(&bars[0]), q_bytes + bytes);
    bulk_load(smem_u32(qbuf), p.q + out_at, q_bytes, smem_u32(&bars[0]));
  };
  const bool skip0 = p.test_skip >= 0 && seg == 0 && rank == p.test_skip;  // failure-path tests
  const bool early = !LIST && rank * kTile < L && !skip0;
  if (early && tid == kWarps * 32) {
    expect_first(kStageBytes);
    issue(0, rank * kTile);
  }
  const int pos = p.positions[b];
  __syncthreads();  // barriers initialised
  if (!rows_in_cache(pos, 0, L)) {  // the same for the whole cluster
    if (rank == 0) {
      if (tid == 0) set_status(p.status, ATTN_DEV_BAD_POSITION);
      for (int i = tid; i < g * kD / 8; i += kClusterThreads)
        reinterpret_cast<uint4*>(p.out + out_at)[i] =
            make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
    }
    if (early && tid == kWarps * 32) {
      mbar_arrive(smem_u32(&bars[0]));  // for the scales; then the copies land before the exit
      mbar_wait(smem_u32(&bars[0]), 0u, abort_flag);
    }
    return;
  }
  // this CTA runs: the matching wait comes before any write into another's
  // shared memory, so that one is known to have started by then
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int nt = LIST ? (int)((((long long)p.count << p.lb) + kTile - 1) / kTile) : pos / kTile + 1;
  const int mine = rank < nt ? (nt - rank + C - 1) / C : 0;  // tiles rank + i*C

  if (warp >= kWarps) {
    // ----------------------------------------------------------- producers --
    const bool copies = warp == kWarps;
    const int ti = lane >> 3, slice = lane & 7;
    const int entry_rows = 1 << p.lb;
    const int in_block = (slice * 16) & (entry_rows - 1);
    const int entry = (slice * 16) >> p.lb, per_tile = kTile >> p.lb;
    auto fetch = [&](int i) -> int {  // the block slice `slice` of my tile i lies in
      const long long e = (long long)(rank + i * C) * per_tile + entry;
      return i < mine && e < p.count ? p.index[(size_t)seg * p.count + e] : -1;
    };
    auto row_of = [&](int i, int blk) -> int {
      if (i >= mine) return kNoRow;
      int row;
      if (LIST) {
        if (blk < -1 || blk >= p.nb) {
          if (copies) set_status(p.status, ATTN_DEV_BAD_BLOCK);
          blk = -1;
        }
        row = blk >= 0 ? (blk << p.lb) + in_block : kNoRow;
      } else {
        row = (rank + i * C) * kTile + slice * 16;
      }
      return row <= pos ? row : kNoRow;
    };
    int s = 0;
    uint32_t pass = 0;
    auto wait_empty = [&]() -> bool {
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
    auto skipped = [&](int i) {  // failure-path tests only
      return p.test_skip >= 0 && seg == 0 && rank + i * C == p.test_skip;
    };
    if (copies && !LIST) {
      for (int i = 0; i < mine; ++i) {
        if (!wait_empty()) break;
        const int row = (rank + i * C) * kTile;
        if (lane == 0 && !(i == 0 && early) && !skipped(i) && range_ok(row < L, p.status)) {
          if (i == 0) expect_first(kStageBytes);
          else mbar_arrive_expect_tx(smem_u32(&bars[s]), kStageBytes);
          issue(s, row);
        }
        __syncwarp();
        turn();
      }
      // a first copy that no consumer waits for lands before the CTA exits
      if (early && mine == 0 && lane == 0) {
        mbar_arrive(smem_u32(&bars[0]));
        mbar_wait(smem_u32(&bars[0]), 0u, abort_flag);
      }
    } else if (copies) {
      int blk = fetch(ti);
      bool ok = true;
      for (int base = 0; ok && base < mine; base += 4) {
        const int i = base + ti, row = row_of(i, blk);
        blk = fetch(i + 4);
        const bool have = row != kNoRow && in_block == 0 && !skipped(i) &&
                          range_ok(row >= 0 && row < L, p.status);
        const uint32_t boxes = __ballot_sync(0xffffffffu, have);
        for (int q = 0; q < 4 && base + q < mine; ++q) {
          if (!wait_empty()) {
            ok = false;
            break;
          }
          const uint32_t full = smem_u32(&bars[s]);
          if (lane == 8 * q && !skipped(i)) {
            const uint32_t bytes =
                __popc((boxes >> (8 * q)) & 0xffu) * (uint32_t)entry_rows * 2u * kD;
            if (i == 0) expect_first(bytes);
            else mbar_arrive_expect_tx(full, bytes);
          }
          __syncwarp();
          if (ti == q && have) {
            const uint32_t sK = smem_u32(stages + (size_t)s * kStageBytes) + slice * 16 * kD;
            tma_load_3d(sK, &tm_k, 0, row, seg, full);
            tma_load_3d(sK + kOpBytes, &tm_v, 0, row, seg, full);
          }
          turn();
        }
      }
    } else {
      auto look_up = [&](int i, int blk, int& row, float& ks, float& vs) {
        row = row_of(i, blk);
        ks = vs = 1.f;
        if (row != kNoRow && range_ok((row >> p.lb) < p.nb, p.status)) {
          const size_t at = (size_t)seg * p.nb + (row >> p.lb);
          ks = p.k_scale[at];
          vs = p.v_scale[at];
        }
      };
      int row;
      float ks, vs;
      look_up(ti, LIST ? fetch(ti) : 0, row, ks, vs);
      int blk = LIST ? fetch(ti + 4) : 0;
      bool ok = true;
      for (int base = 0; ok && base < mine; base += 4) {
        int row_next;
        float ks_next, vs_next;
        look_up(base + 4 + ti, blk, row_next, ks_next, vs_next);
        if (LIST) blk = fetch(base + 8 + ti);
        const SliceMeta mt = slice_meta(row == kNoRow ? 0 : min(16, pos + 1 - row), ks, vs);
        for (int q = 0; q < 4 && base + q < mine; ++q) {
          if (!wait_empty()) {
            ok = false;
            break;
          }
          if (ti == q) meta[s * kSlices + slice] = mt;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars[s]));
          turn();
        }
        row = row_next;
        ks = ks_next;
        vs = vs_next;
      }
    }
    __syncwarp();
  } else {
    // ----------------------------------------------------------- consumers --
    ConsumerSync csync{smem_u32(&bars[2 * NS]), abort_flag, p.status, 0u};
    Consumer8<NT> cs;
    cs.c = lane >> 2;
    cs.t = lane & 3;
    cs.reset();
    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < mine; ++i) {
      if (!consumer_wait(smem_u32(&bars[s]), ph, abort_flag, p.status, lane)) break;
      if (i == 0) cs.load_q(qbuf, g, p.qscale);
      const SliceMeta mt = meta[s * kSlices + warp];
      const uint8_t* Ks = stages + (size_t)s * kStageBytes + warp * 16 * kD;
      if (mt.rows > 0) cs.slice(Ks, Ks + kOpBytes, mt.rows, mt);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars[NS + s]));
      if (++s == NS) {
        s = 0;
        ph ^= 1u;
      }
    }
    cs.stash(merge_o, merge_ml, warp, g);
    csync(lane);
  }
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (tid < kConsumers) {
    for (int i = tid; i < g * (kD / 4); i += kConsumers) {
      Landing x;
      merge_warps8(merge_o, merge_ml, i, g, x.m, x.l, x.o);
      const int owner = i / cols;
      if (!range_ok(owner < C && rank < C, p.status)) continue;
      Landing* to = cluster.map_shared_rank(land, owner) + rank * cols + (i - owner * cols);
      to->o = x.o;
      *reinterpret_cast<float2*>(&to->m) = make_float2(x.m, x.l);
    }
  }
  cluster.sync();
  for (int j = tid; j < cols; j += kClusterThreads) {
    const int i = rank * cols + j;
    if (i >= g * (kD / 4)) break;
    float M = kMInit;
#pragma unroll 4
    for (int r = 0; r < C; ++r) M = fmaxf(M, land[r * cols + j].m);
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int r = 0; r < C; ++r) {
      const Landing& x = land[r * cols + j];
      const float e = ex2(x.m - M);
      l += moved(x.l, x.m - M);
      o.x = fmaf(x.o.x, e, o.x);
      o.y = fmaf(x.o.y, e, o.y);
      o.z = fmaf(x.o.z, e, o.z);
      o.w = fmaf(x.o.w, e, o.w);
    }
    store_column(p, out_at, i, o, l);
  }
  if (*abort_flag) {  // copies in flight land before the shared memory goes
    const uint64_t t_start = globaltimer_ns();
    while (globaltimer_ns() - t_start < 2000000ull) {
    }
  }
}

}  // namespace
}  // namespace gqa
