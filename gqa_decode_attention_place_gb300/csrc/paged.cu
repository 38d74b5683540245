// paged.cu -- the paged cache's append, and the host side of its decode: the
// workspace, the tensor maps of a pool and the choice of the head dim.
#include "common.cuh"
#include "decode_params.h"
#include "internal.h"
#include "paged.h"
#include "tcgen05.cuh"

#include <cmath>

namespace gqa {

__device__ unsigned int g_paged_append_skips;  // debug builds

// Rows k_new, v_new [B, S, Hkv, D] into the pages that hold rows positions[b] + t:
// a bit-exact copy in 16-byte vectors, bound by memory.  A warp takes a token's
// heads, so the position and the table entry are looked up once for all of them,
// and has up to eight vectors under way a lane (K and V of four passes).
constexpr int kAppendWarps = 4;
__global__ void __launch_bounds__(kAppendWarps * 32) paged_append_kernel(
    const uint4* __restrict__ k_new, const uint4* __restrict__ v_new, long long k_stride,
    long long v_stride, const int32_t* __restrict__ positions,
    const int32_t* __restrict__ lengths, const int32_t* __restrict__ table, PagedPool pool,
    int B, int S, int M, int lp, int tokens_per_warp) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int lane = threadIdx.x & 31;
  const int lv = pool.D == 128 ? 4 : 3;  // log2 of a row's vectors
  const int vecs = pool.Hkv << lv;       // of a token
  const int page = 1 << lp;
  const long long cap = min((long long)M << lp, (long long)0x7fffffff);
  long long at = ((long long)blockIdx.x * kAppendWarps + (threadIdx.x >> 5)) * tokens_per_warp;
  for (int i = 0; i < tokens_per_warp && at < (long long)B * S; ++i, ++at) {
    const int b = (int)(at / S), t = (int)(at - (long long)b * S);
    const int n = lengths ? lengths[b] : S, pos = positions[b];
    // a sequence whose rows do not fit is skipped; the decode reports it
    if (t >= n || n > S || n > cap || !rows_in_cache(pos, n - 1, (int)cap)) continue;
    const int row = pos + t;
    if (!range_ok_count((row >> lp) < M, &g_paged_append_skips)) continue;
    const int pg = table[(size_t)b * M + (row >> lp)];
    if (pg < 0 || pg >= pool.P) continue;  // no such page: reported likewise
    const size_t base = (size_t)pg * (pool.page_stride >> 3) +
                        (size_t)(row & (page - 1)) * (pool.row_stride >> 3);
    const uint4* ks = k_new + at * (k_stride >> 3);
    const uint4* vs = v_new + at * (v_stride >> 3);
    uint4* kd = reinterpret_cast<uint4*>(pool.k) + base;
    uint4* vd = reinterpret_cast<uint4*>(pool.v) + base;
    for (int j0 = lane; j0 < vecs; j0 += 128) {
      uint4 x[4], y[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (j0 + 32 * u < vecs) {
          x[u] = ks[j0 + 32 * u];
          y[u] = vs[j0 + 32 * u];
        }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (j0 + 32 * u < vecs) {
          const int j = j0 + 32 * u, h = j >> lv, c = j & ((1 << lv) - 1);
          const size_t to = (size_t)h * (pool.head_stride >> 3) + c;
          kd[to] = x[u];
          vd[to] = y[u];
        }
    }
  }
}

cudaError_t launch_paged_append(const void* k_new, const void* v_new, long long k_stride,
                                long long v_stride, const int32_t* positions,
                                const int32_t* lengths, const int32_t* table,
                                const PagedPool& pool, int B, int S, int M, cudaStream_t stream) {
  const long long tokens = (long long)B * S;
  const int per = (int)((tokens + (1ll << 24) - 1) >> 24);  // more than 2^24 tokens: several a warp
  const long long warps = (tokens + per - 1) / per;
  return launch_pdl(paged_append_kernel, dim3((unsigned)((warps + kAppendWarps - 1) / kAppendWarps)),
                    dim3(kAppendWarps * 32), 0, stream, static_cast<const uint4*>(k_new),
                    static_cast<const uint4*>(v_new), k_stride, v_stride, positions, lengths,
                    table, pool, B, S, M, log2_of(pool.page), per);
}

PagedWorkspace paged_workspace_layout(int B, int S, int Hq, int Hkv, int D) {
  auto align256 = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t R = (size_t)S * (Hq / Hkv), slots = 2 * kPagedMaxGrid;
  PagedWorkspace w;
  w.counters_off = 256;
  w.ml_off = align256(w.counters_off + (size_t)B * Hkv * sizeof(uint32_t));
  w.o_off = align256(w.ml_off + slots * R * 2 * sizeof(float));
  w.total = align256(w.o_off + slots * R * D * sizeof(float));
  return w;
}

// A pool as a 5-D tensor map (64 dims, rows, halves of a row, heads, pages); a
// box is a page's rows of one head, [half][row][64 dims] in shared memory with the
// 128-byte swizzle.
static bool pool_map(CUtensorMap* m, const void* ptr, const PagedPool& pool) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t half = 64 * 2;
  cuuint64_t dims[5] = {64, (cuuint64_t)pool.page, (cuuint64_t)(pool.D / 64),
                        (cuuint64_t)pool.Hkv, (cuuint64_t)pool.P};
  cuuint64_t strides[4] = {(cuuint64_t)pool.row_stride * 2, half,
                           (cuuint64_t)pool.head_stride * 2, (cuuint64_t)pool.page_stride * 2};
  cuuint32_t box[5] = {64, (cuuint32_t)pool.page, (cuuint32_t)(pool.D / 64), 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(ptr), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

bool paged_maps(const PagedPool& pool, CUtensorMap* mk, CUtensorMap* mv) {
  return pool_map(mk, pool.k, pool) && pool_map(mv, pool.v, pool);
}

cudaError_t launch_paged_decode(const void* q, const int32_t* positions, const int32_t* lengths,
                                const int32_t* table, const PagedPool& pool, int B, int S, int Hq,
                                int M, float scale, void* out, void* workspace,
                                cudaStream_t stream) {
  const PagedWorkspace ws = paged_workspace_layout(B, S, Hq, pool.Hkv, pool.D);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  PagedParams p;
  p.q = static_cast<const uint16_t*>(q);
  p.positions = positions;
  p.lengths = lengths;
  p.table = table;
  p.out = static_cast<uint16_t*>(out);
  p.status = reinterpret_cast<uint32_t*>(base);
  p.counters = reinterpret_cast<uint32_t*>(base + ws.counters_off);
  p.part_ml = reinterpret_cast<float*>(base + ws.ml_off);
  p.part_o = reinterpret_cast<float*>(base + ws.o_off);
  p.k = reinterpret_cast<const uint16_t*>(pool.k);
  p.v = reinterpret_cast<const uint16_t*>(pool.v);
  p.page_stride = pool.page_stride;
  p.head_stride = pool.head_stride;
  p.row_stride = pool.row_stride;
  p.B = B;
  p.S = S;
  p.Hq = Hq;
  p.Hkv = pool.Hkv;
  p.g = Hq / pool.Hkv;
  p.P = pool.P;
  p.M = M;
  p.R = S * p.g;
  p.g_inverse = (65536 + p.g - 1) / p.g;
  p.lp = log2_of(pool.page);
  p.cap = M * pool.page;
  p.stages = 0;
  p.test_skip = g_decode_test_skip;
  // (a scale of zero: tiny, so that masked scores stay -inf times it; NaN stays NaN, where
  // fmaxf would take the other operand)
  p.qscale = std::isnan(scale) ? scale : fmaxf(fabsf(scale) * 1.4426950408889634f, 1e-37f);
  p.flip = scale < 0.f ? 0x80008000u : 0u;
  if (pool.D == 64)
    return S == 1 ? launch_paged_decode_64(p, pool, stream)
                  : launch_paged_decode_64_drafts(p, pool, stream);
  return S == 1 ? launch_paged_decode_128(p, pool, stream)
                : launch_paged_decode_128_drafts(p, pool, stream);
}

cudaError_t paged_append_read_skips(uint32_t* count) {
  return read_and_clear(g_paged_append_skips, count);
}

}  // namespace gqa
