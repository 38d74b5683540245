// paged.h -- the paged cache's pools and the decode's launch parameters, shared
// by the kernels and the host code.
#pragma once

#include <cuda.h>

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace gqa {

// k and v hold P pages [Hkv][page][D] of bf16, alike: element (p, h, r, d) at
// p * page_stride + h * head_stride + r * row_stride + d.
struct PagedPool {
  uint8_t* k;
  uint8_t* v;
  long long page_stride, head_stride, row_stride;  // elements
  int P, Hkv, page, D;
};

constexpr int kPagedMaxB = 4096;     // sequences per decode launch
constexpr int kPagedMaxRows = 32;    // query rows (new tokens x heads) per KV head
constexpr int kPagedMaxGrid = 192;   // CTAs of the decode (workspace partial slots)

struct PagedParams {
  const uint16_t* q;
  const int32_t* positions;
  const int32_t* lengths;  // new tokens of each sequence, or null: S
  const int32_t* table;    // [B, M]
  uint16_t* out;
  uint32_t* status;
  uint32_t* counters;
  float* part_ml;          // [slots][R][2]
  float* part_o;           // [slots][R][D]
  const uint16_t* k;       // the pool, for copies that need no tensor map
  const uint16_t* v;
  long long page_stride, head_stride, row_stride;
  int B, S, Hq, Hkv, g, P, M;
  int R;                   // S * g
  int g_inverse;           // 2^16 / g, rounded up
  int lp;                  // log2 of the page's rows
  int cap;                 // rows that a sequence's pages can hold
  int stages;
  int test_skip;
  float qscale;            // |scale| * log2(e), above zero
  uint32_t flip;           // sign bits of two bf16 if scale is negative, else 0
};

// Makes the pool's tensor maps, for copies of a head's rows of a page.
bool paged_maps(const PagedPool& pool, CUtensorMap* mk, CUtensorMap* mv);
// (a page has 16, 32, 64 or 128 rows)
inline int log2_of(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }
// For head dims 64 and 128, one new token or several (paged_decode_d*.cu).
cudaError_t launch_paged_decode_64(PagedParams& p, const PagedPool& pool, cudaStream_t stream);
cudaError_t launch_paged_decode_64_drafts(PagedParams& p, const PagedPool& pool,
                                          cudaStream_t stream);
cudaError_t launch_paged_decode_128(PagedParams& p, const PagedPool& pool, cudaStream_t stream);
cudaError_t launch_paged_decode_128_drafts(PagedParams& p, const PagedPool& pool,
                                           cudaStream_t stream);

struct PagedWorkspace {
  size_t counters_off, ml_off, o_off, total;  // the status word comes first
};
PagedWorkspace paged_workspace_layout(int B, int S, int Hq, int Hkv, int D);
cudaError_t launch_paged_decode(const void* q, const int32_t* positions, const int32_t* lengths,
                                const int32_t* table, const PagedPool& pool, int B, int S, int Hq,
                                int M, float scale, void* out, void* workspace,
                                cudaStream_t stream);
cudaError_t launch_paged_append(const void* k_new, const void* v_new, long long k_stride,
                                long long v_stride, const int32_t* positions,
                                const int32_t* lengths, const int32_t* table,
                                const PagedPool& pool, int B, int S, int M, cudaStream_t stream);

// Pages: given out, shared and freed, moved (pages.cu).
// The pages that S >= 1 rows in a row can touch; S may be any int.
constexpr long long pages_touched(int S, int page) { return (S - 1ll + page - 1) / page + 1; }
struct PagesWorkspace {
  size_t copies_off, list_off, total;  // the status word comes first
};
PagesWorkspace pages_reserve_layout(int B, int S, int page);
PagesWorkspace pages_compact_layout(int P);
cudaError_t launch_pages_reserve(int32_t* table, int32_t* refs, const int32_t* positions,
                                 const int32_t* lengths, const PagedPool& pool, int B, int S, int M,
                                 int32_t* taken, void* workspace, cudaStream_t stream);
cudaError_t launch_pages_fork(int32_t* table, int32_t* refs, const int32_t* parents,
                              const int32_t* lengths, int B, int M, int P, int page,
                              void* workspace, cudaStream_t stream);
cudaError_t launch_pages_compact(int32_t* table, int32_t* refs, const PagedPool& pool, int B,
                                 int M, int32_t* page_map, void* workspace, cudaStream_t stream);
// Debug builds: accesses a range check skipped since the last call; 0 in others.
cudaError_t paged_append_read_skips(uint32_t* count);

}  // namespace gqa
