// capi.cu -- the extern "C" entry points declared in include/gqa_attn.h:
// argument validation on the host, then one launch on the caller's stream.
#include <cstdint>

#include "gqa_attn.h"
#include "decode_params.h"
#include "internal.h"

namespace gqa {
bool decode_supported(int B, int Hq, int Hkv, int L, int D);
bool prefill_supported(int Hq, int Hkv, int d);
}  // namespace gqa

namespace {

thread_local int g_last_cuda_error = 0;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return ATTN_OK;
  g_last_cuda_error = static_cast<int>(e);
  return ATTN_ERR_CUDA;
}

}  // namespace

extern "C" {

int attn_kv_append(const void* k_new, const void* v_new, const int32_t* positions,
                   void* k_cache, void* v_cache, int B, int Hkv, int L, int D,
                   cudaStream_t stream) {
  if (!k_new || !v_new || !positions || !k_cache || !v_cache) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Hkv <= 0 || L <= 0 || D <= 0) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(positions) & 3u))
    return ATTN_ERR_INVALID_ARG;
  if (D % 8 != 0 || D > 256) return ATTN_ERR_UNSUPPORTED;
  return cuda_status(
      gqa::launch_kv_append(k_new, v_new, positions, k_cache, v_cache, B, Hkv, L, D, stream));
}

size_t attn_decode_workspace_size(int B, int Hq, int Hkv, int L, int D) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || L <= 0 || D <= 0 || Hq % Hkv != 0) return 0;
  if (!gqa::decode_supported(B, Hq, Hkv, L, D)) return 0;
  return gqa::decode_workspace_layout(B, Hq, Hkv, D).total;
}

int attn_decode_step(const void* q, const int32_t* positions, const void* k_cache,
                     const void* v_cache, int B, int Hq, int Hkv, int L, int D, float scale,
                     void* out, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!q || !positions || !k_cache || !v_cache || !out) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || L <= 0 || D <= 0 || Hq % Hkv != 0)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(positions) & 3u))
    return ATTN_ERR_INVALID_ARG;
  if (!gqa::decode_supported(B, Hq, Hkv, L, D)) return ATTN_ERR_UNSUPPORTED;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < gqa::decode_workspace_layout(B, Hq, Hkv, D).total)
    return ATTN_ERR_WORKSPACE;
  return cuda_status(gqa::launch_decode(q, nullptr, nullptr, nullptr, nullptr, false, positions,
                                        nullptr, k_cache, v_cache, B, Hq, Hkv, L, D, 0, scale, out,
                                        workspace, stream));
}

namespace {

int decode_append(const void* q, const void* k_new, const void* v_new, const float* rope_cos,
                  const float* rope_sin, bool rope_by_pos, const int32_t* positions,
                  int32_t* advance, void* k_cache, void* v_cache, int B, int Hq, int Hkv, int L,
                  int D, float scale, void* out, void* workspace, size_t workspace_bytes,
                  cudaStream_t stream, int window = 0) {
  if (!q || !positions || !k_cache || !v_cache || !out || !k_new != !v_new)
    return ATTN_ERR_INVALID_ARG;
  if (!k_new && (rope_cos || advance)) return ATTN_ERR_INVALID_ARG;
  if (window < 0) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || L <= 0 || D <= 0 || Hq % Hkv != 0)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || (k_new && (!aligned16(k_new) || !aligned16(v_new))) ||
      !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(positions) & 3u))
    return ATTN_ERR_INVALID_ARG;
  if (!gqa::decode_supported(B, Hq, Hkv, L, D)) return ATTN_ERR_UNSUPPORTED;
  // the rotated query takes two operand rows per head (bf16 high and low
  // parts) in the tensor-core kernels' 16 rows: g <= 8 with the rotation
  if (rope_cos && Hq / Hkv > 8) return ATTN_ERR_UNSUPPORTED;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < gqa::decode_workspace_layout(B, Hq, Hkv, D).total)
    return ATTN_ERR_WORKSPACE;
  return cuda_status(gqa::launch_decode(q, k_new, v_new, rope_cos, rope_sin, rope_by_pos,
                                        positions, advance, k_cache, v_cache, B, Hq, Hkv, L, D,
                                        window, scale, out, workspace, stream));
}

}  // namespace

int attn_decode_step_append(const void* q, const void* k_new, const void* v_new,
                            const int32_t* positions, void* k_cache, void* v_cache, int B,
                            int Hq, int Hkv, int L, int D, float scale, void* out,
                            void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!k_new || !v_new) return ATTN_ERR_INVALID_ARG;
  return decode_append(q, k_new, v_new, nullptr, nullptr, false, positions, nullptr, k_cache,
                       v_cache, B, Hq, Hkv, L, D, scale, out, workspace, workspace_bytes, stream);
}

int attn_decode_step_rope_append(const void* q, const void* k_new, const void* v_new,
                                 const float* cos, const float* sin, const int32_t* positions,
                                 void* k_cache, void* v_cache, int B, int Hq, int Hkv, int L,
                                 int D, float scale, void* out, void* workspace,
                                 size_t workspace_bytes, cudaStream_t stream) {
  if (!k_new || !v_new) return ATTN_ERR_INVALID_ARG;
  if (!cos || !sin || !aligned16(cos) || !aligned16(sin)) return ATTN_ERR_INVALID_ARG;
  return decode_append(q, k_new, v_new, cos, sin, false, positions, nullptr, k_cache, v_cache, B,
                       Hq, Hkv, L, D, scale, out, workspace, workspace_bytes, stream);
}

int attn_decode_step_window(const void* q, const void* k_new, const void* v_new,
                            const int32_t* positions, void* k_cache, void* v_cache, int B, int Hq,
                            int Hkv, int L, int D, int window, float scale, void* out,
                            void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (window <= 0) return ATTN_ERR_INVALID_ARG;
  return decode_append(q, k_new, v_new, nullptr, nullptr, false, positions, nullptr, k_cache,
                       v_cache, B, Hq, Hkv, L, D, scale, out, workspace, workspace_bytes, stream,
                       window);
}

int attn_decode_multi(const void* q, const void* k_new, const void* v_new,
                      const int32_t* positions, void* k_cache, void* v_cache, int B, int S,
                      int Hq, int Hkv, int L, int D, float scale, void* out, void* workspace,
                      size_t workspace_bytes, cudaStream_t stream) {
  if (!q || !positions || !k_cache || !v_cache || !out || !k_new != !v_new)
    return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || S <= 0 || Hq <= 0 || Hkv <= 0 || L <= 0 || D <= 0 || Hq % Hkv != 0)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || (k_new && (!aligned16(k_new) || !aligned16(v_new))) ||
      !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(positions) & 3u))
    return ATTN_ERR_INVALID_ARG;
  if ((long long)S * Hq > 65536 || !gqa::decode_supported(B, S * Hq, Hkv, L, D))
    return ATTN_ERR_UNSUPPORTED;  // S * g must be 1, 2, 4, 8 or 16
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < gqa::decode_workspace_layout(B, S * Hq, Hkv, D).total)
    return ATTN_ERR_WORKSPACE;
  if (k_new) {
    const int st = cuda_status(gqa::launch_kv_append(k_new, v_new, positions, k_cache, v_cache, B,
                                                     Hkv, L, D, stream, S));
    if (st != ATTN_OK) return st;
  }
  return cuda_status(gqa::launch_decode(q, nullptr, nullptr, nullptr, nullptr, false, positions,
                                        nullptr, k_cache, v_cache, B, Hq, Hkv, L, D, 0, scale,
                                        out, workspace, stream, S));
}

int attn_decode_stream_step(const void* q, const void* k_new, const void* v_new,
                            const float* cos_table, const float* sin_table, int32_t* positions,
                            void* k_cache, void* v_cache, int B, int Hq, int Hkv, int L, int D,
                            float scale, void* out, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
  if (!k_new || !v_new) return ATTN_ERR_INVALID_ARG;
  if ((cos_table == nullptr) != (sin_table == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (cos_table && (!aligned16(cos_table) || !aligned16(sin_table))) return ATTN_ERR_INVALID_ARG;
  return decode_append(q, k_new, v_new, cos_table, sin_table, true, positions, positions, k_cache,
                       v_cache, B, Hq, Hkv, L, D, scale, out, workspace, workspace_bytes, stream);
}

int attn_decode_step_noalloc(const void* q, const int32_t* positions, const void* k_cache,
                             const void* v_cache, int B, int Hq, int Hkv, int L, int D,
                             float scale, void* out, cudaStream_t stream) {
  if (!q || !positions || !k_cache || !v_cache || !out) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || L <= 0 || D <= 0 || Hq % Hkv != 0)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(positions) & 3u))
    return ATTN_ERR_INVALID_ARG;
  if (!gqa::decode_supported(B, Hq, Hkv, L, D)) return ATTN_ERR_UNSUPPORTED;
  if (gqa::decode_workspace_layout(B, Hq, Hkv, D).total > gqa::noalloc_scratch_bytes())
    return ATTN_ERR_WORKSPACE;  // beyond the built-in scratch
  return cuda_status(gqa::launch_decode_noalloc(q, positions, k_cache, v_cache, B, Hq, Hkv, L,
                                                D, scale, out, stream));
}

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int qk_norm_rope(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                 int64_t v_stride, const void* q_weight, const void* k_weight, float eps,
                 const int32_t* positions, const float* cos_table, const float* sin_table, int B,
                 int S, int Hq, int Hkv, int D, int L, void* q_out, void* k_out, void* k_cache,
                 void* v_cache, cudaStream_t stream) {
  if (B < 0 || S < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || L <= 0) return ATTN_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || eps > 3e38f) return ATTN_ERR_INVALID_ARG;
  if ((long long)B * S >= (1ll << 31)) return ATTN_ERR_INVALID_ARG;
  if (D % 16 != 0 || D > 256) return ATTN_ERR_UNSUPPORTED;
  if (Hq > 65536 || Hkv > 65536) return ATTN_ERR_UNSUPPORTED;
  if ((cos_table == nullptr) != (sin_table == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (B == 0 || S == 0) return ATTN_OK;
  if (!q || !k || !positions || !q_out) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_weight) ||
      !aligned16(k_weight) || !aligned16(cos_table) || !aligned16(sin_table) ||
      !aligned16(q_out) || !aligned16(k_out) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned4(positions))
    return ATTN_ERR_INVALID_ARG;
  if (q_stride < (int64_t)Hq * D || k_stride < (int64_t)Hkv * D || q_stride % 8 || k_stride % 8 ||
      (v && (v_stride < (int64_t)Hkv * D || v_stride % 8)))
    return ATTN_ERR_INVALID_ARG;
  return cuda_status(gqa::launch_qk_norm_rope(q, k, v, q_stride, k_stride, v_stride, q_weight,
                                              k_weight, eps, cos_table, sin_table, positions, B, S,
                                              Hq, Hkv, D, L, q_out, k_out, k_cache, v_cache,
                                              stream));
}

bool block_supported(int block) {
  return block == 16 || block == 32 || block == 64 || block == 128;
}

// Sizes common to the 8-bit cache's calls: ATTN_OK, or the error.
int kv8_sizes(int B, int Hq, int Hkv, int L, int D, int block) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || L <= 0 || D <= 0 || block <= 0 || Hq % Hkv != 0)
    return ATTN_ERR_INVALID_ARG;
  if (D != gqa::kDecodeD || !block_supported(block) || Hq / Hkv > 16 || Hkv > 1024 ||
      B > gqa::kDecodeMaxB || L > (1 << 24))
    return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

int kv8_decode(const void* q, const int32_t* positions, const void* k_cache, const void* v_cache,
               const float* k_scale, const float* v_scale, const int32_t* block_index, int count,
               int B, int Hq, int Hkv, int L, int D, int block, float scale, void* out,
               void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!q || !positions || !k_cache || !v_cache || !k_scale || !v_scale || !out)
    return ATTN_ERR_INVALID_ARG;
  if (const int st = kv8_sizes(B, Hq, Hkv, L, D, block)) return st;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      !aligned4(positions) || !aligned4(k_scale) || !aligned4(v_scale) || !aligned4(block_index))
    return ATTN_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < gqa::kv8_workspace_layout(B, Hq, Hkv).total)
    return ATTN_ERR_WORKSPACE;
  return cuda_status(gqa::launch_kv8_decode(q, positions, k_cache, v_cache, k_scale, v_scale,
                                            block_index, count, B, Hq, Hkv, L, block, scale, out,
                                            workspace, stream));
}

bool list_ok(int count, int block) {
  return count >= 1 && (long long)count * block <= (1ll << 24);
}

// Workspace of the sparse step: the decode's, then the scores, then the list.
struct SparseWorkspace {
  size_t scores_off, index_off, total;
};
SparseWorkspace sparse_layout(int B, int Hq, int Hkv, int L, int block, int count) {
  auto align256 = [](size_t x) { return (x + 255) & ~(size_t)255; };
  SparseWorkspace w;
  w.scores_off = gqa::kv8_workspace_layout(B, Hq, Hkv).total;
  w.index_off = align256(w.scores_off + (size_t)B * Hkv * ((L + block - 1) / block) * 4);
  w.total = align256(w.index_off + (size_t)B * Hkv * count * 4);
  return w;
}

}  // namespace

int attn_qk_norm_rope(const void* q, const void* k, int64_t q_stride, int64_t k_stride,
                      const void* q_weight, const void* k_weight, float eps,
                      const int32_t* positions, const float* cos_table, const float* sin_table,
                      int N, int Hq, int Hkv, int D, int L, void* q_out, void* k_out,
                      cudaStream_t stream) {
  if (N > 0 && !k_out) return ATTN_ERR_INVALID_ARG;
  return qk_norm_rope(q, k, nullptr, q_stride, k_stride, 0, q_weight, k_weight, eps, positions,
                      cos_table, sin_table, N, 1, Hq, Hkv, D, L, q_out, k_out, nullptr, nullptr,
                      stream);
}

int attn_qk_norm_rope_append(const void* q, const void* k_new, const void* v_new,
                             int64_t q_stride, int64_t k_stride, int64_t v_stride,
                             const void* q_weight, const void* k_weight, float eps,
                             const int32_t* positions, const float* cos_table,
                             const float* sin_table, void* k_cache, void* v_cache, int B, int S,
                             int Hq, int Hkv, int D, int L, void* q_out, cudaStream_t stream) {
  if (B > 0 && S > 0 && (!v_new || !k_cache || !v_cache)) return ATTN_ERR_INVALID_ARG;
  return qk_norm_rope(q, k_new, v_new, q_stride, k_stride, v_stride, q_weight, k_weight, eps,
                      positions, cos_table, sin_table, B, S, Hq, Hkv, D, L, q_out, nullptr,
                      k_cache, v_cache, stream);
}

int attn_kv8_append(const void* k_new, const void* v_new, int64_t k_stride, int64_t v_stride,
                    const int32_t* positions, void* k_cache, void* v_cache, float* k_scale,
                    float* v_scale, void* k_bounds, int B, int S, int Hkv, int L, int D,
                    int block, cudaStream_t stream) {
  if (S < 0) return ATTN_ERR_INVALID_ARG;
  if (const int st = kv8_sizes(B, Hkv, Hkv, L, D, block)) return st;
  if (S == 0) return ATTN_OK;
  if (!k_new || !v_new || !positions || !k_cache || !v_cache || !k_scale || !v_scale)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(k_bounds) || !aligned4(positions) || !aligned4(k_scale) || !aligned4(v_scale))
    return ATTN_ERR_INVALID_ARG;
  if (k_stride < (int64_t)Hkv * D || v_stride < (int64_t)Hkv * D || k_stride % 8 || v_stride % 8)
    return ATTN_ERR_INVALID_ARG;
  if (S > L) return ATTN_OK;  // no sequence's rows fit: all are skipped
  return cuda_status(gqa::launch_kv8_append(k_new, v_new, k_stride, v_stride, positions, k_cache,
                                            v_cache, k_scale, v_scale, k_bounds, B, S, Hkv, L,
                                            block, stream));
}

size_t attn_kv8_workspace_size(int B, int Hq, int Hkv, int L, int D) {
  if (kv8_sizes(B, Hq, Hkv, L, D, 16) != ATTN_OK) return 0;
  return gqa::kv8_workspace_layout(B, Hq, Hkv).total;
}

size_t attn_kv8_sparse_workspace_size(int B, int Hq, int Hkv, int L, int D, int block,
                                      int count) {
  if (kv8_sizes(B, Hq, Hkv, L, D, block) != ATTN_OK || !list_ok(count, block)) return 0;
  return sparse_layout(B, Hq, Hkv, L, block, count).total;
}

int attn_decode_step_kv8(const void* q, const int32_t* positions, const void* k_cache,
                         const void* v_cache, const float* k_scale, const float* v_scale, int B,
                         int Hq, int Hkv, int L, int D, int block, float scale, void* out,
                         void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return kv8_decode(q, positions, k_cache, v_cache, k_scale, v_scale, nullptr, 0, B, Hq, Hkv, L,
                    D, block, scale, out, workspace, workspace_bytes, stream);
}

int attn_decode_step_kv8_blocks(const void* q, const int32_t* positions, const void* k_cache,
                                const void* v_cache, const float* k_scale, const float* v_scale,
                                const int32_t* block_index, int count, int B, int Hq, int Hkv,
                                int L, int D, int block, float scale, void* out, void* workspace,
                                size_t workspace_bytes, cudaStream_t stream) {
  if (!block_index || !list_ok(count, block)) return ATTN_ERR_INVALID_ARG;
  return kv8_decode(q, positions, k_cache, v_cache, k_scale, v_scale, block_index, count, B, Hq,
                    Hkv, L, D, block, scale, out, workspace, workspace_bytes, stream);
}

int attn_block_scores(const void* q, const int32_t* positions, const void* k_bounds, int B,
                      int Hq, int Hkv, int L, int D, int block, float* scores,
                      cudaStream_t stream) {
  if (!q || !positions || !k_bounds || !scores) return ATTN_ERR_INVALID_ARG;
  if (const int st = kv8_sizes(B, Hq, Hkv, L, D, block)) return st;
  if (!aligned16(q) || !aligned16(k_bounds) || !aligned4(positions) || !aligned4(scores))
    return ATTN_ERR_INVALID_ARG;
  return cuda_status(gqa::launch_block_scores(q, positions, k_bounds, B, Hq, Hkv, L, block,
                                              scores, stream));
}

int attn_block_select(const float* scores, const int32_t* positions, int B, int Hkv, int L,
                      int block, int count, int first, int recent, int32_t* block_index,
                      cudaStream_t stream) {
  if (!scores || !positions || !block_index) return ATTN_ERR_INVALID_ARG;
  if (count < 1 || first < 0 || recent < 0 || first > count - recent)
    return ATTN_ERR_INVALID_ARG;
  if (const int st = kv8_sizes(B, Hkv, Hkv, L, gqa::kDecodeD, block)) return st;
  if (!aligned4(scores) || !aligned4(positions) || !aligned4(block_index))
    return ATTN_ERR_INVALID_ARG;
  return cuda_status(gqa::launch_block_select(scores, positions, B, Hkv, L, block, count, first,
                                              recent, block_index, stream));
}

int attn_decode_step_kv8_sparse(const void* q, const int32_t* positions, const void* k_cache,
                                const void* v_cache, const float* k_scale, const float* v_scale,
                                const void* k_bounds, int count, int first, int recent, int B,
                                int Hq, int Hkv, int L, int D, int block, float scale, void* out,
                                void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!k_cache || !v_cache || !k_scale || !v_scale || !out || !list_ok(count, block) ||
      first < 0 || recent < 0 || first > count - recent)
    return ATTN_ERR_INVALID_ARG;
  if (const int st = kv8_sizes(B, Hq, Hkv, L, D, block)) return st;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned4(k_scale) ||
      !aligned4(v_scale))
    return ATTN_ERR_INVALID_ARG;
  const SparseWorkspace ws = sparse_layout(B, Hq, Hkv, L, block, count);
  if (!workspace || !aligned16(workspace) || workspace_bytes < ws.total)
    return ATTN_ERR_WORKSPACE;
  float* scores = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + ws.scores_off);
  int32_t* index = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + ws.index_off);
  int st = attn_block_scores(q, positions, k_bounds, B, Hq, Hkv, L, D, block, scores, stream);
  if (st == ATTN_OK)
    st = attn_block_select(scores, positions, B, Hkv, L, block, count, first, recent, index,
                           stream);
  if (st == ATTN_OK)
    st = kv8_decode(q, positions, k_cache, v_cache, k_scale, v_scale, index, count, B, Hq, Hkv, L,
                    D, block, scale, out, workspace, ws.scores_off, stream);
  return st;
}

int attn_prefill_causal(const void* q, const void* k, const void* v, int S, int start_pos,
                        int Hq, int Hkv, int d, float scale, void* out, cudaStream_t stream) {
  if (S < 0 || start_pos < 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || Hq % Hkv != 0)
    return ATTN_ERR_INVALID_ARG;
  if ((long long)start_pos + S >= (1ll << 31)) return ATTN_ERR_INVALID_ARG;
  if (!gqa::prefill_supported(Hq, Hkv, d)) return ATTN_ERR_UNSUPPORTED;
  if (S == 0) return ATTN_OK;
  if (!q || !k || !v || !out) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
    return ATTN_ERR_INVALID_ARG;
  return cuda_status(
      gqa::launch_prefill(q, k, v, S, start_pos, Hq, Hkv, d, scale, out, stream));
}

int attn_read_prefill_status(uint32_t* timeouts, cudaStream_t stream) {
  uint32_t n = 0;
  const cudaError_t e = gqa::prefill_read_timeouts(&n, stream);
  if (e != cudaSuccess) return cuda_status(e);
  if (timeouts) *timeouts = n;
  return n ? ATTN_ERR_DEVICE : ATTN_OK;
}

int attn_read_prefill_skips(uint32_t* skips, cudaStream_t stream) {
  uint32_t n = 0;
  const cudaError_t e = gqa::prefill_read_skips(&n, stream);
  if (e != cudaSuccess) return cuda_status(e);
  if (skips) *skips = n;
  return n ? ATTN_ERR_DEVICE : ATTN_OK;
}

int attn_read_range_skips(uint32_t* skips, cudaStream_t stream) {
  uint32_t n[3] = {0, 0, 0};
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess) e = gqa::qk_norm_read_skips(&n[0]);
  if (e == cudaSuccess) e = gqa::kv8_append_read_skips(&n[1]);
  if (e == cudaSuccess) e = gqa::block_read_skips(&n[2]);
  if (e != cudaSuccess) return cuda_status(e);
  const uint32_t all = n[0] + n[1] + n[2];
  if (skips) *skips = all;
  return all ? ATTN_ERR_DEVICE : ATTN_OK;
}

int attn_debug_build(void) {
#ifdef GQA_DEBUG
  return 1;
#else
  return 0;
#endif
}

int attn_read_device_status(void* workspace, uint32_t* bits, cudaStream_t stream) {
  if (!workspace) return ATTN_ERR_INVALID_ARG;
  uint32_t word = 0;
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess) e = cudaMemcpy(&word, workspace, sizeof(word), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemset(workspace, 0, sizeof(word));
  if (e != cudaSuccess) return cuda_status(e);
  if (bits) *bits = word;
  return word ? ATTN_ERR_DEVICE : ATTN_OK;
}

int attn_test_force_schedule(int cluster) {
  if (cluster < -1 || cluster > 16) return ATTN_ERR_INVALID_ARG;
  gqa::g_decode_test_cluster = cluster;
  return ATTN_OK;
}

int attn_test_skip_tile(int tile) {
  if (tile < -1) return ATTN_ERR_INVALID_ARG;
  gqa::g_decode_test_skip = tile;
  return ATTN_OK;
}

const char* attn_status_string(int status) {
  switch (status) {
    case ATTN_OK: return "ok";
    case ATTN_ERR_INVALID_ARG: return "invalid argument";
    case ATTN_ERR_UNSUPPORTED: return "unsupported size";
    case ATTN_ERR_WORKSPACE: return "workspace missing or too small";
    case ATTN_ERR_CUDA: return "CUDA error";
    case ATTN_ERR_DEVICE: return "device flagged an error";
    default: return "unknown status";
  }
}

int attn_last_cuda_error(void) { return g_last_cuda_error; }

}  // extern "C"
