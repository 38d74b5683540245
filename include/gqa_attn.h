/*
 * gqa_attn.h -- C ABI of libgqa_attn.so: in-place static-KV-cache GQA decode
 * attention and causal prefill over a cached prefix, for NVIDIA GB300
 * (sm_103a).
 *
 * Where the operations come from (page title, section):
 *   - "MiniCPM4 `forward_step` Attention Performance Fix", section 4.1: each
 *     decode step writes the new key/value row of every KV head in place into
 *     a preallocated static cache [B, Hkv, max_len, D] at position_id, then
 *     attends the query heads (GQA, enable_gqa) over cache rows
 *     0..position_id only -- no boolean mask and no full-length copy
 *     (section 3).  Sections 2.4 and 6.4: the per-step cost must grow with
 *     position_id + 1, not with max_len.
 *   - "step14_3 -- batched attention", sections "problem" and
 *     "F.scaled_dot_product_attention": prefill of S new tokens whose K/V
 *     include the cached prefix, token-major layout [tokens, heads, d_head].
 *
 * Conventions shared by every call:
 *   - All tensor pointers are DEVICE pointers owned by the caller.  The library
 *     never allocates, frees or keeps device memory.
 *   - Tensors are bf16 (raw 16-bit storage, `const void*`), dense, row-major,
 *     with the shapes given per call.  Every tensor pointer must be 16-byte
 *     aligned.
 *   - GQA: query head h reads KV head h / g, g = Hq / Hkv (contiguous groups,
 *     the repeat-KV convention).
 *   - Kernels are launched with programmatic stream serialisation: a launch
 *     may start its prologue while the previous kernel on `stream` drains,
 *     and waits for that kernel's writes before reading any input.
 *   - Every call is asynchronous on `stream` and returns an int status
 *     (ATTN_OK or an ATTN_ERR_* code).  Argument errors are found on the host
 *     before anything is launched; nothing is then written.  ATTN_ERR_CUDA means
 *     a launch failed; attn_last_cuda_error() returns the CUDA error code.
 *   - Errors that only the device can see (a position outside [0, max_len))
 *     never trap: the affected sequence is skipped, decode writes NaN to its
 *     output rows, and a bit is set in the device status word kept in the
 *     decode workspace (read it with attn_read_device_status).
 */
#ifndef GQA_ATTN_H
#define GQA_ATTN_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. */
#define ATTN_OK                0
#define ATTN_ERR_INVALID_ARG   1  /* null pointer, non-positive size, Hq % Hkv != 0,
                                     pointer not 16-byte aligned, start_pos < 0 */
#define ATTN_ERR_UNSUPPORTED   2  /* a size the library has no kernel for (see each call) */
#define ATTN_ERR_WORKSPACE     3  /* workspace null or smaller than attn_decode_workspace_size() */
#define ATTN_ERR_CUDA          4  /* a CUDA runtime call or launch failed */
#define ATTN_ERR_DEVICE        5  /* attn_read_device_status: the device flagged a fault */

/* Bits of the device status word (attn_read_device_status(..., &bits)). */
#define ATTN_DEV_BAD_POSITION  0x1u  /* some positions[b] was outside [0, max_len) */
#define ATTN_DEV_TIMEOUT       0x2u  /* a pipeline wait gave up (the kernel returned early) */
#define ATTN_DEV_RANGE         0x4u  /* debug builds only (attn_debug_build() == 1): an
                                        index-derived access (a bulk-copy tile coordinate,
                                        a cluster landing slot, a partial-result slot, an
                                        output or new-row address) failed its range check
                                        and was skipped; the launch's outputs are undefined */
#define ATTN_DEV_BAD_BLOCK     0x8u  /* a listed block below -1 or past the cache's last one
                                        (attn_decode_step_kv8_blocks); it was skipped */
#define ATTN_DEV_BAD_PAGE      0x10u /* attn_decode_step_paged: a page table entry that holds
                                        attended rows names no page; its rows were skipped */
#define ATTN_DEV_BAD_PARENT    0x20u /* attn_pages_fork: a parent outside -1 .. B - 1; the row
                                        kept its entries */

/*
 * attn_kv_append -- the in-place cache write of the decode page, section 4.1
 * (key_cache[:, :, position_id, :] = key_states; same for values), with one
 * position per sequence.
 *
 *   k_new, v_new : [B, Hkv, D] bf16, the new rows.
 *   positions    : [B] int32, device memory; row positions[b] of every KV head
 *                  of sequence b is overwritten.
 *   k_cache,
 *   v_cache      : [B, Hkv, L, D] bf16, modified in place.  Every other byte
 *                  is left untouched (bit-exact copy of the new rows).
 *   D            : multiple of 8 (16-byte rows), 8 <= D <= 256.
 *
 * A position outside [0, L) skips that sequence's write (no other effect;
 * attn_decode_step with the same positions reports it).
 */
int attn_kv_append(const void* k_new, const void* v_new, const int32_t* positions,
                   void* k_cache, void* v_cache,
                   int B, int Hkv, int L, int D, cudaStream_t stream);

/*
 * attn_decode_workspace_size -- bytes of device workspace attn_decode_step
 * needs for these sizes (split-KV partial results, per-(sequence, KV head)
 * arrival counters and the device status word).  Returns 0 if the sizes are
 * invalid or unsupported.  The workspace must be zero-filled before its first
 * use (e.g. cudaMemsetAsync).  Every call leaves its arrival counters at zero
 * again, so later calls with the same (B, Hq, Hkv, D) can reuse it as is; zero
 * it again before using it with other sizes, or after a call that reported
 * ATTN_DEV_TIMEOUT.  Calls that share a workspace must not overlap in time.
 */
size_t attn_decode_workspace_size(int B, int Hq, int Hkv, int L, int D);

/*
 * attn_decode_step -- sliced decode attention of the decode page, sections 3
 * and 4.1: for every sequence b and query head h,
 *     out[b,h,:] = softmax_j(scale * q[b,h,:] . K[b,h/g,j,:]) V[b,h/g,j,:]
 * over j = 0..positions[b] inclusive.  Rows above positions[b] are never read
 * (they may hold anything, NaN included).  Call attn_kv_append first for the
 * step's new row (the page writes the row, then attends).
 *
 *   q         : [B, Hq, D] bf16 (one query token per sequence).
 *   positions : [B] int32, device memory.
 *   k_cache,
 *   v_cache   : [B, Hkv, L, D] bf16.
 *   scale     : fp32 score scale (the page's default is 1/sqrt(D)).
 *   out       : [B, Hq, D] bf16 (= [B, Hq*D]), fp32 softmax and accumulation,
 *               rounded to nearest even.  Both contractions of a tile run
 *               on tensor cores with bf16 operands and fp32 accumulation:
 *               per warp (mma.sync) for g <= 8, with the probabilities
 *               entering P.V as two bf16 parts (about 16 bits; an infinite
 *               value in an attended row may give NaN there); on the
 *               tcgen05 tensor cores for g = 16 (and for the rotary entry
 *               points at g = 8), with the probabilities rounded to bf16
 *               before P.V.
 *   workspace : device buffer of at least attn_decode_workspace_size(...)
 *               bytes, zero-filled before first use (see above).
 *
 * Supported: D == 128; g = Hq / Hkv in {1, 2, 4, 8, 16} (g = 16 on the
 * tcgen05 tensor cores); 1 <= B <= 8192;
 * 1 <= L <= 2^24.  Work is split over the attended rows only, so the cost of
 * a step follows sum_b (positions[b] + 1), not B * L.
 */
int attn_decode_step(const void* q, const int32_t* positions,
                     const void* k_cache, const void* v_cache,
                     int B, int Hq, int Hkv, int L, int D, float scale,
                     void* out, void* workspace, size_t workspace_bytes,
                     cudaStream_t stream);

/*
 * attn_decode_step_append -- one decode step of the decode page, section 4.1,
 * in one launch: the cache write of attn_kv_append followed by the attention
 * of attn_decode_step.  Results are those of the two calls in that order:
 * row positions[b] of every KV head of sequence b becomes k_new/v_new
 * (bit-exact) and out is attention over rows 0..positions[b], the new row
 * included.  The new rows are fed to the attention straight from k_new/v_new
 * and written to the cache in the same launch.  For g <= 8 the new row goes
 * through the tile like any cache row, so out is bit-identical to the two
 * calls; on the tcgen05 kernels (g = 16) its score and value are folded in
 * fp32 beside the tile, so out agrees with the two calls to rounding.
 *
 *   q            : [B, Hq, D] bf16.
 *   k_new, v_new : [B, Hkv, D] bf16.
 *   positions    : [B] int32, device memory.
 *   k_cache,
 *   v_cache      : [B, Hkv, L, D] bf16, row positions[b] written in place.
 *   out, workspace, scale and supported sizes: as attn_decode_step.
 *
 * A position outside [0, L) writes nothing for that sequence, gives NaN
 * output rows and sets ATTN_DEV_BAD_POSITION.
 */
int attn_decode_step_append(const void* q, const void* k_new, const void* v_new,
                            const int32_t* positions, void* k_cache, void* v_cache,
                            int B, int Hq, int Hkv, int L, int D, float scale,
                            void* out, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream);

/*
 * attn_decode_step_rope_append -- attn_decode_step_append with the rotary
 * position embedding applied first, as the decode page's forward_step does
 * (section 4.1: apply_rotary_pos_emb(q, k, cos, sin) runs before the cache
 * write).  The page does not define the rotation; this library takes the
 * rotate-half form, for every dim d of a row x:
 *     x'[d] = x[d]*cos[d] - x[d+D/2]*sin[d]          for d <  D/2
 *     x'[d] = x[d]*cos[d] + x[d-D/2]*sin[d]          for d >= D/2
 * in fp32, each product and the sum rounded separately (no fused
 * multiply-add).  The rotated key is rounded to bf16 (nearest even) and that
 * is what the cache row holds; the rotated query is kept in fp32 for the
 * attention.  v_new is appended unrotated.
 *
 *   cos, sin : [B, D] fp32, device memory, 16-byte aligned; row b is the
 *              rotation for sequence b at positions[b] (the caller computes
 *              it, so any frequency base or scaling works).  Read only.
 *   all other arguments, sizes and errors: as attn_decode_step_append.
 *
 * Errors: ATTN_ERR_INVALID_ARG also for a null or misaligned cos or sin;
 * ATTN_ERR_UNSUPPORTED for g = 16 (the rotation serves g <= 8: the
 * tensor-core kernels carry the rotated query as two bf16 rows per head).
 */
int attn_decode_step_rope_append(const void* q, const void* k_new, const void* v_new,
                                 const float* cos, const float* sin,
                                 const int32_t* positions, void* k_cache, void* v_cache,
                                 int B, int Hq, int Hkv, int L, int D, float scale,
                                 void* out, void* workspace, size_t workspace_bytes,
                                 cudaStream_t stream);

/*
 * attn_decode_step_window -- decode attention over a local window: each
 * sequence attends only its last `window` cache rows up to its position,
 *     rows max(0, positions[b] - window + 1) .. positions[b] inclusive,
 * so the current token is always included.  The decode pages name the
 * variant without defining it; this reading takes the W most recent rows.
 * Rows outside the window are never read.  The cost of a step follows
 * min(window, positions[b] + 1), not the position.
 *
 *   k_new, v_new : [B, Hkv, D] bf16 rows to append at positions[b] first
 *                  (as attn_decode_step_append), or both null to attend only
 *                  (as attn_decode_step).
 *   window       : > 0; window >= positions[b] + 1 is the full decode.
 *   all other arguments, sizes and errors: as attn_decode_step_append.
 *
 * Errors: ATTN_ERR_INVALID_ARG also for window <= 0, or for exactly one of
 * k_new and v_new null.
 */
int attn_decode_step_window(const void* q, const void* k_new, const void* v_new,
                            const int32_t* positions, void* k_cache, void* v_cache,
                            int B, int Hq, int Hkv, int L, int D, int window, float scale,
                            void* out, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream);

/*
 * attn_decode_multi -- multi-token decode: S new tokens per sequence (for
 * example draft tokens to verify) in one launch.  Token t of sequence b sits
 * at position positions[b] + t and attends cache rows
 * 0 .. positions[b] + t: the earlier new tokens and itself, not the later
 * ones.  Each KV byte is read once for all S tokens and g query heads of its
 * KV head.  This is the decode page's step for several tokens at once.  The
 * causal rule for the new block is the prefill page's, aligned to the
 * bottom-right corner.
 *
 *   q            : [B, S, Hq, D] bf16.
 *   k_new, v_new : [B, S, Hkv, D] bf16, appended first at rows
 *                  positions[b] .. positions[b] + S - 1 (a separate launch
 *                  ahead of the attention); or both null when the cache
 *                  already holds them.
 *   positions    : [B] int32, device memory: the first new token's position.
 *   out          : [B, S, Hq, D] bf16.
 *   workspace    : at least attn_decode_workspace_size(B, S * Hq, Hkv, L, D)
 *                  bytes, zero-filled before first use.
 *   Supported: D == 128; S * g in {1, 2, 4, 8, 16}; other limits as
 *   attn_decode_step.  S == 1 is attn_decode_step (after the append).
 *
 * A sequence whose positions[b] + S - 1 falls outside [0, L) gets NaN in all
 * of its output rows, no cache write, and ATTN_DEV_BAD_POSITION.
 * Errors: ATTN_ERR_INVALID_ARG for null or misaligned pointers, exactly one
 * of k_new and v_new null, or non-positive sizes; ATTN_ERR_UNSUPPORTED when
 * S * g is not 1, 2, 4, 8 or 16; ATTN_ERR_WORKSPACE as above.
 */
int attn_decode_multi(const void* q, const void* k_new, const void* v_new,
                      const int32_t* positions, void* k_cache, void* v_cache,
                      int B, int S, int Hq, int Hkv, int L, int D, float scale,
                      void* out, void* workspace, size_t workspace_bytes,
                      cudaStream_t stream);

/*
 * attn_decode_stream_step -- one step of a streaming decode loop that a CUDA
 * graph can capture once and replay unchanged.  It performs the fused step of
 * attn_decode_step_append (preceded by the rotary embedding of
 * attn_decode_step_rope_append when tables are given), then adds one to every
 * positions[b] on the device.  The decode page calls forward_step once per
 * new token at position_id, the next one at position_id + 1 (section 4.1);
 * keeping that counter on the device lets one captured launch serve every
 * step of the loop.
 *
 *   positions : [B] int32, device memory.  It is read as this step's positions,
 *               then every entry is incremented by one, out-of-range ones
 *               included.  The increment happens after every part of the
 *               launch has read them, so the result is the same as a step at
 *               the old positions followed by a host-side increment.
 *   cos_table,
 *   sin_table : [L, D] fp32, device memory, 16-byte aligned, or both null for
 *               no rotation.  Row p is the rotation at position p; the step
 *               uses row positions[b] for sequence b.  Read only.
 *   all other arguments, sizes and errors: as attn_decode_step_append.  The
 *   step uses a counter in the workspace and leaves it at zero again.
 *
 * Errors: ATTN_ERR_INVALID_ARG also when exactly one of cos_table and
 * sin_table is null, or either is misaligned; ATTN_ERR_UNSUPPORTED for the
 * rotation at g = 16 (as attn_decode_step_rope_append).
 */
int attn_decode_stream_step(const void* q, const void* k_new, const void* v_new,
                            const float* cos_table, const float* sin_table,
                            int32_t* positions, void* k_cache, void* v_cache,
                            int B, int Hq, int Hkv, int L, int D, float scale,
                            void* out, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream);

/*
 * attn_decode_step_noalloc -- attn_decode_step without a workspace argument.
 * The decode page has no counterpart: this entry point exists for callers
 * that cannot call cudaMalloc, for example plugin or embedded hosts that own
 * all device memory and hand the library none, and real-time streaming loops
 * where the device-wide synchronisation an allocation can imply would stall
 * playback.  It allocates nothing: its split-KV scratch is a fixed 16 MiB
 * device array inside the library, which every GPU that loads the library
 * holds until the process exits.
 *
 * Arguments, supported sizes and results are those of attn_decode_step.
 * Sizes whose attn_decode_workspace_size() exceeds 16 MiB (16777216 bytes)
 * are rejected with ATTN_ERR_WORKSPACE (B=256, Hq=64, Hkv=8, D=128 needs about
 * 12.8 MB and fits).  The first call on a device looks up the array's device
 * address (cudaGetSymbolAddress) while that device is current, and so does
 * the first call after the device's context was replaced (cudaDeviceReset).
 * The lookup is guarded by a mutex, so host threads may make their first
 * calls at the same time.  Every
 * call first clears the array's status word and arrival counters with
 * cudaMemsetAsync on `stream`.  All calls share the one array, so calls that
 * overlap on the GPU (other streams, other host threads) race and give wrong
 * results; serialise them.  The device status word is not readable for this
 * variant: an out-of-range position still gives NaN output rows.
 */
int attn_decode_step_noalloc(const void* q, const int32_t* positions,
                             const void* k_cache, const void* v_cache,
                             int B, int Hq, int Hkv, int L, int D, float scale,
                             void* out, cudaStream_t stream);

/*
 * attn_qk_norm_rope -- RMS norm of every query and key head and the rotary
 * embedding, in one pass.  For each row x (one head of one token, D dims) with
 * the head's weight w (one vector of D for all query heads, one for all key
 * heads):
 *     y[d]  = x[d] * w[d] / sqrt(mean(x^2) + eps)
 *     x'[d] = y[d]*cos[d] - y[d+D/2]*sin[d]          for d <  D/2
 *     x'[d] = y[d]*cos[d] + y[d-D/2]*sin[d]          for d >= D/2
 * in fp32 (the rotate-half form of attn_decode_step_rope_append), rounded to
 * bf16 once at the end.
 *
 *   q            : [N, Hq, D] bf16, token n at q + n * q_stride elements; the
 *                  heads of a token are dense.  k: [N, Hkv, D] with k_stride.
 *                  Strides let both be views of one fused projection buffer.
 *   q_weight,
 *   k_weight     : [D] bf16, or null for ones.
 *   cos_table,
 *   sin_table    : [L, D] fp32, row p the rotation at position p; both null for
 *                  no rotation.
 *   positions    : [N] int32, device memory, token n's position.
 *   q_out, k_out : [N, Hq, D] and [N, Hkv, D] bf16, dense.  They may be q and k
 *                  themselves where those are dense; no other overlap.
 *   Supported: D a multiple of 16, 16 <= D <= 256; N >= 0 (0 does nothing);
 *   strides multiples of 8 and at least a token's heads.
 *
 * A position outside [0, L) gives NaN in that token's rows.
 * Errors: ATTN_ERR_INVALID_ARG also for exactly one of cos_table and sin_table
 * null, a bad stride, or eps negative or not finite.
 */
int attn_qk_norm_rope(const void* q, const void* k, int64_t q_stride, int64_t k_stride,
                      const void* q_weight, const void* k_weight, float eps,
                      const int32_t* positions, const float* cos_table, const float* sin_table,
                      int N, int Hq, int Hkv, int D, int L, void* q_out, void* k_out,
                      cudaStream_t stream);

/*
 * attn_qk_norm_rope_append -- attn_qk_norm_rope for S new tokens per sequence
 * with the cache write of attn_kv_append in the same launch: the normed and
 * rotated keys and the values as they are become rows positions[b] + t of the
 * bf16 cache.  S = 1 is a decode step's, a long S a prompt's.
 *
 *   q            : [B, S, Hq, D] bf16, token b*S + t at q + (b*S + t) * q_stride;
 *                  k_new, v_new: [B, S, Hkv, D] with k_stride and v_stride.
 *   positions    : [B] int32, device memory: the first new token's position.
 *   k_cache,
 *   v_cache      : [B, Hkv, L, D] bf16, written in place.
 *   q_out        : [B, S, Hq, D] bf16, dense.
 *   the rest, sizes and errors: as attn_qk_norm_rope (S = 0 does nothing).
 *
 * A sequence whose rows positions[b] .. positions[b] + S - 1 are not all in
 * [0, L) gets no cache write and NaN in its rows of q_out.
 */
int attn_qk_norm_rope_append(const void* q, const void* k_new, const void* v_new,
                             int64_t q_stride, int64_t k_stride, int64_t v_stride,
                             const void* q_weight, const void* k_weight, float eps,
                             const int32_t* positions, const float* cos_table,
                             const float* sin_table, void* k_cache, void* v_cache, int B, int S,
                             int Hq, int Hkv, int D, int L, void* q_out, cudaStream_t stream);

/*
 * The 8-bit cache.  k_cache and v_cache are [B, Hkv, L, D] e4m3 codes (one
 * byte each); every block of `block` consecutive rows of a KV head has one
 * fp32 scale per operand, k_scale and v_scale [B, Hkv, NB] with
 * NB = ceil(L / block), and row j stands for scale[j / block] * code.  A row
 * costs half of what it does in the bf16 cache.
 *   block : 16, 32, 64 or 128.   D == 128.
 * The append writes scales 2^e with e in [-60, 60]; the decode takes any
 * positive scale in [2^-60, 2^60].
 * k_bounds [B, Hkv, NB, 2, D] bf16 (optional, for block selection): per block
 * and channel the largest (index 0) and the smallest (1) key value appended,
 * before rounding to 8 bits.
 *
 * attn_kv8_append -- S new rows per sequence, k_new and v_new [B, S, Hkv, D]
 * bf16, to rows positions[b] .. positions[b] + S - 1.  Token b*S + t lies at
 * k_new + (b*S + t) * k_stride (v_stride) elements, its heads dense; strides are
 * multiples of 8 and at least Hkv * D.  For every block of a
 * KV head that gets new rows, and for K and V apart:
 *     s_new = 2^e, e the least integer with max |x| <= 448 * 2^e over the
 *             block's new rows x (finite values only)
 *     s     = s_new if the block held no row before (positions[b] <= its
 *             first row), else max(s_old, s_new)
 *     its earlier rows, if s > s_old: code <- e4m3(code * s_old / s)
 *     its new rows:                   code <- e4m3(x / s)
 * rounded to nearest even, beyond +-448 saturating, NaN kept.  x / s is
 * x * (1 / s) in fp32: exact for the powers of two that the append writes; in a
 * block that holds rows at another scale, 1 / s is rounded first.  Only codes of
 * rows up to the last new one are written.  The bounds of a block become those
 * of its new rows and, if it held rows before, what they were (NaN ignored;
 * -inf and +inf for a channel with nothing else).
 *   k_bounds : or null.
 *   S        : >= 0 (0 does nothing).
 * A sequence whose rows are not all in [0, L) is skipped (the decode call
 * reports it).  Supported: B <= 8192, Hkv <= 1024, L <= 2^24.
 */
int attn_kv8_append(const void* k_new, const void* v_new, int64_t k_stride, int64_t v_stride,
                    const int32_t* positions, void* k_cache, void* v_cache, float* k_scale,
                    float* v_scale, void* k_bounds, int B, int S, int Hkv, int L, int D,
                    int block, cudaStream_t stream);

/*
 * attn_kv8_workspace_size -- bytes of device workspace the 8-bit decode calls
 * need; 0 if the sizes are invalid or unsupported.  The rules of
 * attn_decode_workspace_size hold: zero-filled before first use and before use
 * with other sizes, no overlapping calls on one workspace (two captured graphs
 * that may run at once need one each).  Its first word is the device status
 * word of attn_read_device_status.
 */
size_t attn_kv8_workspace_size(int B, int Hq, int Hkv, int L, int D);

/*
 * attn_decode_step_kv8 -- attn_decode_step over the 8-bit cache: for every
 * sequence b and query head h, over rows j = 0..positions[b],
 *     out[b,h,:] = softmax_j(scale * q[b,h,:] . ks_j k_j) (vs_j v_j)
 * with the codes k_j, v_j and scales ks_j, vs_j of row j and KV head h / g.
 * Codes enter both products exactly (as fp16), q exactly to 2^-22 of its
 * head's largest element, the probabilities (relative to the row that
 * contributes most) as two fp16 parts for g <= 8 (22 bits) and rounded once to
 * fp16 for g > 8; sums in fp32.  Codes and scales of rows above positions[b] are not used and may hold
 * anything.
 *
 *   Supported: D == 128; any g = Hq / Hkv from 1 to 16; B <= 8192;
 *   B * Hkv < 2^31 / 16; L <= 2^24.
 * A position outside [0, L) gives NaN output rows and ATTN_DEV_BAD_POSITION.
 * Errors: as attn_decode_step; ATTN_ERR_UNSUPPORTED also for another block.
 */
int attn_decode_step_kv8(const void* q, const int32_t* positions, const void* k_cache,
                         const void* v_cache, const float* k_scale, const float* v_scale, int B,
                         int Hq, int Hkv, int L, int D, int block, float scale, void* out,
                         void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * attn_block_scores -- an upper bound of what a query can score with a block's
 * keys as they were appended, summed over the g query heads of a KV head:
 *     scores[b,hk,j] = sum_h sum_d max(q[b,h,d] * max_jd, q[b,h,d] * min_jd)
 * over the heads h of KV head hk, from k_bounds; -inf for blocks past
 * positions[b] / block (and for all blocks of a position outside [0, L)).
 * Their bounds are not read.  fp32 sums.  (A bound for positive score scales.)
 * The decode attends the keys' codes, which may lie beyond the bounds by their
 * rounding, half an e4m3 step (up to 2^-4 of a value), so a code's score may
 * exceed the block's by that much: the scores rank blocks, they do not prove
 * that a block left out holds no larger score.
 *
 *   scores : [B, Hkv, NB] fp32.
 *   Sizes as attn_decode_step_kv8.  The bounds are taken as finite.
 */
int attn_block_scores(const void* q, const int32_t* positions, const void* k_bounds, int B,
                      int Hq, int Hkv, int L, int D, int block, float* scores,
                      cudaStream_t stream);

/*
 * attn_block_select -- per sequence and KV head, `count` of the blocks
 * 0 .. positions[b] / block: all of them if there are no more, else the first
 * `first`, the last `recent`, and of the others those with the largest scores,
 * ties to the lowest index (NaN counts as -inf).  block_index [B, Hkv, count]
 * int32, ascending, -1 behind the last (all -1 for a position outside [0, L)).
 *
 *   Errors: ATTN_ERR_INVALID_ARG also for count < 1, first or recent < 0, or
 *   first + recent > count.
 */
int attn_block_select(const float* scores, const int32_t* positions, int B, int Hkv, int L,
                      int block, int count, int first, int recent, int32_t* block_index,
                      cudaStream_t stream);

/*
 * attn_decode_step_kv8_blocks -- attn_decode_step_kv8 over the rows of listed
 * blocks only, up to each position: block_index [B, Hkv, count] int32, any
 * order, -1 for none.  A block listed twice counts twice; one past the
 * position adds nothing; a list without any row gives zeros.  An index below
 * -1 or not below NB is skipped and sets ATTN_DEV_BAD_BLOCK.
 *   count : >= 1, count * block <= 2^24.  The rest as attn_decode_step_kv8.
 */
int attn_decode_step_kv8_blocks(const void* q, const int32_t* positions, const void* k_cache,
                                const void* v_cache, const float* k_scale, const float* v_scale,
                                const int32_t* block_index, int count, int B, int Hq, int Hkv,
                                int L, int D, int block, float scale, void* out, void* workspace,
                                size_t workspace_bytes, cudaStream_t stream);

/*
 * attn_decode_step_kv8_sparse -- attn_block_scores, attn_block_select and
 * attn_decode_step_kv8_blocks in turn on `stream`: one decode step that attends
 * `count` blocks per KV head.  The block of the position itself is attended if
 * recent >= 1.  Scores and indices lie in the workspace, which needs
 * attn_kv8_sparse_workspace_size(...) bytes (0: invalid or unsupported).
 */
size_t attn_kv8_sparse_workspace_size(int B, int Hq, int Hkv, int L, int D, int block, int count);
int attn_decode_step_kv8_sparse(const void* q, const int32_t* positions, const void* k_cache,
                                const void* v_cache, const float* k_scale, const float* v_scale,
                                const void* k_bounds, int count, int first, int recent, int B,
                                int Hq, int Hkv, int L, int D, int block, float scale, void* out,
                                void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * The paged cache.  Keys and values lie in a pool of P pages, k_pages and
 * v_pages [P, Hkv, page, D] bf16, laid out alike: element (p, h, r, d) at
 * p * page_stride + h * head_stride + r * row_stride + d elements from either
 * base.  Strides are multiples of 8, row_stride >= D, and rows do not overlap
 * (any order of the three; a stride whose size is 1 counts for nothing).  The
 * calls that write into the pool want two different bases.
 *   page       : 16, 32, 64 or 128 rows.   D: 64 or 128.
 *   page_table : [B, M] int32: row j of sequence b is row j % page of page
 *                page_table[b][j / page], -1 for none.  A sequence can hold
 *                M * page rows (at most 2^30).
 *   page_refs  : [P] int32: how many table entries name a page; 0: it is free.
 *                Sequences may share pages (forked ones do); rows are written
 *                only into pages of one's own, which attn_pages_reserve sees to.
 *   positions  : [B] int32: the row of each sequence's first new token.
 *   lengths    : [B] int32, 0 .. S new tokens of each sequence in a padded
 *                batch, or null for S each.
 * All of these are device memory.  A step is: attn_pages_reserve,
 * attn_paged_append, attn_decode_step_paged; attn_pages_fork passes pages on,
 * cuts sequences and frees them; attn_pages_compact moves what is in use to the
 * front of the pool.
 *
 * attn_paged_append -- rows k_new, v_new [B, S, Hkv, D] (token b*S + t at
 * (b*S + t) * k_stride or v_stride elements, its heads dense) to rows
 * positions[b] + t for t < lengths[b], bit-exact.  Nothing else is written.
 * A sequence whose rows are not all in [0, M * page), or whose lengths[b] is not
 * in 0 .. S, is skipped, and so are rows without a page (the decode call reports
 * both).  S = 0 does nothing.
 *   Limits: Hkv <= 1024, P <= 2^26.
 */
int attn_paged_append(const void* k_new, const void* v_new, int64_t k_stride, int64_t v_stride,
                      const int32_t* positions, const int32_t* lengths,
                      const int32_t* page_table, void* k_pages, void* v_pages,
                      int64_t page_stride, int64_t head_stride, int64_t row_stride, int B, int S,
                      int Hkv, int D, int P, int page, int M, cudaStream_t stream);

/*
 * attn_paged_workspace_size -- bytes of device workspace attn_decode_step_paged
 * needs; 0 if the sizes are invalid or unsupported.  The rules of
 * attn_decode_workspace_size hold: zero-filled before first use, before use
 * with other sizes and after ATTN_DEV_TIMEOUT; no overlapping calls on one
 * workspace (two captured graphs that may run at once need one each).  Its
 * first word is the device status word of attn_read_device_status.
 */
size_t attn_paged_workspace_size(int B, int S, int Hq, int Hkv, int D);

/*
 * attn_decode_step_paged -- attn_decode_step (S = 1) and attn_decode_multi over
 * the paged cache: token t of sequence b attends rows 0 .. positions[b] + t,
 *     out[b,t,h] = softmax_j(scale * q[b,t,h] . K_j) V_j
 * with K_j and V_j of KV head h / g.  The rows must be there already
 * (attn_paged_append).  Rows that a token does not see may hold anything, NaN
 * included, and entries behind the last attended row any number.  An infinite value
 * in a row that it sees makes its output infinite in that dim, if the row's weight
 * is at least 2^-100 of the largest; with less it may be NaN, and infinities of
 * both signs give NaN.  So do scores of +inf or NaN, in all dims.  A token all of
 * whose scores are -inf gets zeros, like one that no row is left for.
 *
 *   q, out : [B, S, Hq, D] bf16.  Tokens t >= lengths[b] get zeros.
 *   Both products in bf16 with fp32 sums, as in attn_decode_step; the
 *   probabilities enter as two bf16 parts (16 bits), at D = 64 and S * g > 16
 *   rounded to bf16 once.
 *   Supported: any g = Hq / Hkv with S * g <= 32; B <= 4096; Hkv <= 1024;
 *   B * Hkv < 2^31 / 16; max(B, Hkv) * (M * page / 128 + 8) < 2^31.
 *
 * A sequence whose rows positions[b] .. positions[b] + lengths[b] - 1 are not
 * all in [0, M * page), or whose lengths[b] is not in 0 .. S, gets NaN output
 * rows and ATTN_DEV_BAD_POSITION; with lengths[b] = 0 its position and pages
 * may be anything.  An entry outside [0, P) that should hold attended rows
 * sets ATTN_DEV_BAD_PAGE and its rows are left out (zeros if none is left).
 */
int attn_decode_step_paged(const void* q, const int32_t* positions, const int32_t* lengths,
                           const int32_t* page_table, const void* k_pages, const void* v_pages,
                           int64_t page_stride, int64_t head_stride, int64_t row_stride, int B,
                           int S, int Hq, int Hkv, int D, int P, int page, int M, float scale,
                           void* out, void* workspace, size_t workspace_bytes,
                           cudaStream_t stream);

/*
 * attn_pages_workspace_size -- bytes of device workspace that the three calls
 * below need for these sizes (S: the most new tokens of a reserve); 0 if they
 * are invalid.  It must be zero-filled before its first use; its first word is
 * the device status word.  Calls that share a workspace must not overlap in time.
 */
size_t attn_pages_workspace_size(int B, int S, int P, int page);

/*
 * attn_pages_reserve -- pages for the new rows positions[b] .. positions[b] +
 * lengths[b] - 1.  Of the entries that hold them, one without a page (outside
 * [0, P)) takes a free page, and one whose page is shared (page_refs > 1) takes
 * a free page for itself: the rows before positions[b] that the shared page holds
 * are copied, and the shared page counts one entry less.  So every sequence that
 * shares a page and writes into it leaves it, the last one too: two that share one
 * take two, and a page that all of them left is free afterwards (not before).
 * The free pages (those whose count was 0 before the call) are taken from the
 * lowest on, in the order of the sequences and their rows.
 *
 *   taken : [B] int32: how many pages the sequence took; -1 if the pages that
 *           it and the sequences before it need are more than there are, or its
 *           rows do not fit (ATTN_DEV_BAD_POSITION): nothing of it is changed.
 *   S     : >= 1.  Other limits: B <= 65536, B * (ceil((S - 1) / page) + 1) <= 2^28.
 * One launch for up to 16384 pages and 1024 pages that the rows can touch, else two.
 */
int attn_pages_reserve(int32_t* page_table, int32_t* page_refs, const int32_t* positions,
                       const int32_t* lengths, void* k_pages, void* v_pages, int64_t page_stride,
                       int64_t head_stride, int64_t row_stride, int B, int S, int Hkv, int D,
                       int P, int page, int M, int32_t* taken, void* workspace,
                       size_t workspace_bytes, cudaStream_t stream);

/*
 * attn_pages_fork -- every sequence b becomes a copy of what sequence parents[b]
 * was before the call, cut to the pages of its first lengths[b] rows:
 *     table'[b][j] = table[parents[b]][j]  if j * page < lengths[b], else -1
 * with parents[b] = b for a sequence that stays and -1 for one that ends, and
 * page_refs follows the entries that change.  No row is copied: the sequences
 * share their pages (attn_pages_reserve parts them where rows are written).
 * Forks, reordered beams, dropped tokens and freed sequences are all this.
 *
 *   parents : [B] int32, or null: every sequence stays.
 *   lengths : [B] int32, or null: no sequence is cut; below 0 counts as 0.
 *   A parent outside -1 .. B - 1 leaves that sequence's pages in place (to be cut
 *   by lengths) and sets ATTN_DEV_BAD_PARENT.  Entries outside [0, P) count for
 *   no page.  Limits: B <= 4096 with parents, else 65536.
 */
int attn_pages_fork(int32_t* page_table, int32_t* page_refs, const int32_t* parents,
                    const int32_t* lengths, int B, int M, int P, int page, void* workspace,
                    size_t workspace_bytes, cudaStream_t stream);

/*
 * attn_pages_compact -- moves the n pages in use (page_refs > 0) to pages
 * 0 .. n - 1: the k-th of those at n or above goes to the k-th free page below
 * n, with its rows, its count and every table entry that names it.
 *
 *   page_map : [P] int32, written: where each page went (p for one that stayed),
 *              -1 for a free one: for page numbers kept elsewhere.
 *   Table entries outside [0, P) stay.  B * M may be 0.  One launch for a small pool
 *   (P up to 8192 and P * Hkv * page up to 786432 rows), else two.
 */
int attn_pages_compact(int32_t* page_table, int32_t* page_refs, void* k_pages, void* v_pages,
                       int64_t page_stride, int64_t head_stride, int64_t row_stride, int B,
                       int M, int Hkv, int D, int P, int page, int32_t* page_map, void* workspace,
                       size_t workspace_bytes, cudaStream_t stream);

/*
 * attn_prefill_causal -- causal prefill over a cached prefix (prefill page,
 * section "F.scaled_dot_product_attention"; decode page section 5: batch
 * prefill is causal).  New token i (absolute position start_pos + i) attends
 * keys 0..start_pos + i: the causal mask aligned to the bottom-right corner.
 *
 *   q         : [S, Hq, d] bf16, the S new tokens (token-major).
 *   k, v      : [start_pos + S, Hkv, d] bf16, cached prefix rows first.
 *   out       : [S, Hq, d] bf16 (= [S, Hq*d]).
 *
 * Supported: d == 64 or d == 128; g = Hq / Hkv >= 1; S >= 0 (S == 0 does nothing);
 * start_pos >= 0; start_pos + S < 2^31.  QK^T and PV run on the tcgen05
 * tensor cores (bf16 operands, fp32 accumulation in tensor memory).
 *
 * Every wait in the kernel is bounded: one that runs out ends the launch
 * early, leaves some output rows unwritten, and is counted on the device;
 * attn_read_prefill_status reads (and clears) that count.
 */
int attn_prefill_causal(const void* q, const void* k, const void* v,
                        int S, int start_pos, int Hq, int Hkv, int d, float scale,
                        void* out, cudaStream_t stream);

/*
 * attn_read_prefill_status -- synchronise `stream`, read into *timeouts the
 * number of prefill waits that gave up since the last call on this device,
 * clear it, and return ATTN_OK if there were none, ATTN_ERR_DEVICE if there
 * were, or ATTN_ERR_CUDA.  `timeouts` may be NULL.
 */
int attn_read_prefill_status(uint32_t* timeouts, cudaStream_t stream);

/*
 * attn_read_device_status -- synchronise `stream`, read the device status
 * word from a decode workspace into *bits (ATTN_DEV_* flags), clear it, and
 * return ATTN_OK if no bit was set, ATTN_ERR_DEVICE if one was, or
 * ATTN_ERR_INVALID_ARG / ATTN_ERR_CUDA.  `bits` may be NULL.
 */
int attn_read_device_status(void* workspace, uint32_t* bits, cudaStream_t stream);

/* Human-readable name of a status code (static string; never NULL). */
const char* attn_status_string(int status);

/* CUDA error code (cudaError_t as int) of the last ATTN_ERR_CUDA on this host
 * thread, 0 if none. */
int attn_last_cuda_error(void);

/*
 * attn_test_skip_tile -- for tests of the failure path only.  From the next
 * decode launch on, the bulk copy of tile `tile` (128 rows) of the first
 * (sequence, KV head) segment is never issued.  The waits for that tile
 * therefore run out: every wait in the kernels gives up
 * after 500 ms.  The kernel then sets ATTN_DEV_TIMEOUT in the workspace's
 * status word and returns, and the CUDA context stays usable; the outputs of
 * that launch are undefined, and its workspace must be zero-filled again
 * before reuse.  -1 (the default) turns this off.  Process-wide and not
 * thread-safe.
 * Errors: ATTN_ERR_INVALID_ARG for tile < -1.
 */
int attn_test_skip_tile(int tile);

/*
 * attn_test_force_schedule -- for tests of the split schedules only.  From
 * the next decode launch on, every segment (sequence, KV head) is split the
 * way `cluster` says instead of by the automatic choice: 0 = stream-K (all
 * tiles of all segments in one flat list over a persistent grid, split
 * segments merged through the workspace), C in 1..16 = cluster mode with
 * clusters of C CTAs (one cluster per segment, partials merged in rank 0's
 * shared memory), -1 (the default) = automatic.  Results agree with the
 * automatic choice up to the rounding of a different merge order.  A decode
 * call whose kernel cannot run clusters of C (too many landing slots for its
 * shared memory, or more than 8 where the device allows no larger clusters)
 * fails with ATTN_ERR_CUDA (cudaErrorNotSupported).  Process-wide and not
 * thread-safe.
 * Errors: ATTN_ERR_INVALID_ARG for cluster < -1 or > 16.
 */
int attn_test_force_schedule(int cluster);

/*
 * attn_debug_build -- 1 if this library was compiled with the device range
 * checks (-DGQA_DEBUG), else 0.  In such a build every decode kernel checks
 * the index-derived addresses named under ATTN_DEV_RANGE before it uses them,
 * both prefill kernels check their bulk-copy tile coordinates and output
 * rows, and the calls without a workspace (norm with rotation, 8-bit append,
 * block scores and selection) check the blocks, rows and list places that they
 * write; a failed check skips the access and records it (no trap, no assert).
 * Release builds contain no checks.
 */
int attn_debug_build(void);

/*
 * attn_read_prefill_skips -- synchronise `stream`, read into *skips the
 * number of prefill accesses that failed a range check since the last call on
 * this device, clear it, and return ATTN_OK if there were none,
 * ATTN_ERR_DEVICE if there were, or ATTN_ERR_CUDA.  Always 0 in release
 * builds.  `skips` may be NULL.
 */
int attn_read_prefill_skips(uint32_t* skips, cudaStream_t stream);

/*
 * attn_read_range_skips -- the same count for attn_qk_norm_rope,
 * attn_qk_norm_rope_append, attn_kv8_append, attn_block_scores,
 * attn_block_select and attn_paged_append, which have no status word.
 */
int attn_read_range_skips(uint32_t* skips, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GQA_ATTN_H */
