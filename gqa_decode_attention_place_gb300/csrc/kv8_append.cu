// kv8_append.cu -- new key and value rows into the 8-bit cache: e4m3 codes
// with one power-of-two scale per block of `block` tokens, KV head and
// operand, and (optionally) the channel bounds of each block's keys.
//
// For every block the append touches, over its new rows x (bf16):
//   s_new = 2^e, e the least integer with max|x| <= 448 * 2^e  (block_scale)
//   s     = max(s_old, s_new) if the block already held rows, else s_new
//   old rows (if s > s_old): code <- e4m3(code * s_old / s)
//   new rows:                code <- e4m3(x / s)     (x * (1/s): exact, s = 2^e; a
//                            block that came with another scale keeps that,
//                            1/s then rounded to fp32)
//   bounds: per channel, max and min of the new rows and, if the block
//           already held rows, of what was there.
//
// One CTA per (block, KV head), keys and values together: 16 rows of 16 lanes
// x 16 bytes per pass, all passes in registers, so the rows are read once and
// all in flight together; the maxima go through one block reduction.  Bound by
// memory for prompts (2 bytes read and 1 written per value): two of 8190
// tokens, 8 heads, 102 MB, take 18.5 us, 81% of the copy rate.  Single tokens
// are bound by latency and have a kernel of their own.
#include "fp8.cuh"
#include "internal.h"

namespace gqa {
namespace {

constexpr int kD8 = 128;
__device__ unsigned int g_append_skips;  // debug builds: accesses a range check skipped

__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2_min(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Largest finite magnitude of two bf16, as bf16 bits.
__device__ __forceinline__ uint32_t finite_abs_max(uint32_t w) {
  const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
  return max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u);
}

// Largest magnitudes of two pairs of bf16, half by half (as bits: NaN and
// infinities come out largest).
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t w) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(m), "r"(w & 0x7fff7fffu));
  return d;
}

// 8 codes moved to another scale: code <- e4m3(code * ratio).
__device__ __forceinline__ uint2 rescale8(uint2 w, float ratio) {
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = f16x2_to_f32x2(e4m3x2_to_f16x2(((k & 2) ? w.y : w.x) >> ((k & 1) * 16)));
    o[k] = f32x2_to_e4m3x2(f.x * ratio, f.y * ratio);
  }
  return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}
// 8 bf16 to codes: e4m3(x * inv).
__device__ __forceinline__ uint2 encode8(const uint4& x, float inv) {
  const uint32_t w4[4] = {x.x, x.y, x.z, x.w};
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = f32x2_to_e4m3x2(bf16lo(w4[k]) * inv, bf16hi(w4[k]) * inv);
  return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}

template <int P>  // passes of 16 rows: block = 16 * P
__global__ void __launch_bounds__(256) kv8_append_kernel(
    const uint4* __restrict__ k_new, const uint4* __restrict__ v_new, long long k_stride,
    long long v_stride, const int32_t* __restrict__ positions, uint8_t* k_cache,
    uint8_t* v_cache, float* k_scale, float* v_scale, uint32_t* k_bounds, int B, int S, int Hkv,
    int L, int nb) {
  constexpr int T = 16 * P;
  __shared__ uint32_t s_max[2][8];
  __shared__ uint32_t s_hi[8][64], s_lo[8][64];
  grid_dependency_wait();
  grid_dependents_launch();
  const int h = blockIdx.y, b = blockIdx.z;
  const int pos = positions[b];
  if (!rows_in_cache(pos, S - 1, L)) return;  // reported by the decode call
  const int j = pos / T + blockIdx.x;
  if (j > (pos + S - 1) / T) return;
  if (!range_ok_count(j >= 0 && j < nb && b < B && h < Hkv, &g_append_skips)) return;
  const int tid = threadIdx.x, c = tid & 15, warp = tid >> 5, lane = tid & 31;
  const size_t seg = (size_t)b * Hkv + h;
  const int row0 = j * T;
  const int t0 = row0 + (tid >> 4) - pos;  // new token of pass 0; 16 more each pass
  const bool had = row0 < pos;

  uint4 x[2][P];
#pragma unroll
  for (int op = 0; op < 2; ++op)
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int t = t0 + i * 16;
      x[op][i] = make_uint4(0u, 0u, 0u, 0u);
      if (t >= 0 && t < S)
        x[op][i] = (op ? v_new : k_new)[((long long)b * S + t) * (op ? v_stride : k_stride) +
                                        h * 16 + c];
    }
  float s_old[2] = {0.f, 0.f};
  if (had) {
    s_old[0] = k_scale[seg * nb + j];
    s_old[1] = v_scale[seg * nb + j];
  }
  // this thread's word of the block's bounds: 0..63 the maxima, 64..127 the minima
  uint32_t* bound = k_bounds + (seg * nb + j) * 128 + tid;
  const bool bounds = k_bounds != nullptr && tid < 128;
  const uint32_t was = bounds && had ? *bound : 0u;
  // The block's maxima, two halves of a word at a time.  That takes
  // infinities and NaN for the largest: where one turns up, the block looks
  // again, at finite values only.
#pragma unroll
  for (int op = 0; op < 2; ++op) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < P; ++i)
      m = abs_max2(abs_max2(abs_max2(abs_max2(m, x[op][i].x), x[op][i].y), x[op][i].z),
                   x[op][i].w);
    m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
    if (lane == 0) s_max[op][warp] = m;
  }
  if (k_bounds != nullptr) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      hi[w] = 0xff80ff80u;  // -inf, -inf
      lo[w] = 0x7f807f80u;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int t = t0 + i * 16;
      if (t >= 0 && t < S) {
        const uint32_t w4[4] = {x[0][i].x, x[0][i].y, x[0][i].z, x[0][i].w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          hi[w] = bf16x2_max(hi[w], w4[w]);
          lo[w] = bf16x2_min(lo[w], w4[w]);
        }
      }
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      hi[w] = bf16x2_max(hi[w], __shfl_xor_sync(0xffffffffu, hi[w], 16));
      lo[w] = bf16x2_min(lo[w], __shfl_xor_sync(0xffffffffu, lo[w], 16));
      if (lane < 16) {
        s_hi[warp][c * 4 + w] = hi[w];
        s_lo[warp][c * 4 + w] = lo[w];
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int op = 0; op < 2; ++op) {
    uint32_t amax = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) amax = max(amax, s_max[op][w]);
    if (amax >= 0x7f80u) {  // the same for the whole block
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < P; ++i)
        m = max(max(max(m, finite_abs_max(x[op][i].x)), max(finite_abs_max(x[op][i].y),
                finite_abs_max(x[op][i].z))), finite_abs_max(x[op][i].w));
      m = __reduce_max_sync(0xffffffffu, m);
      __syncthreads();  // every thread has read the maxima
      if (lane == 0) s_max[op][warp] = m;
      __syncthreads();
      amax = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) amax = max(amax, s_max[op][w]);
    }
    const float s_new = block_scale(__uint_as_float(amax << 16));
    const float s = had ? fmaxf(s_old[op], s_new) : s_new;
    // every thread's read of s_old came before the barrier
    if (tid == 0) (op ? v_scale : k_scale)[seg * nb + j] = s;
    const float inv = 1.f / s;
    uint8_t* cache = (op ? v_cache : k_cache) + seg * L * kD8;

    if (had && s > s_old[op]) {  // the block's scale grew: move the older rows
      const float ratio = s_old[op] * inv;
      for (int r = row0 + (tid >> 4); r < pos; r += 16) {
        if (!range_ok_count(r >= 0 && r < L, &g_append_skips)) continue;
        uint2* at = reinterpret_cast<uint2*>(cache + (size_t)r * kD8 + c * 8);
        *at = rescale8(*at, ratio);
      }
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int t = t0 + i * 16;
      if (t >= 0 && t < S && range_ok_count(t + pos >= 0 && t + pos < L, &g_append_skips)) {
        *reinterpret_cast<uint2*>(cache + (size_t)(t + pos) * kD8 + c * 8) = encode8(x[op][i], inv);
      }
    }
  }
  if (bounds) {
    const int w = tid & 63;
    uint32_t m = tid < 64 ? s_hi[0][w] : s_lo[0][w];
#pragma unroll
    for (int i = 1; i < 8; ++i)
      m = tid < 64 ? bf16x2_max(m, s_hi[i][w]) : bf16x2_min(m, s_lo[i][w]);
    if (had) m = tid < 64 ? bf16x2_max(m, was) : bf16x2_min(m, was);
    *bound = m;
  }
}

// One new token per sequence: a warp per (sequence, KV head), its lower half
// the key and its upper half the value (16 bytes a lane), no block barrier.
// The new rows are fetched before the position is read.  (64 sequences, 8 heads:
// 5.2 us by the kernel above, 1.7 us by this one.  That is while no scale grows:
// where one does, its half-warp moves the block's earlier rows four at a time.
// All 64 x 8 segments growing at once, eight rows before their block's end: 3.3
// us at blocks of 16, 21 at 64 and 68 at 128.)
constexpr int kTokenWarps = 4;
__global__ void __launch_bounds__(kTokenWarps * 32) kv8_append_token_kernel(
    const uint4* __restrict__ k_new, const uint4* __restrict__ v_new, long long k_stride,
    long long v_stride, const int32_t* __restrict__ positions, uint8_t* k_cache,
    uint8_t* v_cache, float* k_scale, float* v_scale, uint4* k_bounds, int segs, int Hkv, int L,
    int nb, int lb) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int seg = blockIdx.x * kTokenWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (seg >= segs) return;
  const int c = lane & 15;
  const bool op = lane >= 16;  // the value's half
  const int b = seg / Hkv, h = seg - b * Hkv;
  const uint4 x = (op ? v_new : k_new)[b * (op ? v_stride : k_stride) + h * 16 + c];
  const int pos = positions[b];
  if (!rows_in_cache(pos, 0, L)) return;  // reported by the decode call
  const int j = pos >> lb, row0 = j << lb;
  if (!range_ok_count(j >= 0 && j < nb && pos < L, &g_append_skips)) return;
  const bool had = row0 < pos;
  float* scale = (op ? v_scale : k_scale) + (size_t)seg * nb + j;
  const float s_old = had ? *scale : 0.f;
  // lower half: the maxima, upper half: the minima
  uint4* bound = k_bounds + ((size_t)seg * nb + j) * 32 + lane;
  uint4 was = make_uint4(0u, 0u, 0u, 0u);
  if (k_bounds != nullptr && had) was = *bound;

  uint32_t amax = max(max(finite_abs_max(x.x), finite_abs_max(x.y)),
                      max(finite_abs_max(x.z), finite_abs_max(x.w)));
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  const float s_new = block_scale(__uint_as_float(amax << 16));
  const float s = had ? fmaxf(s_old, s_new) : s_new;
  __syncwarp();  // every lane's read of s_old comes before the write
  if (c == 0) *scale = s;
  const float inv = 1.f / s;
  uint8_t* cache = (op ? v_cache : k_cache) + (size_t)seg * L * kD8 + c * 8;
  if (had && s > s_old) {  // the block's scale grew: move the older rows
    const float ratio = s_old * inv;
#pragma unroll 4
    for (int r = row0; r < pos; ++r) {
      uint2* at = reinterpret_cast<uint2*>(cache + (size_t)r * kD8);
      *at = rescale8(*at, ratio);
    }
  }
  *reinterpret_cast<uint2*>(cache + (size_t)pos * kD8) = encode8(x, inv);
  if (k_bounds != nullptr) {
    uint4 k = x;  // the key's dims, for both halves
    k.x = __shfl_sync(0xffffffffu, x.x, c);
    k.y = __shfl_sync(0xffffffffu, x.y, c);
    k.z = __shfl_sync(0xffffffffu, x.z, c);
    k.w = __shfl_sync(0xffffffffu, x.w, c);
    // a NaN leaves the bound as it is, and a first NaN the identity
    const uint32_t id = op ? 0x7f807f80u : 0xff80ff80u;
    if (!had) was = make_uint4(id, id, id, id);
    uint4 m;
    m.x = op ? bf16x2_min(k.x, was.x) : bf16x2_max(k.x, was.x);
    m.y = op ? bf16x2_min(k.y, was.y) : bf16x2_max(k.y, was.y);
    m.z = op ? bf16x2_min(k.z, was.z) : bf16x2_max(k.z, was.z);
    m.w = op ? bf16x2_min(k.w, was.w) : bf16x2_max(k.w, was.w);
    *bound = m;
  }
}

}  // namespace

cudaError_t kv8_append_read_skips(uint32_t* count) { return read_and_clear(g_append_skips, count); }

cudaError_t launch_kv8_append(const void* k_new, const void* v_new, long long k_stride,
                              long long v_stride, const int32_t* positions,
                              void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                              void* k_bounds, int B, int S, int Hkv, int L, int block,
                              cudaStream_t stream) {
  const int nb = (L + block - 1) / block;
  if (S == 1) {
    const int segs = B * Hkv;
    const int lb = block == 16 ? 4 : block == 32 ? 5 : block == 64 ? 6 : 7;
    return launch_pdl(kv8_append_token_kernel, dim3((segs + kTokenWarps - 1) / kTokenWarps),
                      dim3(kTokenWarps * 32), 0, stream, static_cast<const uint4*>(k_new),
                      static_cast<const uint4*>(v_new), k_stride / 8, v_stride / 8, positions,
                      static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache), k_scale,
                      v_scale, static_cast<uint4*>(k_bounds), segs, Hkv, L, nb, lb);
  }
  const int touched = min(nb, (S + block - 2) / block + 1);
  auto kernel = block == 16   ? kv8_append_kernel<1>
                : block == 32 ? kv8_append_kernel<2>
                : block == 64 ? kv8_append_kernel<4>
                              : kv8_append_kernel<8>;
  return launch_pdl(kernel, dim3(touched, Hkv, B), dim3(256), 0, stream,
                    static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new),
                    k_stride / 8, v_stride / 8, positions, static_cast<uint8_t*>(k_cache),
                    static_cast<uint8_t*>(v_cache), k_scale, v_scale,
                    static_cast<uint32_t*>(k_bounds), B, S, Hkv, L, nb);
}

}  // namespace gqa
