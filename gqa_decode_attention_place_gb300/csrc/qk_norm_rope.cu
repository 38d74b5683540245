// qk_norm_rope.cu -- RMS norm of every query and key head followed by the
// rotary embedding, in one pass, with the key and value rows written to the
// bf16 cache in the same launch when there is one.
//
// For a row x of D dims (one head of one token), weight w, and the rotation
// row (cos, sin) of the token's position:
//   y      = x * rsqrt(mean(x^2) + eps) * w
//   out[d] = y[d]*cos[d] - y[d+D/2]*sin[d]      for d <  D/2
//   out[d] = y[d]*cos[d] + y[d-D/2]*sin[d]      for d >= D/2
// all in fp32, rounded to bf16 once at the end.
//
// A lane holds dims 8c..8c+7 and their partners D/2 further on, so the
// rotation needs no exchange between lanes; the row's D/16 lanes (padded to
// a power of two) share only the sum of squares.  A warp stays with one
// token, so weight and rotation are multiplied into one set of factors (32
// values per lane) that serves every query head, and another every key head,
// the warp takes.  Bound by memory for prompts, by latency for single tokens.
// The heads come through a ring of asynchronous copies, private to each lane:
// with loads into registers too few bytes were under way (8191 tokens of
// 32 + 8 heads of 128: 35.4 us, 30.0 us this way; copying as many bytes takes
// 26).
#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace gqa {
namespace {

__device__ unsigned int g_norm_skips;  // debug builds: accesses a range check skipped

struct NormRopeParams {
  const uint16_t *q, *k, *v;
  long long q_stride, k_stride, v_stride;  // elements from token to token
  const uint16_t *q_weight, *k_weight;     // [D] or null (ones)
  const float *cos, *sin;                  // [L, D] or null (no rotation)
  const int32_t* positions;                // [B]; token t of sequence b sits at positions[b] + t
  uint16_t *q_out, *k_out;                 // k_out null: keys and values go to the caches
  uint8_t *k_cache, *v_cache;
  float eps;
  int N, S, Hq, Hkv, D, L;                 // N = B * S tokens
};

constexpr int kNormWarps = 4;
constexpr int kNormDepth = 4;  // steps whose copies are in flight

// Asynchronous 16-byte copy to shared memory, and the thread's own groups of them.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 8 bf16 as 4 packed fp32 pairs, and back.
__device__ __forceinline__ void unpack8(const uint4& u, f2 (&f)[4]) {
  f[0] = mk2(bf16lo(u.x), bf16hi(u.x));
  f[1] = mk2(bf16lo(u.y), bf16hi(u.y));
  f[2] = mk2(bf16lo(u.z), bf16hi(u.z));
  f[3] = mk2(bf16lo(u.w), bf16hi(u.w));
}
__device__ __forceinline__ uint32_t pack2(f2 x) {
  float lo, hi;
  brk2(x, lo, hi);
  return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ void load8f(const float* p, f2 (&f)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = mk2(a.x, a.y);
  f[1] = mk2(a.z, a.w);
  f[2] = mk2(b.x, b.y);
  f[3] = mk2(b.z, b.w);
}

// What a lane multiplies its dims x (first half) and y (second half) by, with
// weight and rotation in one factor (r: the row's 1/rms):
//   out x = r * (x * xx - y * yx),  out y = r * (y * yy + x * xy)
struct Coef {
  f2 xx[4], yx[4], yy[4], xy[4];
};

// LPR lanes per row (a power of two >= D/16).  A warp handles 32/LPR heads at
// a time, `steps` times, of one token.
template <int LPR>
__global__ void __launch_bounds__(kNormWarps * 32) qk_norm_rope_kernel(const NormRopeParams p,
                                                                       int warps_per_token,
                                                                       int steps) {
  constexpr int RPW = 32 / LPR;
  grid_dependency_wait();
  grid_dependents_launch();
  const int lane = threadIdx.x & 31;
  const long long gw = (long long)blockIdx.x * kNormWarps + (threadIdx.x >> 5);
  const long long n = gw / warps_per_token;
  if (n >= p.N) return;
  const int part = (int)(gw % warps_per_token);
  const int c = lane % LPR, D = p.D, half = D >> 1;
  const bool on = c * 16 < D;  // lanes past D/16 only take part in the shuffles
  const int d0 = c * 8;
  const int heads = p.Hq + p.Hkv * (p.k_out ? 1 : 2);
  const int head0 = part * steps * RPW + lane / LPR;
  // This lane's two pieces of a head (zeros past the last head) into its own
  // places of the ring: no other lane reads them, so the lane's own wait for
  // its copies is all the synchronisation there is.
  __shared__ uint4 ring[kNormDepth][2][kNormWarps * 32];
  auto fetch = [&](int st) {
    const int head = head0 + st * RPW, s = st % kNormDepth;
    if (st >= steps || !on || head >= heads) {
      ring[s][0][threadIdx.x] = ring[s][1][threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
      return;
    }
    const bool is_q = head < p.Hq, is_v = head >= p.Hq + p.Hkv;
    const uint16_t* src = is_q   ? p.q + n * p.q_stride + (size_t)head * D
                          : is_v ? p.v + n * p.v_stride + (size_t)(head - p.Hq - p.Hkv) * D
                                 : p.k + n * p.k_stride + (size_t)(head - p.Hq) * D;
    copy16(smem_u32(&ring[s][0][threadIdx.x]), src + d0);
    copy16(smem_u32(&ring[s][1][threadIdx.x]), src + d0 + half);
  };
  // The first copies go out before the position is read: the rotation row's
  // address hangs on it, the heads' do not.
#pragma unroll
  for (int st = 0; st < kNormDepth - 1; ++st) {
    fetch(st);
    copy_commit();
  }
  const int b = (int)(n / p.S), t = (int)(n % p.S);
  const int pos0 = p.positions[b];
  const bool ok = rows_in_cache(pos0, p.S - 1, p.L);
  const int pos = pos0 + t;
  const float inv_d = 1.f / (float)D;
  Coef cf;
  int kind = -1;  // of cf: 0 queries, 1 keys
  for (int st = 0; st < steps; ++st) {
    const int head = head0 + st * RPW;
    fetch(st + kNormDepth - 1);  // into the place that the step before has used up
    copy_commit();
    copy_wait<kNormDepth - 1>();
    uint4 ua = ring[st % kNormDepth][0][threadIdx.x], ub = ring[st % kNormDepth][1][threadIdx.x];
    const bool row_on = on && head < heads;
    const bool is_q = head < p.Hq, is_v = head >= p.Hq + p.Hkv;
    const int h = is_q ? head : is_v ? head - p.Hq - p.Hkv : head - p.Hq;
    f2 xa[4], xb[4];
    unpack8(ua, xa);
    unpack8(ub, xb);
    f2 s2 = mul2(xa[0], xa[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) s2 = fma2(xa[i], xa[i], s2);
#pragma unroll
    for (int i = 0; i < 4; ++i) s2 = fma2(xb[i], xb[i], s2);
    float s_lo, s_hi;
    brk2(s2, s_lo, s_hi);
    float ss = s_lo + s_hi;
#pragma unroll
    for (int off = 1; off < LPR; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    if (!row_on) continue;
    if (!is_v) {
      if (kind != (is_q ? 0 : 1)) {  // at the first head, and from queries to keys
        kind = is_q ? 0 : 1;
        const float one = ok ? 1.f : __uint_as_float(0x7fffffffu);  // bad position: NaN rows
        f2 wa[4], wb[4], ca[4], cb[4], sa[4], sb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          wa[i] = wb[i] = ca[i] = cb[i] = mk2(one, one);
          sa[i] = sb[i] = mk2(0.f, 0.f);
        }
        const uint16_t* w = is_q ? p.q_weight : p.k_weight;
        if (w) {
          unpack8(*reinterpret_cast<const uint4*>(w + d0), wa);
          unpack8(*reinterpret_cast<const uint4*>(w + d0 + half), wb);
        }
        if (p.cos && ok && range_ok_count(pos >= 0 && pos < p.L, &g_norm_skips)) {
          const size_t row = (size_t)pos * D + d0;
          load8f(p.cos + row, ca);
          load8f(p.cos + row + half, cb);
          load8f(p.sin + row, sa);
          load8f(p.sin + row + half, sb);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          cf.xx[i] = mul2(wa[i], ca[i]);
          cf.yx[i] = mul2(wb[i], mul2(sa[i], mk2(-1.f, -1.f)));
          cf.yy[i] = mul2(wb[i], cb[i]);
          cf.xy[i] = mul2(wa[i], sb[i]);
        }
      }
      const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
      const f2 r2 = mk2(r, r);
      uint32_t oa[4], ob[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        oa[i] = pack2(mul2(r2, fma2(xb[i], cf.yx[i], mul2(xa[i], cf.xx[i]))));
        ob[i] = pack2(mul2(r2, fma2(xa[i], cf.xy[i], mul2(xb[i], cf.yy[i]))));
      }
      ua = make_uint4(oa[0], oa[1], oa[2], oa[3]);
      ub = make_uint4(ob[0], ob[1], ob[2], ob[3]);
    }
    if (!range_ok_count(n >= 0 && n < p.N && h >= 0 && h < (is_q ? p.Hq : p.Hkv) &&
                            (!ok || (pos >= 0 && pos < p.L)),
                        &g_norm_skips))
      continue;
    uint16_t* dst;
    if (is_q) {
      dst = p.q_out + ((size_t)n * p.Hq + h) * D;
    } else if (p.k_out) {
      dst = p.k_out + ((size_t)n * p.Hkv + h) * D;
    } else {
      if (!ok) continue;  // nothing of this sequence is written to the cache
      dst = reinterpret_cast<uint16_t*>(is_v ? p.v_cache : p.k_cache) +
            (((size_t)b * p.Hkv + h) * p.L + pos) * D;
    }
    *reinterpret_cast<uint4*>(dst + d0) = ua;
    *reinterpret_cast<uint4*>(dst + d0 + half) = ub;
  }
}

// The current device's SMs, asked for once.
cudaError_t sm_count(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev < 0 || dev >= 64)) e = cudaErrorInvalidDevice;
  if (e != cudaSuccess) return e;
  *sms = known[dev].load(std::memory_order_relaxed);
  if (*sms == 0) {
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) known[dev].store(*sms, std::memory_order_relaxed);
  }
  return e;
}

}  // namespace

cudaError_t qk_norm_read_skips(uint32_t* count) { return read_and_clear(g_norm_skips, count); }

cudaError_t launch_qk_norm_rope(const void* q, const void* k, const void* v, long long q_stride,
                                long long k_stride, long long v_stride, const void* q_weight,
                                const void* k_weight, float eps, const float* cos,
                                const float* sin, const int32_t* positions, int B, int S, int Hq,
                                int Hkv, int D, int L, void* q_out, void* k_out, void* k_cache,
                                void* v_cache, cudaStream_t stream) {
  NormRopeParams p;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_weight = static_cast<const uint16_t*>(q_weight);
  p.k_weight = static_cast<const uint16_t*>(k_weight);
  p.cos = cos;
  p.sin = sin;
  p.positions = positions;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_out = static_cast<uint16_t*>(k_out);
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.eps = eps;
  p.N = B * S;
  p.S = S;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.L = L;
  int lpr = 1;
  while (lpr * 16 < D) lpr *= 2;
  const int rpw = 32 / lpr;
  const int all = (Hq + Hkv * (k_out ? 1 : 2) + rpw - 1) / rpw;  // steps of one warp for a token
  // Few tokens: a warp for every step, for latency.  Many: a warp keeps its
  // token's rotation row over several steps, as long as 24 warps are left for
  // every SM.  (20 are resident at 96 registers.  Of 16, 20, 24, 28 and 32 none
  // is best for every count: 32 + 8 heads of 128, 650 tokens 6.1 us with 20
  // and 7.1 with 24, 1100 tokens 8.3 and 7.7, 1600 tokens 11.2 and 9.8.)
  int sms = 0;
  if (const cudaError_t e = sm_count(&sms)) return e;
  const long long full = 24ll * sms;
  int steps = 1;
  while (steps < all && (long long)p.N * ((all + 2 * steps - 1) / (2 * steps)) >= full) steps *= 2;
  steps = min(steps, all);
  const int wpt = (all + steps - 1) / steps;
  const long long blocks = ((long long)p.N * wpt + kNormWarps - 1) / kNormWarps;
  auto kernel = lpr == 1   ? qk_norm_rope_kernel<1>
                : lpr == 2 ? qk_norm_rope_kernel<2>
                : lpr == 4 ? qk_norm_rope_kernel<4>
                : lpr == 8 ? qk_norm_rope_kernel<8>
                           : qk_norm_rope_kernel<16>;
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kNormWarps * 32), 0, stream, p, wpt,
                    steps);
}

}  // namespace gqa
