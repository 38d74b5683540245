// warp_ops.cuh -- warp-level pieces shared by the decode kernels: the bounded
// barrier among a block's consumer warps and their bounded wait for a tile,
// the CTA that holds a tile of the flat list, 8x8 transposes and byte
// permutes in registers, and the 128-byte swizzle of the tiled copies.
#pragma once

#include "common.cuh"

namespace gqa {
namespace {

// Barrier among the NW consumer warps.  It sits on an
// mbarrier (count NW, one arrival per warp from lane 0 once the warp's lanes
// have synced) so that its wait is bounded like every other: a named barrier
// has no time limit, and a warp that gave up on a tile after a timeout would
// leave the others waiting at one for ever.
struct ConsumerSync {
  uint32_t bar;
  volatile int* abort_flag;
  uint32_t* status;
  uint32_t n;  // completed phases
  __device__ __forceinline__ void operator()(int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    if (!mbar_wait(bar, n & 1u, abort_flag) && lane == 0) {
      *abort_flag = 1;
      set_status(status, ATTN_DEV_TIMEOUT);
    }
    ++n;
    __syncwarp();
  }
};

// CTA whose tile range [c*T/G, (c+1)*T/G) contains flat tile t.
__device__ __forceinline__ int cta_of(long long t, long long T, int G) {
  return (int)(((unsigned long long)(t + 1) * G + T - 1) / T) - 1;
}

// Transpose of an 8x8 matrix of 16-bit values held as one row pair per lane
// (lane 4r + c holds row r, columns 2c and 2c+1).
__device__ __forceinline__ uint32_t movm_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Bytes of a and b picked by `sel` (prmt): 0x5410 gives {a.lo, b.lo},
// 0x7632 gives {a.hi, b.hi}.
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

__device__ __forceinline__ uint4 lds128(const uint8_t* p) {
  return *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ uint32_t word(const uint4& u, int i) {
  return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
}
// Byte offset of row r, dims 8c..8c+7 within one 64-dim box of a tile, as the
// 128-byte swizzle of the tiled copy lays it out (16-byte chunk c of row r
// sits at chunk c ^ (r mod 8); the stage buffers are 1024-byte aligned).
__device__ __forceinline__ int sw128(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// A consumer warp's wait for a tile, with the outcome made warp-uniform (the
// tile math uses full-warp shuffles, so either every lane goes on or every
// lane leaves the loop).
__device__ __forceinline__ bool consumer_wait(uint32_t bar, uint32_t parity,
                                              volatile int* abort_flag, uint32_t* status,
                                              int lane) {
  if (__all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag))) return true;
  if (lane == 0) {
    *abort_flag = 1;
    set_status(status, ATTN_DEV_TIMEOUT);
  }
  return false;
}

}  // namespace
}  // namespace gqa
