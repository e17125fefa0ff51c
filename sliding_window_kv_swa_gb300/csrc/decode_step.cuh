// decode_step.cuh -- the staged 16-slot step of the int8 cache that a warp
// attends to: its layout in shared memory, its copies and loads, and the
// power-of-two scalings, shared by the decode kernel (decode.cu) and the
// shared-prefix decode's own part (shared_decode.cu).
#pragma once

#include "nd_common.cuh"

namespace nd {

constexpr int kStep = 16;         // slots per warp step (one MMA k-step)
constexpr float kLazyLog2 = 8.f;  // p is taken against a max at most 2^8 below the true one

template <int D>
struct Stage {
  static constexpr int kCodes = kStep * D;              // bytes of K (or V) codes per step
  static constexpr int kScales = kStep * (D / 32) * 4;  // bytes of K (or V) scales per step
  static constexpr int kBytes = 2 * kCodes + 2 * kScales;
};

__device__ __forceinline__ int ilog2_floor(float x) {  // x > 0, finite
  int e = int((__float_as_uint(x) >> 23) & 0xff) - 127;
  if (e == -127) e = -127 + (31 - __clz(__float_as_uint(x) & 0x7fffff)) - 22;  // subnormal
  return e;
}

// 2^e for e in [-126, 127]
__device__ __forceinline__ float exp2i(int e) {
  e = max(-126, min(127, e));
  return __uint_as_float(uint32_t(e + 127) << 23);
}

// Byte offset inside a stage: 16-byte chunks XOR-swizzled by the 128-byte
// line index, a bijection inside every 128-byte line.
__device__ __forceinline__ uint32_t swz(uint32_t a) { return a ^ (((a >> 7) & 7u) << 4); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float ldsf(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 lds128f(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

}  // namespace nd
