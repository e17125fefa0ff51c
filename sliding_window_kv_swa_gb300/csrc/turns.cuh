// turns.cuh -- rotation angles as fractions of a turn, and the small loads that
// the row kernels of qk_norm.cu and rope_positions.cu share.
//
// The fraction of a turn that position p makes, p * freq / (2 pi) mod 1, is one
// 64-bit integer product: the host scales freq / (2 pi) to 2^64 and the
// wrap-around of the multiply is the reduction.  Its upper 32 bits give the
// angle to 2^-32 of a turn at any 32-bit position (the fp64 frequency itself
// limits that to 2^-53 p turns); as the fp32 argument of sincospif it keeps 24
// bits of up to half a turn, so it is within 2^-26 of a turn, 9.4e-8 radians: a
// rounding or two more of the fp32 result.  The pair of a 64-bit multiply and
// sincospif costs no fp64 instruction, of which this part issues two per clock
// and SM.
#pragma once

#include <math.h>

#include "nd_common.cuh"
#include "nd_internal.h"

namespace nd {

// freq_i / (2 pi) mod 1, in units of 2^-64
struct Turns {
  unsigned long long f[kMaxHalf];
};

inline unsigned long long turn_of(double freq) {
  double turn = freq * 0.15915494309189533576888376337251;
  turn -= floor(turn);
  // turn < 1, so the product is below 2^64 (it may only reach it by the
  // rounding of the subtraction above, where the wrap to 0 is the same angle)
  const double scaled = turn * 18446744073709551616.0;
  return scaled >= 18446744073709551616.0 ? 0ull : (unsigned long long)scaled;
}

__device__ __forceinline__ float2 turn_cs(int pos, unsigned long long f) {
  const long long turn = (long long)((unsigned long long)(long long)pos * f);
  float s, c;
  sincospif(float(int(turn >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
  return make_float2(c, s);
}

// The CTA's copy of the frequencies: indexed by lane, kernel parameters are
// read one address at a time.
template <int D>
__device__ __forceinline__ void stage_turns(const Turns &t, unsigned long long *s_f) {
  for (int i = threadIdx.x; i < D / 2; i += blockDim.x) s_f[i] = t.f[i];
  __syncthreads();
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

}  // namespace nd
