// decode_step.cuh -- one warp's attention over staged 16-slot steps of the int8
// cache: shared by the decode kernel (decode.cu) and the shared-prefix decode's
// own part (shared_decode.cu).
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
// The NG group scales of one slot, which sit together in the stage (16 or 8
// bytes).  At head_dim 128 one 16-byte load replaces four 4-byte loads for
// each of the eight K and V scale rows a thread reads per step (the kernel
// is issue-bound there: 4-5 points of HBM at B128-B512); at head_dim 64 the
// two 4-byte loads stay, since the 8-byte form adds a spill to the 96-register
// builds.
template <int NG>
__device__ __forceinline__ void lds_scales(uint32_t a, float *s) {
  if constexpr (NG == 4) {
    const float4 v = lds128f(a);
    s[0] = v.x, s[1] = v.y, s[2] = v.z, s[3] = v.w;
  } else {
    s[0] = ldsf(a);
    s[1] = ldsf(a + 4);
  }
}

// One warp's attention over 16-slot steps (thread (g, t) = (lane / 4, lane % 4)).
// Query fragments of heads g: channels as fp16, pre-scaled by 2^Eq.
template <int D>
struct HeadQ {
  uint32_t qa[D / 32][2][2];
  float coef;  // 2^-Eq * log2(e) / sqrt(D), for head g
};

// w: thread t's channels 32*grp + 8t .. +7 of head g, bf16
template <int D>
__device__ __forceinline__ void make_q(const uint4 (&w)[D / 32], HeadQ<D> &hq) {
  constexpr int NG = D / 32;
  float qm = 0.f;
#pragma unroll
  for (int grp = 0; grp < NG; ++grp) {
    const uint32_t ws[4] = {w[grp].x, w[grp].y, w[grp].z, w[grp].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) qm = fmaxf(qm, fmaxf(fabsf(bf16_lo(ws[i])), fabsf(bf16_hi(ws[i]))));
  }
  qm = fmaxf(qm, __shfl_xor_sync(0xffffffffu, qm, 1));
  qm = fmaxf(qm, __shfl_xor_sync(0xffffffffu, qm, 2));
  const int eq = qm > 0.f ? 14 - ilog2_floor(qm) : 0;
  const float up = exp2i(eq);
  hq.coef = exp2i(-eq) * (1.4426950408889634f * rsqrtf(float(D)));
#pragma unroll
  for (int grp = 0; grp < NG; ++grp) {
    const uint32_t ws[4] = {w[grp].x, w[grp].y, w[grp].z, w[grp].w};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      hq.qa[grp][s][0] = pack_half2(bf16_lo(ws[2 * s]) * up, bf16_hi(ws[2 * s]) * up);
      hq.qa[grp][s][1] = pack_half2(bf16_lo(ws[2 * s + 1]) * up, bf16_hi(ws[2 * s + 1]) * up);
    }
  }
}

template <int D>
struct RunState {
  float o[D / 32][2][4];  // heads 2t, 2t+1; channels 32*grp + 4g + 2*tile (+1)
  float m = -INFINITY, l = 0.f;  // m: the max p is taken against (log2 units); l: this thread's share
  int e = 127;                   // power-of-two pre-scale of P' (never increases; 127 = unset)
  __device__ __forceinline__ RunState() { reset(); }
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int grp = 0; grp < D / 32; ++grp)
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[grp][tt][i] = 0.f;
    m = -INFINITY;
    l = 0.f;
    e = 127;
  }
};

// One step staged at st: vis[i] says whether this thread's slot col[i] counts.
template <int D>
__device__ __forceinline__ void attend_step(uint32_t st, const HeadQ<D> &hq, const bool (&vis)[4], bool head_ok,
                                            int lane, RunState<D> &r) {
  constexpr int NG = D / 32;
  using S = Stage<D>;
  const int g = lane >> 2, t = lane & 3;
  const int col[4] = {2 * t, 2 * t + 1, 8 + 2 * t, 9 + 2 * t};
  // ---- QK: scores for head g at columns 2t, 2t+1 of tiles 0 and 1
  float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int row = 8 * j + g;
    float ks0[NG], ks1[NG];  // K scales of this thread's two columns
    lds_scales<NG>(st + 2 * S::kCodes + (8 * j + 2 * t) * NG * 4, ks0);
    lds_scales<NG>(st + 2 * S::kCodes + (8 * j + 2 * t + 1) * NG * 4, ks1);
#pragma unroll
    for (int grp = 0; grp < NG; ++grp) {
      const uint2 kw = lds64(st + swz(uint32_t(row * D + 32 * grp + 8 * t)));
      float d0 = 0.f, d1 = 0.f, d2 = 0.f, d3 = 0.f;
      const uint32_t w0 = kw.x ^ 0x80808080u, w1 = kw.y ^ 0x80808080u;
      mma_f16_16816(d0, d1, d2, d3, hq.qa[grp][0][0], 0u, hq.qa[grp][0][1], 0u,
                    codes_to_half2(w0, kSelBytes01), codes_to_half2(w0, kSelBytes23));
      mma_f16_16816(d0, d1, d2, d3, hq.qa[grp][1][0], 0u, hq.qa[grp][1][1], 0u,
                    codes_to_half2(w1, kSelBytes01), codes_to_half2(w1, kSelBytes23));
      sc[2 * j] = fmaf(ks0[grp], d0, sc[2 * j]);
      sc[2 * j + 1] = fmaf(ks1[grp], d1, sc[2 * j + 1]);
    }
  }
  // ---- online softmax for head g (log2 domain)
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sc[i] = (vis[i] && head_ok) ? sc[i] * hq.coef : -INFINITY;
    mx = fmaxf(mx, sc[i]);
  }
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  // lazy max: p is taken against r.m, which moves (and O is rescaled)
  // only when a score exceeds it by more than 2^kLazyLog2, so p <= 2^8
  const bool need = mx > r.m + kLazyLog2;
  const float m_new = need ? mx : r.m;
  const float alpha = need ? (r.m == -INFINITY ? 0.f : ex2(r.m - m_new)) : 1.f;
  float pr[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) pr[i] = (m_new == -INFINITY) ? 0.f : ex2(sc[i] - m_new);
  r.l = r.l * alpha + (pr[0] + pr[1]) + (pr[2] + pr[3]);
  r.m = m_new;
  // V scales of the step, and one exponent for all groups that keeps
  // p * v_scale * 2^e below 2^15 (p <= 2^8); the accumulator keeps the
  // smallest exponent seen so far
  float vsc[NG][4];
  float vm = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float vs_i[NG];
    lds_scales<NG>(st + 2 * S::kCodes + S::kScales + col[i] * NG * 4, vs_i);
#pragma unroll
    for (int grp = 0; grp < NG; ++grp) vsc[grp][i] = vs_i[grp];
  }
#pragma unroll
  for (int grp = 0; grp < NG; ++grp)
#pragma unroll
    for (int i = 0; i < 4; ++i) vm = fmaxf(vm, vis[i] ? vsc[grp][i] : 0.f);
  vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, 1));
  vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, 2));
  const int e_step = vm > 0.f ? 14 - int(kLazyLog2) - ilog2_floor(vm) : 127;
  const bool shrink_e = e_step < r.e;
  // rescale O (this thread's columns are heads 2t and 2t+1) only when a
  // head's max moved or the exponent shrank: warp-uniform, and rare
  if (__any_sync(0xffffffffu, need || shrink_e)) {
    const float shrink = shrink_e ? (r.e == 127 ? 0.f : exp2i(e_step - r.e)) : 1.f;
    const float f_lo = __shfl_sync(0xffffffffu, alpha, (2 * t) * 4) * shrink;
    const float f_hi = __shfl_sync(0xffffffffu, alpha, (2 * t + 1) * 4) * shrink;
#pragma unroll
    for (int grp = 0; grp < NG; ++grp)
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        r.o[grp][tt][0] *= f_lo;
        r.o[grp][tt][1] *= f_hi;
        r.o[grp][tt][2] *= f_lo;
        r.o[grp][tt][3] *= f_hi;
      }
    if (shrink_e) r.e = e_step;
  }
  // (while no scale has been seen, every visible scale is 0 and u is moot)
  const float u = r.e == 127 ? 1.f : exp2i(r.e);
  float pu[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) pu[i] = vis[i] ? pr[i] * u : 0.f;
  // ---- PV per group: B = P'^T (slot x head), A = V^T (channel x slot)
#pragma unroll
  for (int grp = 0; grp < NG; ++grp) {
    // masked slots contribute 0 (their scale may be anything, even non-finite)
    const uint32_t b0 = pack_half2(vis[0] ? pu[0] * vsc[grp][0] : 0.f, vis[1] ? pu[1] * vsc[grp][1] : 0.f);
    const uint32_t b1 = pack_half2(vis[2] ? pu[2] * vsc[grp][2] : 0.f, vis[3] ? pu[3] * vsc[grp][3] : 0.f);
    uint32_t vw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      vw[i] = lds32(st + S::kCodes + swz(uint32_t(col[i] * D + 32 * grp + 4 * g)));
    const uint32_t x01 = prmt(vw[0], vw[1], 0x5140u) ^ 0x80808080u;
    const uint32_t x23 = prmt(vw[0], vw[1], 0x7362u) ^ 0x80808080u;
    const uint32_t y01 = prmt(vw[2], vw[3], 0x5140u) ^ 0x80808080u;
    const uint32_t y23 = prmt(vw[2], vw[3], 0x7362u) ^ 0x80808080u;
    // tile 0: rows g <-> channel 4g, rows g+8 <-> channel 4g+1
    mma_f16_16816(r.o[grp][0][0], r.o[grp][0][1], r.o[grp][0][2], r.o[grp][0][3],
                  codes_to_half2(x01, kSelBytes01), codes_to_half2(x01, kSelBytes23),
                  codes_to_half2(y01, kSelBytes01), codes_to_half2(y01, kSelBytes23), b0, b1);
    // tile 1: rows g <-> channel 4g+2, rows g+8 <-> channel 4g+3
    mma_f16_16816(r.o[grp][1][0], r.o[grp][1][1], r.o[grp][1][2], r.o[grp][1][3],
                  codes_to_half2(x23, kSelBytes01), codes_to_half2(x23, kSelBytes23),
                  codes_to_half2(y23, kSelBytes01), codes_to_half2(y23, kSelBytes23), b0, b1);
  }
}

// The warp's (max, sum, O) of its up to eight heads: o [8][D], m [8], l [8].
template <int D>
__device__ __forceinline__ void store_state(RunState<D> &r, int lane, float *o, float *m, float *l) {
  const int g = lane >> 2, t = lane & 3;
  r.l += __shfl_xor_sync(0xffffffffu, r.l, 1);
  r.l += __shfl_xor_sync(0xffffffffu, r.l, 2);
  if (t == 0) {
    m[g] = r.m;
    l[g] = r.l;
  }
  const float down = r.e == 127 ? 0.f : exp2i(-r.e);
  float *w0 = o + (2 * t) * D, *w1 = o + (2 * t + 1) * D;
#pragma unroll
  for (int grp = 0; grp < D / 32; ++grp) {
#pragma unroll
    for (int tt = 0; tt < 2; ++tt) {
      const int ch0 = 32 * grp + 4 * g + 2 * tt;  // row g; row g+8 is ch0 + 1
      w0[ch0] = r.o[grp][tt][0] * down;
      w1[ch0] = r.o[grp][tt][1] * down;
      w0[ch0 + 1] = r.o[grp][tt][2] * down;
      w1[ch0 + 1] = r.o[grp][tt][3] * down;
    }
  }
}

}  // namespace nd
