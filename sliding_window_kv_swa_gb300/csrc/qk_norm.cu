// qk_norm.cu -- RMS norm of each query and key head with the rotary embedding
// in the same pass: over a prefill's tokens, and for one decode token per
// sequence whose key and value are quantised into the cache as they are made.
//
// One row x (a head of a token, D channels, at position p):
//   y = x * rsqrt(mean(x^2) + eps) * w        (w = 1 when no weight is given)
//   z_i       = y_i cos a_i - y_{i+D/2} sin a_i
//   z_{i+D/2} = y_{i+D/2} cos a_i + y_i sin a_i,   a_i = p theta^(-2i/D)
// in fp32 from the load to the store, rounded once.
//
// Work split: D/16 lanes hold a row, lane j the channels 8j..8j+7 and their
// rotation partners D/2 + 8j..; the norm's sum is then log2(D/16) shuffles
// and the rotation stays inside the lane.
//
// Angles: the fraction of a turn that position p makes, p * freq / (2 pi) mod
// 1, is one 64-bit integer product: the host scales freq / (2 pi) to 2^64 and
// the wrap-around of the multiply is the reduction.  Its upper 32 bits give
// the angle to 2^-32 of a turn at any 32-bit position (the fp64 frequency
// itself limits that to 2^-53 p turns); the pair of a 64-bit multiply and
// sincospif costs no fp64 instruction, of which this part issues two per
// clock and SM.
#include "nd_common.cuh"
#include "nd_internal.h"

#include <math.h>

#include <atomic>

namespace nd {

namespace {

// freq_i / (2 pi) mod 1, in units of 2^-64
struct Turns {
  unsigned long long f[kMaxHalf];
};

// The table of a model's head_dim and theta, kept per host thread: building it
// takes a pow per channel pair, about as long as a decode step's kernel.
const Turns &make_turns(int head_dim, float theta) {
  static thread_local Turns t;
  static thread_local int t_dim = 0;
  static thread_local float t_theta = 0.f;
  if (t_dim == head_dim && t_theta == theta) return t;
  const Freqs fr = make_freqs(head_dim, theta);
  for (int i = 0; i < kMaxHalf; ++i) {
    double turn = 0.0;
    if (theta != 0.f && i < head_dim / 2) {
      turn = fr.f[i] * 0.15915494309189533576888376337251;
      turn -= floor(turn);
    }
    // turn < 1, so the product is below 2^64 (it may only reach it by the
    // rounding of the subtraction above, where the wrap to 0 is the same angle)
    const double scaled = turn * 18446744073709551616.0;
    t.f[i] = scaled >= 18446744073709551616.0 ? 0ull : (unsigned long long)scaled;
  }
  t_dim = head_dim;
  t_theta = theta;
  return t;
}

__device__ __forceinline__ float2 turn_cs(int pos, unsigned long long f) {
  const long long turn = (long long)((unsigned long long)(long long)pos * f);
  float s, c;
  sincospif(float(int(turn >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
  return make_float2(c, s);
}

// Eight channels as loaded (bf16: one uint4, fp32: two) and as fp32.
template <typename E>
struct Raw8 {
  uint4 w[sizeof(E) / 2];
  __device__ __forceinline__ void load(const E *p) {
#pragma unroll
    for (int i = 0; i < int(sizeof(E) / 2); ++i) w[i] = reinterpret_cast<const uint4 *>(p)[i];
  }
  __device__ __forceinline__ void get(float *x) const {
    if constexpr (sizeof(E) == 2) {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(u[i]), x[2 * i + 1] = bf16_hi(u[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        x[4 * i] = __uint_as_float(w[i].x), x[4 * i + 1] = __uint_as_float(w[i].y),
              x[4 * i + 2] = __uint_as_float(w[i].z), x[4 * i + 3] = __uint_as_float(w[i].w);
    }
  }
};
template <typename E>
__device__ __forceinline__ void ld8(const E *p, float *x) {
  Raw8<E> r;
  r.load(p);
  r.get(x);
}
__device__ __forceinline__ void st8(uint16_t *p, const float *x) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                             pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void st8(float *p, const float *x) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// The eight angles of a lane's channel pairs i0 .. i0 + 7.  The lanes that hold
// the same pairs of other rows make an eighth to a half of them each.
template <int D>
__device__ __forceinline__ void lane_angles(int pos, const unsigned long long *f, int lane, float2 *cs) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes, kPer = kRows >= 8 ? 1 : 8 / kRows;
  float2 mine[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) mine[j] = turn_cs(pos, f[j]);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int src = (e / kPer) * kLanes + lane % kLanes;
    cs[e].x = __shfl_sync(0xffffffffu, mine[e % kPer].x, src);
    cs[e].y = __shfl_sync(0xffffffffu, mine[e % kPer].y, src);
  }
}
// the frequencies of the angles that this lane makes
template <int D>
__device__ __forceinline__ void lane_freqs(const Turns &t, int lane, unsigned long long *f) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes, kPer = kRows >= 8 ? 1 : 8 / kRows;
  const int i0 = 8 * (lane % kLanes), e0 = (lane / kLanes) * kPer % 8;
#pragma unroll
  for (int j = 0; j < kPer; ++j) f[j] = t.f[i0 + e0 + j];
}

// The row held by D/16 neighbouring lanes: this lane's lo (channels i0..i0+7)
// and hi (D/2 + i0..) become the normalised, rotated row.  Every lane of the
// warp calls this (the sum is a shuffle).
template <int D>
__device__ __forceinline__ void norm_rotate(float *lo, float *hi, const float *wlo, const float *whi,
                                            const float2 *cs, float eps) {
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss = fmaf(lo[e], lo[e], fmaf(hi[e], hi[e], ss));
#pragma unroll
  for (int off = D / 32; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  const float r = __frsqrt_rn(fmaf(ss, 1.f / D, eps));
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a = lo[e] * r * wlo[e], b = hi[e] * r * whi[e];
    rope_pair(a, b, cs[e].x, cs[e].y, lo[e], hi[e]);
  }
}

template <typename E>
struct NormRopeParams {
  const E *x[2];       // q, k
  E *y[2];
  const float *w[2];   // NULL: ones
  int H[2];
  int64_t stride[2];   // elements from one token to the next in x
  int T, tokens;
  float eps;
  const int32_t *pos;
  Turns turns;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

// A warp takes tokens with the stride of the grid, each as batches of rows (kU
// * 32 / (D / 16) heads of q, then of k).  HBM-bound: a row in and a row out;
// what it needs is loads in flight, so each lane copies its own channels kSt -
// 1 batches ahead into a ring in shared memory (its own slots: nothing to
// exchange, no barrier), across the end of a token, while the angles -- once
// per token for all its heads -- and the batches before are computed.
// At 32768 tokens of 32 + 8 heads of 128 (671 MB): 133 us with plain loads
// behind the angles, 120 with one batch ahead in registers.
template <typename E, int D>
struct NormLay {
  static constexpr int kLanes = D / 16, kRows = 32 / kLanes;
  static constexpr int kU = sizeof(E) == 2 ? 2 : 1, kBatch = kU * kRows;
  static constexpr int kSt = 6, kStage = kU * kRows * D * int(sizeof(E));  // 2 KB
  static constexpr int kWarps = 4, kBytes = kWarps * kSt * kStage;
};

template <typename E, int D>
__global__ void __launch_bounds__(128, 4) qk_norm_rope_kernel(const __grid_constant__ NormRopeParams<E> p) {
  using Y = NormLay<E, D>;
  constexpr int kLanes = Y::kLanes, kRows = Y::kRows, kU = Y::kU, kSt = Y::kSt, kVec = sizeof(E) / 2;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i0 = 8 * (lane % kLanes), sub = lane / kLanes;
  // a lane's slots: 16 bytes each, 512 apart
  const uint32_t mine = smem_u32(smem) + warp * kSt * Y::kStage + lane * 16;
  unsigned long long f[8];
  lane_freqs<D>(p.turns, lane, f);
  const int stride = gridDim.x * Y::kWarps;
  pdl_wait();

  // the copies' cursor: a token, q (0) or k (1), the batch's first head
  int c_tok = blockIdx.x * Y::kWarps + warp, c_which = p.H[0] > 0 ? 0 : 1, c_h = 0, in = 0;
  auto issue = [&]() {
    if (c_tok < p.tokens) {
      const int H = c_which ? p.H[1] : p.H[0];
      const E *x = (c_which ? p.x[1] : p.x[0]) + c_tok * (c_which ? p.stride[1] : p.stride[0]) + i0;
      const uint32_t dst = mine + in * Y::kStage;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const E *row = x + min(c_h + u * kRows + sub, H - 1) * D;  // past the end: the last head, not stored
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          copy16(dst + (u * 2 * kVec + j) * 512, row + j * (16 / sizeof(E)));
          copy16(dst + (u * 2 * kVec + kVec + j) * 512, row + D / 2 + j * (16 / sizeof(E)));
        }
      }
      if (++in == kSt) in = 0;
      c_h += Y::kBatch;
      if (c_h >= H) {
        c_h = 0;
        if (c_which == 0 && p.H[1] > 0) {
          c_which = 1;
        } else {
          c_which = p.H[0] > 0 ? 0 : 1;
          c_tok += stride;
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kSt - 1; ++i) issue();

  int tok = blockIdx.x * Y::kWarps + warp, out = 0;
  auto position = [&](int t) { return p.pos ? p.pos[t] : t % p.T; };
  int pos = tok < p.tokens ? position(tok) : 0;
  for (; tok < p.tokens; tok += stride) {
    float2 cs[8];
    lane_angles<D>(pos, f, lane, cs);
    if (tok + stride < p.tokens) pos = position(tok + stride);
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const int H = which ? p.H[1] : p.H[0];
      const float *w = which ? p.w[1] : p.w[0];
      float wlo[8], whi[8];
      if (w) {
        ld8(w + i0, wlo);
        ld8(w + D / 2 + i0, whi);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) wlo[e] = whi[e] = 1.f;
      }
      E *y = (which ? p.y[1] : p.y[0]) + int64_t(tok) * (H * D) + i0;
#pragma unroll 1
      for (int h0 = 0; h0 < H; h0 += Y::kBatch) {
        issue();
        asm volatile("cp.async.wait_group %0;" ::"n"(kSt - 1) : "memory");
        const uint32_t src = mine + out * Y::kStage;
        if (++out == kSt) out = 0;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          Raw8<E> rlo, rhi;
#pragma unroll
          for (int j = 0; j < kVec; ++j) {
            rlo.w[j] = lds16(src + (u * 2 * kVec + j) * 512);
            rhi.w[j] = lds16(src + (u * 2 * kVec + kVec + j) * 512);
          }
          float lo[8], hi[8];
          rlo.get(lo);
          rhi.get(hi);
          norm_rotate<D>(lo, hi, wlo, whi, cs, p.eps);
          const int h = h0 + u * kRows + sub;
          if (h < H) {
            st8(y + h * D, lo);
            st8(y + h * D + D / 2, hi);
          }
        }
      }
    }
  }
}

struct NormAppendParams {
  nd_kv_cache c;
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements from one sequence to the next
  const float *wq, *wk;
  uint16_t *q_out;
  int Hq, to_sink;
  float eps;
  const int32_t *pos_base;
  int *err;
  Turns turns;
};

// The codec on the row (see nd_common.cuh): a 32-channel group is four
// neighbouring lanes' low or high eight channels; at D = 32 the whole row.
template <int D>
__device__ __forceinline__ void store_codes(const float *lo, const float *hi, int i0, bool live, int8_t *codes,
                                            float *scales) {
  float m[2] = {0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    m[0] = fmaxf(m[0], fabsf(lo[e]));
    m[1] = fmaxf(m[1], fabsf(hi[e]));
  }
  if constexpr (D == 32) m[0] = m[1] = fmaxf(m[0], m[1]);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
#pragma unroll
    for (int off = D == 32 ? 1 : 2; off >= 1; off >>= 1)
      m[half] = fmaxf(m[half], __shfl_xor_sync(0xffffffffu, m[half], off));
    const float *x = half ? hi : lo;
    const float scale = __fdiv_rn(m[half], 127.0f), inv = __frcp_rn(scale);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float r = 0.f;
      if (m[half] != 0.f) r = fminf(fmaxf(codec_rint(x[e], scale, inv), -127.f), 127.f);
      w[e / 4] |= uint32_t(int(r) & 0xff) << (8 * (e % 4));
    }
    const int ch = half * (D / 2) + i0;
    if (live) {
      *reinterpret_cast<uint2 *>(codes + ch) = make_uint2(w[0], w[1]);
      if (ch % 32 == 0) scales[ch / 32] = scale;
    }
  }
}

// One CTA per sequence, D/16 lanes per row: the query heads, then K's, then
// V's.  Every thread reads the sequence's four metadata words itself, beside
// its row; the last thing the CTA does is advance them.
template <int D>
__global__ void __launch_bounds__(512) qk_norm_append_kernel(const __grid_constant__ NormAppendParams p) {
  constexpr int kLanes = D / 16;
  const nd_kv_cache &c = p.c;
  const int b = blockIdx.x, i0 = 8 * (threadIdx.x % kLanes), per = blockDim.x / kLanes;
  const int Hkv = c.n_kv_heads, nslot = c.sink_cap + c.ring_cap, n_rows = p.Hq + 2 * Hkv, lane = threadIdx.x & 31;
  unsigned long long f[8];
  lane_freqs<D>(p.turns, lane, f);
  pdl_wait();
  const int sl = c.sink_len[b], rs = c.ring_start[b], rl = c.ring_len[b], sq = c.seq_len[b];
  const int pos = sq + (p.pos_base ? *p.pos_base : 0);
  const bool sane = sl >= 0 && sl <= c.sink_cap && rl >= 0 && rl <= c.ring_cap && rs >= 0 &&
                    rs < (c.ring_cap > 0 ? c.ring_cap : 1);
  int slot = -1;
  if (sane) {
    if (p.to_sink) slot = rl == 0 && sl < c.sink_cap ? sl : -1;
    else if (c.ring_cap > 0) slot = c.sink_cap + (rl < c.ring_cap ? (rs + rl) % c.ring_cap : rs);
  }
  if (slot < 0) {  // the same for the whole CTA
    if (threadIdx.x == 0) raise_device_error(p.err, ND_DEVERR_METADATA);
    return;
  }
  float2 cs[8];
  lane_angles<D>(pos, f, lane, cs);
  for (int r0 = 0; r0 < n_rows; r0 += per) {
    const int r = r0 + threadIdx.x / kLanes, rr = min(r, n_rows - 1);
    const bool live = r < n_rows;
    const int kind = rr < p.Hq ? 0 : (rr < p.Hq + Hkv ? 1 : 2);  // q, k, v
    const int h = rr - (kind == 0 ? 0 : (kind == 1 ? p.Hq : p.Hq + Hkv));
    const uint16_t *x = kind == 0 ? p.q + b * p.q_stride : (kind == 1 ? p.k + b * p.k_stride : p.v + b * p.v_stride);
    float lo[8], hi[8];
    ld8(x + size_t(h) * D + i0, lo);
    ld8(x + size_t(h) * D + D / 2 + i0, hi);
    const float *w = kind == 0 ? p.wq : p.wk;
    float wlo[8], whi[8];
    if (w && kind < 2) {
      ld8(w + i0, wlo);
      ld8(w + D / 2 + i0, whi);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) wlo[e] = whi[e] = 1.f;
    }
    float zlo[8], zhi[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) zlo[e] = lo[e], zhi[e] = hi[e];
    norm_rotate<D>(zlo, zhi, wlo, whi, cs, p.eps);
    if (kind < 2) {
      // the key is rounded to bf16 before it is quantised, so a token that a
      // step appends has the codes of one that a prefill (which writes bf16
      // keys) and the handoff put there
#pragma unroll
      for (int e = 0; e < 8; ++e) lo[e] = round_bf16(zlo[e]), hi[e] = round_bf16(zhi[e]);
    }
    const size_t row = (size_t(b) * Hkv + h) * nslot + slot;
    store_codes<D>(lo, hi, i0, live && kind > 0, (kind == 2 ? c.v_codes : c.k_codes) + row * D,
                   (kind == 2 ? c.v_scale : c.k_scale) + row * (D / 32));
    if (live && kind == 0) {
      uint16_t *y = p.q_out + (size_t(b) * p.Hq + h) * D + i0;
      st8(y, lo);
      st8(y + D / 2, hi);
    }
  }
  __syncthreads();  // every thread has read the metadata
  if (threadIdx.x == 0) {
    if (p.to_sink) c.sink_len[b] = sl + 1;
    else if (rl < c.ring_cap) c.ring_len[b] = rl + 1;
    else c.ring_start[b] = (rs + 1) % c.ring_cap;
    c.seq_len[b] = sq + 1;
  }
}

template <typename E, int D>
cudaError_t launch_norm_rope_d(const NormRopeParams<E> &p, cudaStream_t stream) {
  using Y = NormLay<E, D>;
  auto kern = qk_norm_rope_kernel<E, D>;
  static std::atomic<unsigned long long> smem_set{0};  // the opt-in, once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
  if (!bit || !(smem_set.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Y::kBytes);
    if (e != cudaSuccess) return e;
    smem_set.fetch_or(bit, std::memory_order_release);
  }
  const int blocks = (p.tokens + Y::kWarps - 1) / Y::kWarps, most = 152 * 4;
  return launch_pdl(kern, dim3(unsigned(blocks < most ? blocks : most)), dim3(32 * Y::kWarps), size_t(Y::kBytes), stream, p);
}

template <typename E>
cudaError_t launch_norm_rope_t(const QkNormRope &a, cudaStream_t stream) {
  NormRopeParams<E> p;
  p.x[0] = static_cast<const E *>(a.q);
  p.x[1] = static_cast<const E *>(a.k);
  p.y[0] = static_cast<E *>(a.q_out);
  p.y[1] = static_cast<E *>(a.k_out);
  p.w[0] = a.q_weight;
  p.w[1] = a.k_weight;
  p.H[0] = a.Hq;
  p.H[1] = a.Hk;
  p.stride[0] = a.q_stride;
  p.stride[1] = a.k_stride;
  p.T = a.T;
  p.tokens = a.batch * a.T;
  p.eps = a.eps;
  p.pos = a.positions;
  p.turns = make_turns(a.head_dim, a.theta);
  switch (a.head_dim) {
    case 32: return launch_norm_rope_d<E, 32>(p, stream);
    case 64: return launch_norm_rope_d<E, 64>(p, stream);
    case 128: return launch_norm_rope_d<E, 128>(p, stream);
    case 256: return launch_norm_rope_d<E, 256>(p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormRope &a, bool f32, cudaStream_t stream) {
  return f32 ? launch_norm_rope_t<float>(a, stream) : launch_norm_rope_t<uint16_t>(a, stream);
}

cudaError_t launch_qk_norm_append(const nd_kv_cache &c, const QkNormRope &a, const void *v, int64_t v_stride,
                                  const int32_t *pos_base, int to_sink, int *err, cudaStream_t stream) {
  NormAppendParams p;
  p.c = c;
  p.q = static_cast<const uint16_t *>(a.q);
  p.k = static_cast<const uint16_t *>(a.k);
  p.v = static_cast<const uint16_t *>(v);
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = v_stride;
  p.wq = a.q_weight;
  p.wk = a.k_weight;
  p.q_out = static_cast<uint16_t *>(a.q_out);
  p.Hq = a.Hq;
  p.to_sink = to_sink;
  p.eps = a.eps;
  p.pos_base = pos_base;
  p.err = err;
  p.turns = make_turns(c.head_dim, a.theta);
  const int lanes = (a.Hq + 2 * c.n_kv_heads) * (c.head_dim / 16);
  const int threads = lanes >= 512 ? 512 : (lanes + 31) / 32 * 32;
  const dim3 grid(c.batch), blk(threads);
  switch (c.head_dim) {
    case 32: return launch_pdl(qk_norm_append_kernel<32>, grid, blk, 0, stream, p);
    case 64: return launch_pdl(qk_norm_append_kernel<64>, grid, blk, 0, stream, p);
    case 128: return launch_pdl(qk_norm_append_kernel<128>, grid, blk, 0, stream, p);
    case 256: return launch_pdl(qk_norm_append_kernel<256>, grid, blk, 0, stream, p);
  }
  return cudaErrorInvalidValue;
}

}  // namespace nd
