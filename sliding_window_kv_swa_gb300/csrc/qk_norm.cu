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
// Angles: turns.cuh.
#include "nd_common.cuh"
#include "nd_internal.h"
#include "turns.cuh"

namespace nd {

namespace {

// The table of a model's head_dim and theta, kept per host thread: building it
// takes a pow per channel pair, about as long as a decode step's kernel.
const Turns &make_turns(int head_dim, float theta) {
  static thread_local Turns t;
  static thread_local int t_dim = 0;
  static thread_local float t_theta = 0.f;
  if (t_dim == head_dim && t_theta == theta) return t;
  const Freqs fr = make_freqs(head_dim, theta);
  for (int i = 0; i < kMaxHalf; ++i) t.f[i] = turn_of(theta != 0.f && i < head_dim / 2 ? fr.f[i] : 0.0);
  t_dim = head_dim;
  t_theta = theta;
  return t;
}

// Which channels lane j of a row's D / 16 lanes holds in each half: 16 bytes
// at a time, neighbouring lanes side by side.  bf16: 8j .. 8j + 7; fp32: 4j ..
// 4j + 3 and D/4 + 4j .. (eight in a row would leave every access half of its
// sectors).  Element e is channel base + (e % kPiece) + (e / kPiece) * kStep.
template <typename E, int D>
struct Chan {
  static constexpr int kPiece = 16 / sizeof(E), kStep = D / 16 * kPiece, kPieces = 8 / kPiece;
  __device__ __forceinline__ static int base(int j) { return kPiece * j; }
  __device__ __forceinline__ static int of(int j, int e) { return kPiece * j + e % kPiece + e / kPiece * kStep; }
};

// A lane's eight channels of one half as loaded, and as fp32.
template <typename E, int D>
struct Raw8 {
  uint4 w[sizeof(E) / 2];
  __device__ __forceinline__ void load(const E *p) {  // p: the half's channel Chan::base
#pragma unroll
    for (int i = 0; i < int(sizeof(E) / 2); ++i) w[i] = *reinterpret_cast<const uint4 *>(p + i * Chan<E, D>::kStep);
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
// the weights (fp32) of the lane's channels of one half
template <typename E, int D>
__device__ __forceinline__ void load_weights(const float *p, float *x) {
  constexpr int kStep = Chan<E, D>::kStep, kPiece = Chan<E, D>::kPiece;
#pragma unroll
  for (int e = 0; e < 8; e += 4) {
    const float4 v = *reinterpret_cast<const float4 *>(p + e % kPiece + e / kPiece * kStep);
    x[e] = v.x, x[e + 1] = v.y, x[e + 2] = v.z, x[e + 3] = v.w;
  }
}
template <int D>
__device__ __forceinline__ void store_half(uint16_t *p, const float *x) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                             pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
template <int D>
__device__ __forceinline__ void store_half(float *p, const float *x) {
  *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4 *>(p + Chan<float, D>::kStep) = make_float4(x[4], x[5], x[6], x[7]);
}

// The angles of a lane's eight channel pairs at the position that all rows of
// the warp have.  The lanes that hold the same pairs of other rows make an
// eighth to a half of them each.
template <typename E, int D>
__device__ __forceinline__ void shared_angles(int pos, const unsigned long long *s_f, int lane, float2 *cs) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes, kPer = kRows >= 8 ? 1 : 8 / kRows;
  const int j = lane % kLanes, e0 = (lane / kLanes) * kPer % 8;
  float2 mine[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) mine[i] = turn_cs(pos, s_f[Chan<E, D>::of(j, e0 + i)]);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int src = (e / kPer) * kLanes + j;
    cs[e].x = __shfl_sync(0xffffffffu, mine[e % kPer].x, src);
    cs[e].y = __shfl_sync(0xffffffffu, mine[e % kPer].y, src);
  }
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

// Many heads: a warp takes a token, as batches of rows (kU * 32 / (D / 16)
// heads of q, then of k).  HBM-bound: a row in and a row out; what it needs is
// loads in flight, so each lane copies its own channels kSt - 1 batches ahead
// into its own slots of shared memory (nothing to exchange, no barrier) while
// the angles, once per token for all its heads, and the batches before are
// computed.  One token to a warp: more, with the copies running on across
// them, spread the accesses of the moment over more of memory (117 us at 13
// tokens a warp).
// At 32768 tokens of 32 + 8 heads of 128 (671 MB): 99.8 us, 6.72 TB/s; 133 us
// with plain loads behind the angles, 120 with one batch ahead in registers.
template <typename E, int D>
struct NormLay {
  static constexpr int kLanes = D / 16, kRows = 32 / kLanes;
  static constexpr int kU = sizeof(E) == 2 ? 2 : 1, kBatch = kU * kRows;
  static constexpr int kSt = 4, kStage = kU * kRows * D * int(sizeof(E));  // 2 KB
  static constexpr int kWarps = 4, kBytes = kWarps * kSt * kStage;
};

template <typename E, int D>
__global__ void __launch_bounds__(128, 4) qk_norm_token_kernel(const __grid_constant__ NormRopeParams<E> p) {
  using Y = NormLay<E, D>;
  using Ch = Chan<E, D>;
  constexpr int kRows = Y::kRows, kU = Y::kU, kSt = Y::kSt, kVec = Ch::kPieces;
  __shared__ __align__(16) uint8_t s_ring[Y::kBytes];
  __shared__ unsigned long long s_f[D / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i0 = Ch::base(lane % Y::kLanes), sub = lane / Y::kLanes;
  // a lane's slots: 16 bytes each, 512 apart
  const uint32_t mine = smem_u32(s_ring) + warp * kSt * Y::kStage + lane * 16;
  const int tok = blockIdx.x * Y::kWarps + warp;
  stage_turns<D>(p.turns, s_f);
  pdl_wait();
  if (tok >= p.tokens) return;

  // the copies' cursor: q (0), k (1) or the end (2), and the batch's first head
  int c_which = p.H[0] > 0 ? 0 : 1, c_h = 0, in = 0, out = 0;
  auto issue = [&]() {
    if (c_which < 2) {
      const int H = c_which ? p.H[1] : p.H[0];
      const E *x = (c_which ? p.x[1] : p.x[0]) + tok * (c_which ? p.stride[1] : p.stride[0]) + i0;
      const uint32_t dst = mine + in * Y::kStage;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const E *row = x + min(c_h + u * kRows + sub, H - 1) * D;  // past the end: the last head, not stored
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          copy16(dst + (u * 2 * kVec + j) * 512, row + j * Ch::kStep);
          copy16(dst + (u * 2 * kVec + kVec + j) * 512, row + D / 2 + j * Ch::kStep);
        }
      }
      if (++in == kSt) in = 0;
      c_h += Y::kBatch;
      if (c_h >= H) c_h = 0, c_which += c_which == 0 && p.H[1] == 0 ? 2 : 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kSt - 1; ++i) issue();

  float2 cs[8];
  shared_angles<E, D>(p.pos ? p.pos[tok] : tok % p.T, s_f, lane, cs);
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int H = which ? p.H[1] : p.H[0];
    const float *w = which ? p.w[1] : p.w[0];
    float wlo[8], whi[8];
    if (w) {
      load_weights<E, D>(w + i0, wlo);
      load_weights<E, D>(w + D / 2 + i0, whi);
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
        Raw8<E, D> rlo, rhi;
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
          store_half<D>(y + h * D, lo);
          store_half<D>(y + h * D + D / 2, hi);
        }
      }
    }
  }
}

// Few heads: a token's rows would leave most of a warp's lanes idle and its
// angles serve hardly any row, so the rows of all tokens lie in one line (of a
// token q's heads, then k's) and every lane makes the angles of its own.
template <typename E, int D>
__global__ void __launch_bounds__(128) qk_norm_rows_kernel(const __grid_constant__ NormRopeParams<E> p) {
  using Ch = Chan<E, D>;
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;
  __shared__ unsigned long long s_f[D / 2];
  const int lane = threadIdx.x & 31, j = lane % kLanes, i0 = Ch::base(j), H = p.H[0] + p.H[1];
  stage_turns<D>(p.turns, s_f);
  pdl_wait();
  const unsigned n_rows = unsigned(p.tokens) * H;  // below 2^32: see the launch
  const unsigned row = (blockIdx.x * 4u + (threadIdx.x >> 5)) * kRows + lane / kLanes, rr = min(row, n_rows - 1);
  const int tok = int(rr / H), hh = int(rr % H);
  const int which = hh >= p.H[0], h = which ? hh - p.H[0] : hh;
  const E *x = (which ? p.x[1] : p.x[0]) + tok * (which ? p.stride[1] : p.stride[0]) + h * D + i0;
  Raw8<E, D> rlo, rhi;
  rlo.load(x);
  rhi.load(x + D / 2);
  const int pos = p.pos ? p.pos[tok] : tok % p.T;
  const float *w = which ? p.w[1] : p.w[0];
  float wlo[8], whi[8];
  if (w) {
    load_weights<E, D>(w + i0, wlo);
    load_weights<E, D>(w + D / 2 + i0, whi);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) wlo[e] = whi[e] = 1.f;
  }
  float2 cs[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) cs[e] = turn_cs(pos, s_f[Ch::of(j, e)]);
  float lo[8], hi[8];
  rlo.get(lo);
  rhi.get(hi);
  norm_rotate<D>(lo, hi, wlo, whi, cs, p.eps);
  if (row < n_rows) {
    E *y = (which ? p.y[1] : p.y[0]) + (int64_t(tok) * (which ? p.H[1] : p.H[0]) + h) * D + i0;
    store_half<D>(y, lo);
    store_half<D>(y + D / 2, hi);
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
// V's.  A step is a chain of latencies, so the loads of the first pass go out
// at once: every thread reads the sequence's four metadata words itself, beside
// its row and weights; the last thing the CTA does is advance them.  Above 192
// lanes the rows take further passes (32 + 8 + 8 heads of 128: two), whose
// loads follow the pass before: 6.5 us for 512 sequences, the bytes 1.9.
template <int D>
__global__ void __launch_bounds__(192, 4) qk_norm_append_kernel(const __grid_constant__ NormAppendParams p) {
  constexpr int kLanes = D / 16;
  using Ch = Chan<uint16_t, D>;
  const nd_kv_cache &c = p.c;
  const int b = blockIdx.x, j = threadIdx.x % kLanes, i0 = Ch::base(j), per = blockDim.x / kLanes;
  const int Hkv = c.n_kv_heads, n_rows = p.Hq + 2 * Hkv, lane = threadIdx.x & 31;
  __shared__ unsigned long long s_f[D / 2];
  stage_turns<D>(p.turns, s_f);
  pdl_wait();
  Raw8<uint16_t, D> rlo, rhi;
  auto load = [&](int r) {
    const uint16_t *x = r < p.Hq         ? p.q + b * p.q_stride + r * D
                        : r < p.Hq + Hkv ? p.k + b * p.k_stride + (r - p.Hq) * D
                                         : p.v + b * p.v_stride + (r - p.Hq - Hkv) * D;
    rlo.load(x + i0);
    rhi.load(x + D / 2 + i0);
  };
  load(min(int(threadIdx.x) / kLanes, n_rows - 1));
  const int sl = c.sink_len[b], rs = c.ring_start[b], rl = c.ring_len[b], sq = c.seq_len[b];
  const int pos = sq + (p.pos_base ? *p.pos_base : 0);
  const bool sane = sl >= 0 && sl <= c.sink_cap && rl >= 0 && rl <= c.ring_cap && rs >= 0 &&
                    rs < (c.ring_cap > 0 ? c.ring_cap : 1);
  int slot = -1;
  if (sane) {
    if (p.to_sink) {
      slot = rl == 0 && sl < c.sink_cap ? sl : -1;
    } else if (c.ring_cap > 0) {
      int r = rl < c.ring_cap ? rs + rl : rs;
      if (r >= c.ring_cap) r -= c.ring_cap;
      slot = c.sink_cap + r;
    }
  }
  if (slot < 0) {  // the same for the whole CTA
    if (threadIdx.x == 0) raise_device_error(p.err, ND_DEVERR_METADATA);
    return;
  }
  float2 cs[8];
  shared_angles<uint16_t, D>(pos, s_f, lane, cs);
  for (int r0 = 0; r0 < n_rows; r0 += per) {
    const int r = r0 + threadIdx.x / kLanes;
    const bool live = r < n_rows, is_v = r >= p.Hq + Hkv;
    if (r0 > 0) load(min(r, n_rows - 1));
    float lo[8], hi[8];
    rlo.get(lo);
    rhi.get(hi);
    if (__any_sync(0xffffffffu, !is_v)) {  // (a warp may hold rows of K and of V)
      const float *w = r < p.Hq ? p.wq : p.wk;
      float wlo[8], whi[8];
      if (w) {
        load_weights<uint16_t, D>(w + i0, wlo);
        load_weights<uint16_t, D>(w + D / 2 + i0, whi);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) wlo[e] = whi[e] = 1.f;
      }
      float zlo[8], zhi[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) zlo[e] = lo[e], zhi[e] = hi[e];
      norm_rotate<D>(zlo, zhi, wlo, whi, cs, p.eps);
      // the key is rounded to bf16 before it is quantised, so a token that a
      // step appends has the codes of one that a prefill (which writes bf16
      // keys) and the handoff put there
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (!is_v) lo[e] = round_bf16(zlo[e]), hi[e] = round_bf16(zhi[e]);
    }
    if (__any_sync(0xffffffffu, live && r >= p.Hq)) {
      const int h = is_v ? r - p.Hq - Hkv : r - p.Hq;
      const size_t row = (size_t(b) * Hkv + h) * (c.sink_cap + c.ring_cap) + slot;
      store_codes<D>(lo, hi, i0, live && r >= p.Hq, (is_v ? c.v_codes : c.k_codes) + row * D,
                     (is_v ? c.v_scale : c.k_scale) + row * (D / 32));
    }
    if (r < p.Hq) {
      uint16_t *y = p.q_out + (size_t(b) * p.Hq + r) * D + i0;
      store_half<D>(y, lo);
      store_half<D>(y + D / 2, hi);
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

// A warp to a token where its heads fill two row sets (8 + 2 heads of 64, just
// more than one: 33 us as rows, 34 as a token; 16 + 2: 56 against 37) and the
// rows are many (40 heads of 128: 250 tokens 4.0 us as rows, 4.5 as tokens;
// 400: 5.3 against 4.5).
constexpr int kMinSets = 2, kFewSets = 2600;
template <typename E, int D>
cudaError_t launch_norm_rope_d(const NormRopeParams<E> &p, cudaStream_t stream) {
  using Y = NormLay<E, D>;
  const int64_t H = p.H[0] + p.H[1], rows = H * p.tokens;
  if ((H >= kMinSets * Y::kRows && rows > kFewSets * Y::kRows) || rows >= (int64_t(1) << 32) - 4 * Y::kRows)
    return launch_pdl(qk_norm_token_kernel<E, D>, dim3(unsigned((p.tokens + Y::kWarps - 1) / Y::kWarps)),
                      dim3(32 * Y::kWarps), 0, stream, p);
  return launch_pdl(qk_norm_rows_kernel<E, D>, dim3(unsigned((rows + 4 * Y::kRows - 1) / (4 * Y::kRows))), dim3(128), 0,
                    stream, p);
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
  // (192 threads at most, four CTAs to an SM and the rows in passes: 512 tokens
  // of 48 rows 6.5 us, against 9 with a thread group per row)
  const int threads = lanes >= 192 ? 192 : (lanes + 31) / 32 * 32;
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
