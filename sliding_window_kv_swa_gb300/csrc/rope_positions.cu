// rope_positions.cu -- rotary embedding of query and key heads at given
// positions: channels paired across halves or as neighbours, the whole head or
// its first channels, frequencies scaled for long contexts, or the gradient.
//
// For pair (a, b) of the first r channels of a head at position p,
//   a' = m (a cos t - b sin t),  b' = m (b cos t + a sin t),  t = +-p f_i,
// the channels behind r copied as they are.  The gradient of a rotation is the
// rotation by the opposite angle, so it is the same kernel with -t.
//
// Work split: a lane holds two 16-byte pieces of a row (P = 8 bf16 or 4 fp32
// channels each), D / 2P lanes a row, neighbouring lanes side by side.  Halves:
// the two pieces are each other's partners, P pairs.  Neighbours: every piece
// holds P/2 pairs of its own, so the same two pieces serve (taking the pieces
// 2j and 2j+1 instead would leave every access half of its sectors).  Lanes
// whose pieces lie behind r move them unchanged.
//
// HBM-bound: a row in and a row out.  32768 bf16 tokens of 40 heads of 128, half of
// each turned (671 MB): 98 us, 6.85 TB/s.  Angles: turns.cuh.
#include <string.h>

#include "nd_common.cuh"
#include "nd_internal.h"
#include "turns.cuh"

namespace nd {

namespace {

// What a lane of a row's D / 2P lanes holds.
template <typename E, int D, bool kNeighbours>
struct Pieces {
  static constexpr int P = 16 / sizeof(E), kLanes = D / (2 * P);
  int a, b;     // first channels of its pieces
  bool ta, tb;  // whether they are turned
  __device__ __forceinline__ Pieces(int j, int r) {
    if constexpr (kNeighbours) {
      a = j * P;
      b = D / 2 + j * P;
      ta = a < r;
      tb = b < r;
    } else {
      const int half = r / (2 * P);  // lanes with pairs
      ta = tb = j < half;
      a = ta ? j * P : r + (j - half) * P;
      b = ta ? r / 2 + j * P : r + (D - r) / 2 + (j - half) * P;
    }
  }
  // the pair of angle e, e < P
  __device__ __forceinline__ int pair(int e) const {
    if constexpr (kNeighbours) return e < P / 2 ? a / 2 + e : b / 2 + e - P / 2;
    else return a + e;
  }
};

template <typename E>
struct RopeParams {
  const E *x[2];  // q, k
  E *y[2];
  int H[2];
  int64_t stride[2];  // elements from one token to the next in x
  int T, tokens, r;
  float cos_by, sin_by;  // the magnitude, and with the direction's sign
  const int32_t *pos;
  Turns turns;
};

// (cos, sin) of pair i; pairs of pieces behind r turn by nothing that is used
template <typename E, int D>
__device__ __forceinline__ float2 angle(const RopeParams<E> &p, int pos, const unsigned long long *s_f, int i) {
  const float2 cs = turn_cs(pos, s_f[min(i, D / 2 - 1)]);
  return make_float2(cs.x * p.cos_by, cs.y * p.sin_by);
}

template <bool kNeighbours, typename E, int D>
__device__ __forceinline__ void turn_pieces(uint4 &wa, uint4 &wb, const Pieces<E, D, kNeighbours> &pc, const float2 *cs) {
  constexpr int P = 16 / sizeof(E);
  float x[2][P], y[2][P];
  const uint4 w[2] = {wa, wb};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t u[4] = {w[h].x, w[h].y, w[h].z, w[h].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(E) == 2) x[h][2 * i] = bf16_lo(u[i]), x[h][2 * i + 1] = bf16_hi(u[i]);
      else x[h][i] = __uint_as_float(u[i]);
    }
  }
  if constexpr (kNeighbours) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < P / 2; ++e) {
        const float2 c = cs[h * (P / 2) + e];
        rope_pair(x[h][2 * e], x[h][2 * e + 1], c.x, c.y, y[h][2 * e], y[h][2 * e + 1]);
      }
  } else {
#pragma unroll
    for (int e = 0; e < P; ++e) rope_pair(x[0][e], x[1][e], cs[e].x, cs[e].y, y[0][e], y[1][e]);
  }
  uint4 o[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (sizeof(E) == 2)
      o[h] = make_uint4(pack_bf16x2(y[h][0], y[h][1]), pack_bf16x2(y[h][2], y[h][3]), pack_bf16x2(y[h][4], y[h][5]),
                        pack_bf16x2(y[h][6], y[h][7]));
    else
      o[h] = make_uint4(__float_as_uint(y[h][0]), __float_as_uint(y[h][1]), __float_as_uint(y[h][2]), __float_as_uint(y[h][3]));
  }
  if (pc.ta) wa = o[0];
  if (pc.tb) wb = o[1];
}

// Many heads: a warp takes a token, as batches of rows of q, then of k.  Each
// lane copies its own pieces kSt - 1 batches ahead into its own slots of shared
// memory; the angles, once per token, are made meanwhile, every lane a part of
// those that the lanes of its column need.
template <typename E, int D>
struct RopeLay {
  static constexpr int kLanes = D / (2 * (16 / int(sizeof(E)))), kRows = 32 / kLanes, kU = 2, kBatch = kU * kRows;
  static constexpr int kSt = 4, kStage = kU * 2 * 32 * 16;  // 2 KB
  static constexpr int kWarps = 4, kBytes = kWarps * kSt * kStage;
};

template <typename E, int D, bool kNeighbours>
__global__ void __launch_bounds__(128, 4) rope_token_kernel(const __grid_constant__ RopeParams<E> p) {
  using Y = RopeLay<E, D>;
  constexpr int kRows = Y::kRows, kU = Y::kU, kSt = Y::kSt, P = 16 / sizeof(E);
  __shared__ __align__(16) uint8_t s_ring[Y::kBytes];
  __shared__ unsigned long long s_f[D / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / Y::kLanes;
  const Pieces<E, D, kNeighbours> pc(lane % Y::kLanes, p.r);
  const uint32_t mine = smem_u32(s_ring) + warp * kSt * Y::kStage + lane * 16;  // 16 bytes each, 512 apart
  const int tok = blockIdx.x * Y::kWarps + warp;
  stage_turns<D>(p.turns, s_f);
  pdl_wait();
  if (tok >= p.tokens) return;

  // the copies' cursor: q (0), k (1) or the end (2), and the batch's first head
  int c_which = p.H[0] > 0 ? 0 : 1, c_h = 0, in = 0, out = 0;
  auto issue = [&]() {
    if (c_which < 2) {
      const int H = c_which ? p.H[1] : p.H[0];
      const E *x = (c_which ? p.x[1] : p.x[0]) + tok * (c_which ? p.stride[1] : p.stride[0]);
      const uint32_t dst = mine + in * Y::kStage;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const E *row = x + min(c_h + u * kRows + sub, H - 1) * D;  // past the end: the last head, not stored
        copy16(dst + u * 1024, row + pc.a);
        copy16(dst + u * 1024 + 512, row + pc.b);
      }
      if (++in == kSt) in = 0;
      c_h += Y::kBatch;
      if (c_h >= H) c_h = 0, c_which += c_which == 0 && p.H[1] == 0 ? 2 : 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kSt - 1; ++i) issue();

  float2 cs[P];
  {
    const int pos = p.pos ? p.pos[tok] : tok % p.T;
    constexpr int kPer = kRows >= P ? 1 : P / kRows;
    const int e0 = sub * kPer % P;
    float2 part[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) part[i] = angle<E, D>(p, pos, s_f, pc.pair(e0 + i));
#pragma unroll
    for (int e = 0; e < P; ++e) {
      const int src = (e / kPer) * Y::kLanes + lane % Y::kLanes;
      cs[e].x = __shfl_sync(0xffffffffu, part[e % kPer].x, src);
      cs[e].y = __shfl_sync(0xffffffffu, part[e % kPer].y, src);
    }
  }
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int H = which ? p.H[1] : p.H[0];
    E *y = (which ? p.y[1] : p.y[0]) + int64_t(tok) * (H * D);
#pragma unroll 1
    for (int h0 = 0; h0 < H; h0 += Y::kBatch) {
      issue();
      asm volatile("cp.async.wait_group %0;" ::"n"(kSt - 1) : "memory");
      const uint32_t src = mine + out * Y::kStage;
      if (++out == kSt) out = 0;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        uint4 wa = lds16(src + u * 1024), wb = lds16(src + u * 1024 + 512);
        turn_pieces<kNeighbours, E, D>(wa, wb, pc, cs);
        const int h = h0 + u * kRows + sub;
        if (h < H) {
          *reinterpret_cast<uint4 *>(y + h * D + pc.a) = wa;
          *reinterpret_cast<uint4 *>(y + h * D + pc.b) = wb;
        }
      }
    }
  }
}

// Few heads or few tokens: the rows of all tokens lie in one line (of a token
// q's heads, then k's) and every lane makes the angles of its own.
template <typename E, int D, bool kNeighbours>
__global__ void __launch_bounds__(128) rope_rows_kernel(const __grid_constant__ RopeParams<E> p) {
  using Y = RopeLay<E, D>;
  constexpr int kRows = Y::kRows, P = 16 / sizeof(E);
  __shared__ unsigned long long s_f[D / 2];
  const int lane = threadIdx.x & 31, H = p.H[0] + p.H[1];
  const Pieces<E, D, kNeighbours> pc(lane % Y::kLanes, p.r);
  stage_turns<D>(p.turns, s_f);
  pdl_wait();
  const unsigned n_rows = unsigned(p.tokens) * H;  // below 2^32: see the launch
  const unsigned row = (blockIdx.x * 4u + (threadIdx.x >> 5)) * kRows + lane / Y::kLanes;
  if (row >= n_rows) return;
  const int tok = int(row / H), hh = int(row % H);
  const int which = hh >= p.H[0], h = which ? hh - p.H[0] : hh;
  const E *x = (which ? p.x[1] : p.x[0]) + tok * (which ? p.stride[1] : p.stride[0]) + h * D;
  uint4 wa = *reinterpret_cast<const uint4 *>(x + pc.a), wb = *reinterpret_cast<const uint4 *>(x + pc.b);
  const int pos = p.pos ? p.pos[tok] : tok % p.T;
  float2 cs[P];
  if (pc.ta || pc.tb) {
#pragma unroll
    for (int e = 0; e < P; ++e) cs[e] = angle<E, D>(p, pos, s_f, pc.pair(e));
    turn_pieces<kNeighbours, E, D>(wa, wb, pc, cs);
  }
  E *y = (which ? p.y[1] : p.y[0]) + (int64_t(tok) * (which ? p.H[1] : p.H[0]) + h) * D;
  *reinterpret_cast<uint4 *>(y + pc.a) = wa;
  *reinterpret_cast<uint4 *>(y + pc.b) = wb;
}

// The table of a configuration, kept per host thread: building it takes a pow
// per pair, about as long as a small call's kernel.
const Turns &rope_turns(const nd_rope_cfg &c) {
  static thread_local Turns t;
  static thread_local nd_rope_cfg kept;
  static thread_local bool made = false;
  const auto same = [](const nd_rope_cfg &a, const nd_rope_cfg &b) {
    return a.rotary_dim == b.rotary_dim && a.scaling == b.scaling && a.theta == b.theta && a.factor == b.factor &&
           a.low == b.low && a.high == b.high && a.orig_len == b.orig_len;
  };
  if (made && same(kept, c)) return t;
  const Freqs fr = make_freqs(c.rotary_dim, c.theta);
  for (int i = 0; i < kMaxHalf; ++i) {
    double f = i < c.rotary_dim / 2 ? fr.f[i] : 0.0;
    if (c.scaling == ND_ROPE_LINEAR) {
      f /= double(c.factor);
    } else if (c.scaling == ND_ROPE_BY_PARTS) {
      const double turns = double(c.orig_len) * f * 0.15915494309189533576888376337251;
      const double g = fmin(fmax((turns - c.low) / (double(c.high) - c.low), 0.0), 1.0);
      f = (1.0 - g) * f / double(c.factor) + g * f;
    }
    t.f[i] = turn_of(f);
  }
  kept = c;
  made = true;
  return t;
}

// A warp to a token where its heads fill two row sets (a warp's rows: 4 of bf16 at
// D = 128) and the rows are many.  By token against by row, us: bf16, 40 heads of
// 128, 1280 sets 3.2 and 2.7, 2560 3.4 and 3.4, 5120 3.3 and 4.5, 40960 15.3 and 24.3
// (neighbours and a quarter of each head turned alike); 72 heads of 32 cross there
// too, 20 heads of 256 at 1900.  fp32 crosses later: 40 heads of 128, 2560 sets 4.2
// and 2.7, 5120 4.2 and 3.6, 10240 4.2 and 5.3.  5 heads of 64, less than a set, by
// token lose at every length: 2560 sets 5.2 and 3.2.
constexpr int kMinSets = 2, kFewSets = 2600;

template <typename E, int D, bool kNeighbours>
cudaError_t launch_rope_n(const RopeParams<E> &p, cudaStream_t stream) {
  using Y = RopeLay<E, D>;
  const int64_t H = p.H[0] + p.H[1], rows = H * p.tokens;
  if ((H >= kMinSets * Y::kRows && rows > kFewSets * Y::kRows) || rows >= (int64_t(1) << 32) - 4 * Y::kRows)
    return launch_pdl(rope_token_kernel<E, D, kNeighbours>, dim3(unsigned((p.tokens + Y::kWarps - 1) / Y::kWarps)),
                      dim3(32 * Y::kWarps), 0, stream, p);
  return launch_pdl(rope_rows_kernel<E, D, kNeighbours>, dim3(unsigned((rows + 4 * Y::kRows - 1) / (4 * Y::kRows))),
                    dim3(128), 0, stream, p);
}

template <typename E, int D>
cudaError_t launch_rope_d(const RopeParams<E> &p, bool neighbours, cudaStream_t stream) {
  return neighbours ? launch_rope_n<E, D, true>(p, stream) : launch_rope_n<E, D, false>(p, stream);
}

template <typename E>
cudaError_t launch_rope_t(const QkNormRope &a, const nd_rope_cfg &c, cudaStream_t stream) {
  RopeParams<E> p;
  p.x[0] = static_cast<const E *>(a.q);
  p.x[1] = static_cast<const E *>(a.k);
  p.y[0] = static_cast<E *>(a.q_out);
  p.y[1] = static_cast<E *>(a.k_out);
  p.H[0] = a.Hq;
  p.H[1] = a.Hk;
  p.stride[0] = a.q_stride;
  p.stride[1] = a.k_stride;
  p.T = a.T;
  p.tokens = a.batch * a.T;
  p.r = c.rotary_dim;
  p.cos_by = c.magnitude;
  p.sin_by = c.inverse ? -c.magnitude : c.magnitude;
  p.pos = a.positions;
  p.turns = rope_turns(c);
  switch (a.head_dim) {
    case 32: return launch_rope_d<E, 32>(p, c.interleaved, stream);
    case 64: return launch_rope_d<E, 64>(p, c.interleaved, stream);
    case 128: return launch_rope_d<E, 128>(p, c.interleaved, stream);
    case 256: return launch_rope_d<E, 256>(p, c.interleaved, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rope_positions(const QkNormRope &a, const nd_rope_cfg &c, bool f32, cudaStream_t stream) {
  return f32 ? launch_rope_t<float>(a, c, stream) : launch_rope_t<uint16_t>(a, c, stream);
}

}  // namespace nd
