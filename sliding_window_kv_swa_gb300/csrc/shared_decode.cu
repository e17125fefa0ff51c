// shared_decode.cu -- the sequences' own part of a decode step over a shared
// prefix, and the merge with the prefix's partials (shared_prefix.cu).
//
// Each (sequence, KV head) attends to its own sink and ring slots as the
// decode kernel does (decode_step.cuh; the mask is "recent | sink"), and the
// triples (m, l, O) of the shared prefix join that softmax exactly:
//   m = max(m_a, m_b),  l = sum l_i 2^(m_i - m),  O = sum O_i 2^(m_i - m).
//
// HBM-bound: 2 (D + D/8) bytes per own slot and KV head.  A session's ring is
// short (256 slots are 73 KB), so a CTA per pair would spend as long starting
// and ending as reading.  Here a warp walks several units one after the other,
// and its copies run on across the boundary: while a unit is merged and
// written, the next one's steps are in flight.  As many units as make whole
// rounds of all warps are each one warp's own (sixteen steps per start and end
// where the four warps of a CTA together would take four); the rest are
// walked by a CTA's warps together, so the last round is as long as its share.
// The merge needs no memory of its own: of a warp's ST stages ST - 1 are being
// filled, and the one just read holds its state.
// 512 sequences of 256 slots, 8 heads of 128 (302 MB): 66 us (4.6 TB/s), of
// which the bytes take 44; the decode kernel, on walks of 1280 slots, moves the
// same format at 5.5 TB/s.  While a warp walks, a step takes 2000 cycles, three
// warps to a scheduler whose issue slots they fill to 70 % (400 instructions of
// the products, their operands and the softmax, 100 of the copies); a walk is
// 16 steps, and about a quarter of a warp's time goes between walks (metadata,
// query, the merge, and the loads of the prefix's partials, which are asked for
// only there), so over the whole kernel the slots are 41 % used and loads are
// the longest stall.  Copies by one lane and a tensor map, two steps to a
// softmax update, and four CTAs to an SM were no faster.  At 168 registers the
// kernel spills 66 bytes a thread (82 at D = 64, at 96 registers), at the 128
// of four CTAs more.
//
// A unit is a (sequence, KV head) pair, or a part of one where the pairs are
// too few for the SMs; the parts' triples then go to the workspace and a merge
// kernel joins them with the prefix's.  A short prefix that few sequences
// share is cheaper read again by each of them than multiplied apart (kInline):
// its slots then are the first steps of every unit.
#include <atomic>

#include "decode_step.cuh"
#include "nd_common.cuh"
#include "nd_internal.h"
#include "shared_prefix.cuh"

namespace nd {

namespace {

struct OwnParams {
  const uint16_t *q;
  nd_kv_cache c;       // the sequences
  nd_kv_cache pre;     // the shared prefix (one row)
  int Hq, G, window;
  int n_split, slots_per_unit, n_units;  // units = pairs * n_split
  int solo;            // units that every warp takes alone, before those of the whole CTA
  int inline_slots;    // prefix slots walked by every unit (a multiple of kStep), or 0
  uint16_t *out;
  float *lse;
  float *ws_ml, *ws_o; // n_split > 1: [pair][n_split][G][2], [..][G][D]
  PrefixParts parts;   // the prefix's partials, when prefix_grid > 0
  int streams;         // prefix_streams
  int prefix_grid;
  bool early;          // the kernel before this one is the call's own prefix kernel: see shared_own_kernel
  int *err;
};

// ------------------------------------------------------------------ a warp's step
// Thread (g, t) = (lane / 4, lane % 4).  QK: D[head][slot] = q (fp16, rows =
// heads) x codes^T per 32-channel group, so that a group's fp32 scale
// multiplies its own sum; PV: D[channel][head] = codes^T x P'^T with P' = p *
// v_scale * 2^e; the scores' registers are the weights' (decode.cu has the
// layout).  What this step does to need about half the instructions of a
// straightforward one, which bound it (a step of the first form was 750
// instructions a warp, twice its share of the bytes' time):
//   - addresses of the swizzled chunks are one XOR from a per-step base;
//   - the code's bias stays in K's operands (1024 + 128 + code is exact in
//     fp16) and comes off the group's sum at once, as 1152 * sum q.  (fp32 holds 1152 * 32 |q| to 2^-8 |q| against sums
//     of about 240 |q|.  V's sums run over all slots, where the same would
//     cancel away bits, so V's bias comes off each pair of codes.)
//   - the running maximum and V's exponent are compared without exchange
//     between lanes; only a step that moves one (rare) reduces and rescales;
//   - a step whose slots are all visible, the common one, masks nothing.
template <int D>
struct HeadQ {
  uint32_t qa[D / 32][2][2];
  float bias[D / 32];  // -1152 * the group's sum of q, for head g
  float coef;          // 2^-Eq * log2(e) / sqrt(D), for head g
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
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hq.qa[grp][i >> 1][i & 1] = pack_half2(bf16_lo(ws[i]) * up, bf16_hi(ws[i]) * up);
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hq.qa[grp][i >> 1][i & 1]));
      sum += f.x + f.y;  // of the rounded values: what the products see
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    hq.bias[grp] = -1152.f * sum;
  }
}

template <int D>
struct RunState {
  float o[D / 32][2][4];  // heads 2t, 2t+1; channels 32*grp + 4g + 2*tile (+1)
  float m, l;             // head g: the max p is taken against (log2 units); this thread's share of the sum
  int e;                  // power-of-two pre-scale of P' (never increases; 127 = unset)
  float u, lim;           // 2^e (1 while unset); the v_scale from which e has to shrink
  __device__ __forceinline__ RunState() {
#pragma unroll
    for (int grp = 0; grp < D / 32; ++grp)
#pragma unroll
      for (int i = 0; i < 8; ++i) o[grp][i >> 2][i & 3] = 0.f;
    m = -INFINITY, l = 0.f, e = 127, u = 1.f, lim = exp2i(-120);
  }
};

// fp16 pairs 1152 + code of bytes (0, 1) and (2, 3) of a word of codes
__device__ __forceinline__ uint32_t biased_half2(uint32_t w_biased, uint32_t sel) {
  return prmt(w_biased, 0x64646464u, sel);
}

// The group scales of two neighbouring slots.
template <int NG>
__device__ __forceinline__ void lds_scales2(uint32_t a, float (&s0)[NG], float (&s1)[NG]) {
  const float4 x = lds128f(a);
  if constexpr (NG == 4) {
    const float4 y = lds128f(a + 16);
    s0[0] = x.x, s0[1] = x.y, s0[2] = x.z, s0[3] = x.w;
    s1[0] = y.x, s1[1] = y.y, s1[2] = y.z, s1[3] = y.w;
  } else {
    s0[0] = x.x, s0[1] = x.y, s1[0] = x.z, s1[1] = x.w;
  }
}

// One step staged at st (a multiple of 128).  vis_bits: bit i = slot col[i] of
// this thread counts, col = {2t, 2t+1, 8+2t, 9+2t}; all_vis (the same in the
// whole warp): every slot does.
template <int D>
__device__ __forceinline__ void attend_step(uint32_t st, const HeadQ<D> &hq, bool all_vis, uint32_t vis_bits, int lane,
                                            RunState<D> &r) {
  constexpr int NG = D / 32;
  using S = Stage<D>;
  const int g = lane >> 2, t = lane & 3;
  // row 8 lies 8 rows on; at D = 64 (two rows a line) its line's swizzle also
  // differs in bit 6
  constexpr uint32_t kRow8 = 8 * D, kFlip8 = D == 64 ? 64u : 0u;
  const uint32_t kb = st + swz(uint32_t(g * D + 8 * t));
  const uint32_t vb0 = st + S::kCodes + swz(uint32_t(2 * t * D + 4 * g)),
                 vb1 = st + S::kCodes + swz(uint32_t((2 * t + 1) * D + 4 * g));
  const uint32_t sb = st + 2 * S::kCodes + 2 * t * NG * 4;
  // ---- QK: scores of head g at slots col[0..3]
  float sc[4];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float ks0[NG], ks1[NG];
    lds_scales2<NG>(sb + j * 8 * NG * 4, ks0, ks1);
#pragma unroll
    for (int grp = 0; grp < NG; ++grp) {
      const uint2 kw = lds64((kb ^ (grp * 32 + j * kFlip8)) + j * kRow8);
      float d0 = 0.f, d1 = 0.f, d2 = 0.f, d3 = 0.f;
      const uint32_t w0 = kw.x ^ 0x80808080u, w1 = kw.y ^ 0x80808080u;
      mma_f16_16816(d0, d1, d2, d3, hq.qa[grp][0][0], 0u, hq.qa[grp][0][1], 0u, biased_half2(w0, kSelBytes01),
                    biased_half2(w0, kSelBytes23));
      mma_f16_16816(d0, d1, d2, d3, hq.qa[grp][1][0], 0u, hq.qa[grp][1][1], 0u, biased_half2(w1, kSelBytes01),
                    biased_half2(w1, kSelBytes23));
      d0 += hq.bias[grp];
      d1 += hq.bias[grp];
      sc[2 * j] = grp ? fmaf(ks0[grp], d0, sc[2 * j]) : ks0[grp] * d0;
      sc[2 * j + 1] = grp ? fmaf(ks1[grp], d1, sc[2 * j + 1]) : ks1[grp] * d1;
    }
  }
  float vs[4][NG];
  lds_scales2<NG>(sb + S::kScales, vs[0], vs[1]);
  lds_scales2<NG>(sb + S::kScales + 8 * NG * 4, vs[2], vs[3]);
  // ---- online softmax for head g (log2 domain)
#pragma unroll
  for (int i = 0; i < 4; ++i) sc[i] *= hq.coef;
  if (!all_vis) {  // masked slots count 0, whatever their scales are
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!((vis_bits >> i) & 1u)) {
        sc[i] = -INFINITY;
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) vs[i][grp] = 0.f;
      }
  }
  float mx = fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3])), vm = 0.f;
#pragma unroll
  for (int grp = 0; grp < NG; ++grp) vm = fmaxf(vm, fmaxf(fmaxf(vs[0][grp], vs[1][grp]), fmaxf(vs[2][grp], vs[3][grp])));
  if (__any_sync(0xffffffffu, mx > r.m + kLazyLog2 || vm >= r.lim)) {
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, 1));
    vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, 2));
    const bool need = mx > r.m + kLazyLog2;
    const float alpha = need ? ex2(r.m - mx) : 1.f;  // 0 from the empty state
    r.l *= alpha;
    r.m = need ? mx : r.m;
    // p * v_scale * 2^e stays below 2^15 (p <= 2^8)
    float shrink = 1.f;
    if (vm >= r.lim) {
      const int e = 14 - int(kLazyLog2) - ilog2_floor(vm);
      shrink = r.e == 127 ? 0.f : exp2i(e - r.e);
      r.e = e;
      r.u = exp2i(e);
      r.lim = exp2i(7 - e);
    }
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
  }
  const float m_ref = r.m == -INFINITY ? 0.f : r.m;
  float pu[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) pu[i] = ex2(sc[i] - m_ref);
  r.l += (pu[0] + pu[1]) + (pu[2] + pu[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) pu[i] *= r.u;
  // ---- PV per group: B = P'^T (slot x head), A = V^T (channel x slot)
#pragma unroll
  for (int grp = 0; grp < NG; ++grp) {
    const uint32_t b0 = pack_half2(pu[0] * vs[0][grp], pu[1] * vs[1][grp]);
    const uint32_t b1 = pack_half2(pu[2] * vs[2][grp], pu[3] * vs[3][grp]);
    uint32_t vw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      vw[i] = lds32((((i & 1) ? vb1 : vb0) ^ (grp * 32 + (i >> 1) * kFlip8)) + (i >> 1) * kRow8);
    const uint32_t x01 = prmt(vw[0], vw[1], 0x5140u) ^ 0x80808080u, x23 = prmt(vw[0], vw[1], 0x7362u) ^ 0x80808080u;
    const uint32_t y01 = prmt(vw[2], vw[3], 0x5140u) ^ 0x80808080u, y23 = prmt(vw[2], vw[3], 0x7362u) ^ 0x80808080u;
    // tile 0: rows g <-> channel 4g, rows g+8 <-> channel 4g+1; tile 1: 4g+2, 4g+3
    mma_f16_16816(r.o[grp][0][0], r.o[grp][0][1], r.o[grp][0][2], r.o[grp][0][3], codes_to_half2(x01, kSelBytes01),
                  codes_to_half2(x01, kSelBytes23), codes_to_half2(y01, kSelBytes01),
                  codes_to_half2(y01, kSelBytes23), b0, b1);
    mma_f16_16816(r.o[grp][1][0], r.o[grp][1][1], r.o[grp][1][2], r.o[grp][1][3], codes_to_half2(x23, kSelBytes01),
                  codes_to_half2(x23, kSelBytes23), codes_to_half2(y23, kSelBytes01),
                  codes_to_half2(y23, kSelBytes23), b0, b1);
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
  float *w0 = o + (2 * t) * D + 4 * g, *w1 = w0 + D;
#pragma unroll
  for (int grp = 0; grp < D / 32; ++grp) {
    const auto &a = r.o[grp];  // channels 4g .. 4g+3: tile 0 rows g, g+8, tile 1 rows g, g+8
    *reinterpret_cast<float4 *>(w0 + 32 * grp) = make_float4(a[0][0] * down, a[0][2] * down, a[1][0] * down, a[1][2] * down);
    *reinterpret_cast<float4 *>(w1 + 32 * grp) = make_float4(a[0][1] * down, a[0][3] * down, a[1][1] * down, a[1][3] * down);
  }
}

// ------------------------------------------------------------------ merging
// The prefix's partials of one row of a KV head: n of them, evenly spaced (a
// slot apart, or half a slot with two streams).
struct RowParts {
  const float2 *ml;
  const float *o;
  int n;
};

template <int D>
__device__ __forceinline__ RowParts row_parts(const OwnParams &p, const PrefixPlan &pl, int hkv, int row) {
  RowParts r;
  const int rr = row % (2 * kPrefixBlock), item = hkv * pl.pairs + row / (2 * kPrefixBlock);
  const int c0 = pl.first_cta(item), c1 = pl.last_cta(item);
  const size_t at = (size_t(c0) + item) * 2 + rr / kPrefixBlock;
  r.ml = p.parts.ml + at * kPrefixBlock + rr % kPrefixBlock;
  r.o = p.parts.o + (at * kPrefixBlock + rr % kPrefixBlock / 4 * 4) * D + rr % 4 * 4;
  r.n = (c1 - c0 + 1) * p.streams;
  return r;
}

template <int C>
__device__ __forceinline__ void load_c(const float *p, float *x) {
  if constexpr (C == 4) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const float2 v = *reinterpret_cast<const float2 *>(p);
    x[0] = v.x, x[1] = v.y;
  }
}
template <int C>
__device__ __forceinline__ void store_c(float *p, const float *x) {
  if constexpr (C == 4) *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
  else *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
}

// A softmax state of one row, C channels per lane.
template <int C>
struct LaneState {
  float m = -INFINITY, l = 0.f, o[C];
  __device__ __forceinline__ LaneState() {
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] = 0.f;
  }
  // a warp's state in shared memory: O [8][D], max [8], sum [8]
  __device__ __forceinline__ void read(const float *s, int h, int lane) {
    constexpr int D = 32 * C;
    load_c<C>(s + h * D + C * lane, o);
    m = s[8 * D + h];
    l = s[8 * D + 8 + h];
  }
  __device__ __forceinline__ void add(float m2, float l2, const float *o2) {
    const float mn = fmaxf(m, m2), base = mn == -INFINITY ? 0.f : mn;
    const float f1 = ex2(m - base), f2 = ex2(m2 - base);
    l = l * f1 + l2 * f2;
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] = o[i] * f1 + o2[i] * f2;
    m = mn;
  }
};

// Four rows' softmax states across a warp, as a partial's layout has them: lane
// l holds channels 4 (l/4 + 8i) .. + 3 of row l % 4.
constexpr int kHeads = 4;
template <int D>
struct RowState {
  static constexpr int I = D / 32;
  float m = -INFINITY, l = 0.f, o[I][4];
  __device__ __forceinline__ RowState() {
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  }
  __device__ __forceinline__ static int channel(int lane, int i) { return 4 * (lane / 4 + 8 * i); }
  // a warp's state in shared memory: O [8][D], max [8], sum [8]
  __device__ __forceinline__ void read(const float *s, int h, int lane) {
#pragma unroll
    for (int i = 0; i < I; ++i) load_c<4>(s + h * D + channel(lane, i), o[i]);
    m = s[8 * D + h];
    l = s[8 * D + 8 + h];
  }
  __device__ __forceinline__ void write(float *s, int h, int lane) const {
#pragma unroll
    for (int i = 0; i < I; ++i) store_c<4>(s + h * D + channel(lane, i), o[i]);
    if (lane < 4) s[8 * D + h] = m, s[8 * D + 8 + h] = l;
  }
  __device__ __forceinline__ void add(float m2, float l2, const float (&o2)[I][4]) {
    const float mn = fmaxf(m, m2), base = mn == -INFINITY ? 0.f : mn;
    const float f1 = ex2(m - base), f2 = ex2(m2 - base);
    l = l * f1 + l2 * f2;
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = o[i][e] * f1 + o2[i][e] * f2;
    m = mn;
  }
  __device__ __forceinline__ void write_out(const OwnParams &p, size_t row, int lane) const {
    // no key seen, or a query with a NaN or an infinity, whose sum is NaN: 0,
    // whatever O holds
    const bool seen = l > 0.f;
    const float inv = 1.f / l;
#pragma unroll
    for (int i = 0; i < I; ++i)
      *reinterpret_cast<uint2 *>(p.out + row * D + channel(lane, i)) =
          seen ? make_uint2(pack_bf16x2(o[i][0] * inv, o[i][1] * inv), pack_bf16x2(o[i][2] * inv, o[i][3] * inv))
               : make_uint2(0u, 0u);
    if (lane < 4 && p.lse) p.lse[row] = seen ? (m + __log2f(l)) * 0.6931471805599453f : -INFINITY;
  }
};

// Adds partials first, first + step, .. of the lane's row (a KV head's row) to
// its state.
template <int D>
__device__ __forceinline__ void add_parts(const OwnParams &p, const PrefixPlan &pl, int hkv, int row, int first,
                                          int step, int lane, RowState<D> &st) {
  constexpr int I = D / 32;
  const int ml_step = 2 * kPrefixBlock / p.streams;
  const size_t o_step = size_t(D) * ml_step;
  const RowParts rp = row_parts<D>(p, pl, hkv, row);
  const float *o = rp.o + lane / 4 * 16;
#pragma unroll 3
  for (int s = first; s < rp.n; s += step) {
    const float2 ml = rp.ml[s * ml_step];
    float x[I][4];
#pragma unroll
    for (int i = 0; i < I; ++i) load_c<4>(o + s * o_step + i * 128, x[i]);
    // (a stream without a tile wrote no O)
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i][e] = ml.x == -INFINITY ? 0.f : x[i][e];
    st.add(ml.x, ml.y, x);
  }
}

template <int C>
__device__ __forceinline__ void write_out(const OwnParams &p, size_t row, int lane, const LaneState<C> &st) {
  const bool seen = st.l > 0.f;  // else 0, whatever O holds (see RowState)
  const float inv = 1.f / st.l;
  uint16_t *out = p.out + row * (32 * C) + C * lane;
  if constexpr (C == 4)
    *reinterpret_cast<uint2 *>(out) = seen ? make_uint2(pack_bf16x2(st.o[0] * inv, st.o[1] * inv),
                                                        pack_bf16x2(st.o[2] * inv, st.o[3] * inv))
                                           : make_uint2(0u, 0u);
  else
    *reinterpret_cast<uint32_t *>(out) = seen ? pack_bf16x2(st.o[0] * inv, st.o[1] * inv) : 0u;
  if (lane == 0 && p.lse) p.lse[row] = seen ? (st.m + __log2f(st.l)) * 0.6931471805599453f : -INFINITY;
}

template <int D, int NW, int ST, int kCtas, bool kInline>
__global__ void __launch_bounds__(NW * 32, kCtas) shared_own_kernel(const __grid_constant__ OwnParams p) {
  constexpr int NG = D / 32, C = D / 32;
  using S = Stage<D>;
  static_assert(S::kBytes >= 8 * D * 4 + 64, "a stage holds a warp's state");
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ float *s_state[NW];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const nd_kv_cache &c = p.c;
  const int G = p.G, Hkv = c.n_kv_heads, nslot = c.sink_cap + c.ring_cap, pslot = p.pre.sink_cap + p.pre.ring_cap;
  const uint32_t my_stages = smem_u32(smem) + warp * ST * S::kBytes;
  const int v_inline = kInline ? p.inline_slots : 0, v_all = v_inline + nslot;

  // Behind the prefix kernel (p.early) the CTAs may start while it runs: it let
  // them once what came before it was complete, so the caches and q are final
  // and only its partials have to be waited for.  What is read before that
  // wait goes past L1, which may hold an earlier step's lines.
  bool waited = !p.early;
  if (waited) pdl_wait();

  // ---- copies: a cursor that runs ST - 1 steps ahead of the reads
  // The warp's units in order: solo of its own, then units that the CTA's
  // warps walk together (every fourth step each).
  struct Unit {
    int id, first, n, stride;  // the warp's first virtual slot, steps, slots from one step to its next
    bool solo;
  };
  auto unit_at = [&](int i) {
    Unit u;
    u.solo = i < p.solo;
    u.id = ((u.solo ? i * NW + warp : p.solo * NW + i - p.solo)) * gridDim.x + blockIdx.x;
    const int v0 = p.n_split > 1 ? (u.id % p.n_split) * p.slots_per_unit : 0, v1 = min(v0 + p.slots_per_unit, v_all);
    u.first = u.solo ? v0 : v0 + warp * kStep;
    u.stride = u.solo ? kStep : NW * kStep;
    u.n = u.id < p.n_units && v1 > u.first ? (v1 - u.first + u.stride - 1) / u.stride : 0;
    return u;
  };
  // a lane copies 16-byte chunk my_ch of rows my_row0, my_row0 + kRowStride, ..
  // of K and V, and the scales of one row of K (lanes 0-15) or V
  constexpr int kPerLane = kStep * D / 16 / 32, kRowStride = 32 * 16 / D;
  const int my_row0 = lane / (D / 16), my_ch = lane % (D / 16);
  // scales: a slot's row is 16 bytes, or 8 (D = 64): two slots a copy where a
  // pair's first row is 16-byte aligned (an even number of slots), by lanes
  // 0-7 (K) and 8-15 (V), else one slot a lane
  const bool sc_pairs = D == 64 && !kInline && nslot % 2 == 0;
  const int sc_row = sc_pairs ? (lane & 7) * 2 : lane & 15;
  const bool sc_v = sc_pairs ? lane & 8 : lane & 16;
  struct Source {  // this lane's bytes of a step's rows my_row0 and sc_row
    const int8_t *k, *v;
    const float *s;
  };
  auto source = [&](const nd_kv_cache &from, size_t row) {
    const size_t at = (row + my_row0) * D + my_ch * 16;
    return Source{from.k_codes + at, from.v_codes + at,
                  (sc_v ? from.v_scale : from.k_scale) + (row + sc_row) * NG};
  };
  Source src;    // of the cursor's next step
  Unit at;       // the cursor's unit: its next slot, the steps left
  int at_i = 0;  // its place in the order
  auto seek = [&](int pair) {
    if (kInline && at.first < v_inline) src = source(p.pre, size_t(pair % Hkv) * pslot + at.first);
    else src = source(c, size_t(pair) * nslot + (at.first - v_inline));
  };
  auto enter = [&]() {
    // (a warp whose share of a unit is empty goes on to the next one)
    do at = unit_at(at_i++);
    while (at.n == 0 && at.id < p.n_units);
    if (at.n > 0) seek(p.n_split > 1 ? at.id / p.n_split : at.id);
  };
  enter();
  int in = 0, out = 0;  // stage filled next, stage read next
  // (rows kRowStride apart are 512 bytes apart in the stage; the swizzle of
  // every second one differs in bit 6)
  const uint32_t off0 = swz(uint32_t(my_row0 * D + my_ch * 16));
  const uint32_t off_s = 2 * S::kCodes + (sc_v ? S::kScales : 0) + sc_row * NG * 4;
  auto copy_scale = [&](uint32_t dst, const float *from) {
    if constexpr (NG == 4) {
      cp_async16(dst, from);
    } else if (!sc_pairs) {
      cp_async8(dst, from);
    } else if (lane < 16) {
      cp_async16(dst, from);
    }
  };
  auto issue = [&]() {
    if (at.n > 0) {
      const bool pre = kInline && at.first < v_inline;
      const int base = pre ? at.first : at.first - v_inline, slots = pre ? p.pre.sink_cap : nslot;
      const uint32_t st = my_stages + in * S::kBytes;
      const uint32_t d0 = st + off0, d1 = st + (off0 ^ 64u);
      if (base + kStep <= slots) {
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
          cp_async16((i & 1 ? d1 : d0) + i * 512, src.k + i * kRowStride * D);
          cp_async16((i & 1 ? d1 : d0) + i * 512 + S::kCodes, src.v + i * kRowStride * D);
        }
        copy_scale(st + off_s, src.s);
      } else {  // rows past the end: the last slot, masked
        const int last = slots - 1 - base;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
          const int back = (my_row0 + i * kRowStride - min(my_row0 + i * kRowStride, last)) * D;
          cp_async16((i & 1 ? d1 : d0) + i * 512, src.k + i * kRowStride * D - back);
          cp_async16((i & 1 ? d1 : d0) + i * 512 + S::kCodes, src.v + i * kRowStride * D - back);
        }
        // (last is odd where slots go in pairs)
        copy_scale(st + off_s, src.s - (sc_row - min(sc_row, sc_pairs ? last - 1 : last)) * NG);
      }
      if (++in == ST) in = 0;
      at.first += at.stride;
      if (--at.n == 0) {
        enter();
      } else if (pre && at.first >= v_inline) {
        seek(p.n_split > 1 ? at.id / p.n_split : at.id);
      } else {
        src.k += at.stride * D;
        src.v += at.stride * D;
        src.s += at.stride * NG;
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) issue();

  const int pre_len = kInline ? p.pre.sink_len[0] : 0;
  if (kInline && blockIdx.x == 0 && threadIdx.x == 0 && (pre_len < 0 || pre_len > p.pre.sink_cap))
    raise_device_error(p.err, ND_DEVERR_METADATA);
  const int pre_vis = pre_len >= 0 && pre_len <= p.pre.sink_cap ? pre_len : 0;
  PrefixPlan pl;
  pl.nt = 0;
  if (!kInline && p.prefix_grid > 0)
    pl = prefix_plan(__ldcg(p.pre.sink_len), p.pre.sink_cap, Hkv, c.batch * G, p.prefix_grid);

  // A unit's query and metadata are loaded while the unit before it is walked,
  // or where that costs the walk registers it lacks or a launch is one unit
  // per warp, while it is merged (512 sequences at D = 128: 81.4 us against
  // 83.5; 64 at D = 64: 13.7 against 13.4).
  constexpr bool kEarly = D == 128 && kCtas > 1;
  struct {
    uint4 w[NG];
    int sl, rl, rs;
  } next;
  auto fetch = [&](const Unit &un) {
    if (un.id >= p.n_units) return;
    const int pair = p.n_split > 1 ? un.id / p.n_split : un.id, b = pair / Hkv, hkv = pair - b * Hkv;
    const uint16_t *qh = p.q + (size_t(b) * p.Hq + hkv * G + (g < G ? g : 0)) * D;
#pragma unroll
    for (int grp = 0; grp < NG; ++grp)
      next.w[grp] = g < G ? __ldcg(reinterpret_cast<const uint4 *>(qh + 32 * grp + 8 * t)) : make_uint4(0, 0, 0, 0);
    next.sl = __ldcg(c.sink_len + b), next.rl = __ldcg(c.ring_len + b), next.rs = __ldcg(c.ring_start + b);
  };
  Unit un = unit_at(0);
  fetch(un);
  for (int i = 1; un.id < p.n_units; ++i) {  // (units of the whole CTA: the same for its warps)
    const int pair = p.n_split > 1 ? un.id / p.n_split : un.id, b = pair / Hkv, hkv = pair - b * Hkv;
    HeadQ<D> hq;
    make_q<D>(next.w, hq);
    int sl = next.sl, rl = next.rl, rs = next.rs;
    const bool sane = sl >= 0 && sl <= c.sink_cap && rl >= 0 && rl <= c.ring_cap && rs >= 0 &&
                      (c.ring_cap == 0 || rs < c.ring_cap);
    if (!sane) {
      if (lane == 0) raise_device_error(p.err, ND_DEVERR_METADATA);
      sl = rl = rs = 0;
    }
    const int n_vis = min(rl, p.window);
    int rs_eff = rs + rl - n_vis;  // oldest visible entry
    if (rs_eff >= c.ring_cap) rs_eff -= c.ring_cap;

    const Unit un_next = unit_at(i);
    if (kEarly) fetch(un_next);
    RunState<D> run;
    int v = un.first;
    for (int s = 0; s < un.n; ++s, v += un.stride) {
      issue();
      cp_async_wait<ST - 1>();
      __syncwarp();
      const bool pre = kInline && v < v_inline;
      const int base = pre ? v : v - v_inline;
      const bool all_vis = pre ? base + kStep <= pre_vis
                               : base + kStep <= nslot &&
                                     (base + kStep <= sl || (base >= c.sink_cap && n_vis == c.ring_cap));
      uint32_t vis = 0xfu;
      if (!all_vis) {
        vis = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int ps = base + 2 * t + (i & 1) + 8 * (i >> 1);
          bool on;
          if (pre) on = ps < pre_vis;
          else if (ps < c.sink_cap) on = ps < sl;
          else {
            int age = ps - c.sink_cap - rs_eff;
            if (age < 0) age += c.ring_cap;
            on = ps < nslot && age < n_vis;
          }
          vis |= uint32_t(on) << i;
        }
      }
      attend_step<D>(my_stages + out * S::kBytes, hq, all_vis, vis, lane, run);
      __syncwarp();  // every lane is done with this stage before it is refilled
      if (++out == ST) out = 0;
    }

    // ---- merge.  The stage that the next copy will fill is free until then.
    float *state = reinterpret_cast<float *>(smem + (warp * ST + in) * S::kBytes);  // [8][D], max [8], sum [8]
    store_state<D>(run, lane, state, state + 8 * D, state + 8 * D + 8);
    if (!kEarly) fetch(un_next);
    __syncwarp();
    // the prefix's partials: all of them for a unit of the warp's own, else
    // this warp's share, folded into its state
    if (un.solo || (pl.nt > 0 && p.n_split == 1)) {
      if (!waited) pdl_wait();
      waited = true;
      for (int h0 = 0; h0 < G; h0 += kHeads) {
        const int h = h0 + lane % kHeads;
        const bool live = h < G;
        RowState<D> st;
        if (live) {
          st.read(state, h, lane);
          if (pl.nt > 0) add_parts<D>(p, pl, hkv, b * G + h, un.solo ? 0 : warp, un.solo ? 1 : NW, lane, st);
          if (un.solo) st.write_out(p, size_t(b) * p.Hq + hkv * G + h, lane);
        }
        if (!un.solo) {
          // eight lanes read a head's (max, sum) and one of them writes it back;
          // the rows of a group may have different numbers of partials, so the
          // lanes need not come out of the loop above together
          __syncwarp();
          if (live) st.write(state, h, lane);
        }
      }
    }
    if (un.solo) {
      __syncwarp();  // the state is read before its stage is filled again
      un = un_next;
      continue;
    }
    if (lane == 0) s_state[warp] = state;
    __syncthreads();
    for (int h = warp; h < G; h += NW) {
      LaneState<C> st;
#pragma unroll 4
      for (int w = 0; w < NW; ++w) {
        LaneState<C> other;
        other.read(s_state[w], h, lane);
        st.add(other.m, other.l, other.o);
      }
      if (p.n_split > 1) {
        const size_t part = size_t(un.id) * G + h;
        store_c<C>(p.ws_o + part * D + C * lane, st.o);
        if (lane == 0) {
          p.ws_ml[2 * part] = st.m;
          p.ws_ml[2 * part + 1] = st.l;
        }
      } else {
        write_out<C>(p, size_t(b) * p.Hq + hkv * G + h, lane, st);
      }
    }
    __syncthreads();  // the states are read before their stages are filled again
    un = un_next;
  }
  cp_async_wait<0>();
  if (!waited) pdl_wait();  // this kernel is complete only after the one before it
}

// Joins the parts of each pair and the prefix's partials: a CTA per pair, a
// warp takes every eighth of a row's sources, then the warps' states meet in
// shared memory.
constexpr int kMergeWarps = 8;
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) shared_merge_kernel(const __grid_constant__ OwnParams p) {
  constexpr int C = D / 32;
  __shared__ __align__(16) float s_o[8][kMergeWarps][D];
  __shared__ float s_ml[8][kMergeWarps][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pair = blockIdx.x, Hkv = p.c.n_kv_heads, G = p.G, b = pair / Hkv, hkv = pair % Hkv;
  pdl_wait();
  PrefixPlan pl;
  pl.nt = 0;
  if (p.prefix_grid > 0)
    pl = prefix_plan(p.pre.sink_len[0], p.pre.sink_cap, Hkv, p.c.batch * G, p.prefix_grid);
  for (int h0 = 0; h0 < G; h0 += kHeads) {
    const int h = h0 + lane % kHeads;
    if (h >= G) continue;
    RowState<D> st;
    for (int s = warp; s < p.n_split; s += kMergeWarps) {
      const size_t part = (size_t(pair) * p.n_split + s) * G + h;
      float x[C][4];
#pragma unroll
      for (int i = 0; i < C; ++i) load_c<4>(p.ws_o + part * D + RowState<D>::channel(lane, i), x[i]);
      st.add(p.ws_ml[2 * part], p.ws_ml[2 * part + 1], x);
    }
    // (the first partials go to the warps that the parts left out)
    if (pl.nt > 0)
      add_parts<D>(p, pl, hkv, b * G + h, (warp + kMergeWarps - p.n_split % kMergeWarps) % kMergeWarps, kMergeWarps, lane,
                   st);
#pragma unroll
    for (int i = 0; i < C; ++i) store_c<4>(&s_o[h][warp][RowState<D>::channel(lane, i)], st.o[i]);
    if (lane < 4) s_ml[h][warp][0] = st.m, s_ml[h][warp][1] = st.l;
  }
  __syncthreads();
  for (int h = warp; h < G; h += kMergeWarps) {
    LaneState<C> st;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
      float x[C];
      load_c<C>(&s_o[h][w][C * lane], x);
      st.add(s_ml[h][w][0], s_ml[h][w][1], x);
    }
    write_out<C>(p, size_t(b) * p.Hq + hkv * G + h, lane, st);
  }
}

template <int D, int NW, int ST, int kCtas, bool kInline>
cudaError_t launch_own(OwnParams &p, cudaStream_t stream) {
  constexpr size_t smem = size_t(NW) * ST * Stage<D>::kBytes;
  auto kern = shared_own_kernel<D, NW, ST, kCtas, kInline>;
  static std::atomic<unsigned long long> smem_set{0};  // the opt-in, once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
  if (!bit || !(smem_set.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    smem_set.fetch_or(bit, std::memory_order_release);
  }
  const int most = kPrefixCtas * kCtas, grid = p.n_units < most ? p.n_units : most;
  // Whole rounds of the warps take a unit each.  The rest is one more such
  // round, or shared: a CTA's warps then need a fourth of the steps, but each
  // round of theirs has its own start and merge (about seven steps' time; 128
  // sequences of 256 slots: one round alone 21 us, three together 36 us).
  const int steps = p.slots_per_unit / kStep, warps = grid * NW, rest = p.n_units % warps;
  const int rounds = (rest + grid - 1) / grid;
  p.solo = p.n_units / warps;
  if (p.n_split == 1 && steps + 7 < rounds * ((steps + NW - 1) / NW + 7)) ++p.solo;
  return launch_pdl(kern, dim3(unsigned(grid)), dim3(NW * 32), smem, stream, p);
}

// How a call is carried out; the workspace query and the launch agree on it.
struct SharedPlan {
  bool inline_prefix;
  int n_split, slots_per_unit, inline_slots;
  bool wide;  // more warps per unit: few units
  int ctas;   // of the prefix kernel, at most
};

constexpr int kSpareTiles = 6;  // see below

SharedPlan shared_plan(int batch, int G, int n_kv_heads, int head_dim, int prefix_cap, int max_slots) {
  SharedPlan s;
  const long long pairs = (long long)batch * n_kv_heads;
  // The grids and the workspace have to be, so the path is chosen from the
  // prefix's capacity; a short prefix in a long region takes the path of the
  // long one (128 pairs of 128, 300 slots: in a region of 300 8.4 us, of 512
  // 9.9, of 600 to 65536 13.6; 512 pairs 25.8, 25.6 and 25.8 to 26.7).
  // A prefix of up to 512 slots for up to 152 pairs is read again by each of
  // them (2 heads of 64: 64 slots 5.6 us against 10.2; 152 pairs of 128: 256
  // slots 8.2 against 13.7, 512 slots 10.0 against 13.9; 64 pairs of 64: 512
  // slots 7.3 against 8.7, 768 slots 9.3 against 8.7.  256 pairs of 128: 256
  // slots 13.9 against 11.1).
  s.inline_prefix = pairs <= kPrefixCtas && prefix_cap <= 512;
  s.inline_slots = s.inline_prefix ? (prefix_cap + kStep - 1) / kStep * kStep : 0;
  // One CTA of more warps to an SM where the pairs are few, and up to twice
  // the SMs where a pair's walk is long (64 pairs of 128 over 256 slots 16.5 us
  // against 21.5 with three CTAs of four; 192 pairs of 64 over 1024 slots 23.3
  // against 33.6, over 512 20.2 against 23.8, over 256 18.8 against 18.9; 456
  // of 128 over 512 35.7 against 29.7).
  s.wide = pairs <= kPrefixCtas || (pairs <= 2 * kPrefixCtas && max_slots >= 512);
  const int warps = s.wide ? (head_dim == 64 ? 16 : 8) : 4;
  const int steps = (s.inline_slots + max_slots + kStep - 1) / kStep;
  // parts of a pair where the pairs leave SMs idle, each at least two steps
  // of each of its warps
  const long long want = pairs * 2 > kPrefixCtas ? 1 : kPrefixCtas / pairs, cap = steps / (2 * warps);
  const long long n = want < cap ? want : cap;
  s.n_split = n > 1 ? int(n) : 1;
  s.slots_per_unit = (steps + s.n_split - 1) / s.n_split * kStep;
  s.n_split = (steps * kStep + s.slots_per_unit - 1) / s.slots_per_unit;
  // The own part starts beside the prefix kernel where that leaves it SMs: a
  // CTA walks its unit meanwhile and waits only to merge, which saves 3 to 4
  // us.  Worth six more tiles per CTA of the prefix, at 0.45 (D = 64) to 0.55
  // us each (32 pairs of 128 over 4096 slots 12.6 us against 16.2; 128 of 64
  // over 4096, 5 tiles: 12.6 against 13.6; 64 of 128 over 32768, 8 tiles: 31.0
  // against 29.7).
  const long long own = pairs * s.n_split, tiles = (long long)n_kv_heads * prefix_pairs(batch * G) *
                                                   ((prefix_cap + kPrefixTile - 1) / kPrefixTile);
  s.ctas = kPrefixCtas;
  if (own <= kPrefixCtas - 8 &&
      (tiles + kPrefixCtas - own - 1) / (kPrefixCtas - own) <= (tiles + kPrefixCtas - 1) / kPrefixCtas + kSpareTiles)
    s.ctas = int(kPrefixCtas - own);
  return s;
}

}  // namespace

size_t shared_decode_workspace_bytes(int batch, int n_q_heads, int n_kv_heads, int head_dim, int prefix_cap,
                                     int max_slots) {
  const int G = n_q_heads / n_kv_heads;
  const SharedPlan s = shared_plan(batch, G, n_kv_heads, head_dim, prefix_cap, max_slots);
  size_t rows = s.n_split > 1 ? size_t(batch) * n_q_heads * s.n_split : 0;
  if (!s.inline_prefix) rows += prefix_slots(prefix_cap, n_kv_heads, batch * G, s.ctas) * 2 * kPrefixBlock;
  return rows * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_shared_decode(const void *q, const nd_kv_cache &prefix, const nd_kv_cache &c, int n_q_heads,
                                 int window, void *out, float *lse, void *ws, int *err, cudaStream_t stream) {
  const int d = c.head_dim, G = n_q_heads / c.n_kv_heads, rows = c.batch * G;
  const SharedPlan s = shared_plan(c.batch, G, c.n_kv_heads, d, prefix.sink_cap, c.sink_cap + c.ring_cap);
  OwnParams p;
  p.q = static_cast<const uint16_t *>(q);
  p.c = c;
  p.pre = prefix;
  p.Hq = n_q_heads;
  p.G = G;
  p.window = window;
  p.n_split = s.n_split;
  p.slots_per_unit = s.slots_per_unit;
  p.n_units = c.batch * c.n_kv_heads * s.n_split;
  p.inline_slots = s.inline_slots;
  p.out = static_cast<uint16_t *>(out);
  p.lse = lse;
  p.err = err;
  p.parts = {nullptr, nullptr};
  p.prefix_grid = 0;
  p.streams = prefix_streams(rows);
  // (at D = 64 an odd number of slots needs copies that go through L1)
  p.early = !s.inline_prefix && (d == 128 || (c.sink_cap + c.ring_cap) % 2 == 0);
  float *w = static_cast<float *>(ws);
  cudaError_t e;
  if (!s.inline_prefix) {
    const size_t pre_rows = prefix_slots(prefix.sink_cap, c.n_kv_heads, rows, s.ctas) * 2 * kPrefixBlock;
    p.parts.o = w;
    p.parts.ml = reinterpret_cast<float2 *>(w + pre_rows * d);
    p.prefix_grid = prefix_grid(prefix.sink_cap, c.n_kv_heads, rows, s.ctas);
    w += pre_rows * (d + 2);
    e = launch_shared_prefix(q, prefix, c.batch, n_q_heads, p.prefix_grid, p.parts, err, stream);
    if (e != cudaSuccess) return e;
  }
  p.ws_o = w;
  p.ws_ml = w + size_t(c.batch) * n_q_heads * s.n_split * d;
  if (d == 128) {
    e = s.inline_prefix ? launch_own<128, 8, 4, 1, true>(p, stream)
        : s.wide        ? launch_own<128, 8, 4, 1, false>(p, stream)
                        : launch_own<128, 4, 4, 3, false>(p, stream);
  } else {
    e = s.inline_prefix ? launch_own<64, 16, 4, 1, true>(p, stream)
        : s.wide        ? launch_own<64, 16, 4, 1, false>(p, stream)
                        : launch_own<64, 4, 4, 5, false>(p, stream);
  }
  if (e != cudaSuccess || s.n_split == 1) return e;
  return launch_pdl(d == 128 ? shared_merge_kernel<128> : shared_merge_kernel<64>,
                    dim3(unsigned(c.batch) * c.n_kv_heads), dim3(kMergeWarps * 32), 0, stream, p);
}

}  // namespace nd
