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
// and ending as reading.  Here a CTA walks several units one after the other,
// and its copies run on across the boundary: while a unit is merged and
// written, the next one's steps are in flight.  The merge needs no memory of
// its own: of a warp's ST stages ST - 1 are being filled, and the one just
// read holds its state.
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
  int inline_slots;    // prefix slots walked by every unit (a multiple of kStep), or 0
  uint16_t *out;
  float *lse;
  float *ws_ml, *ws_o; // n_split > 1: [pair][n_split][G][2], [..][G][D]
  PrefixParts parts;   // the prefix's partials, when prefix_grid > 0
  int prefix_grid;
  int *err;
};

// The prefix's partials of one row of a KV head: n of them, in adjacent slots.
struct RowParts {
  const float2 *ml;
  const float *o;
  int n;
};
constexpr size_t kMlStep = 2 * kPrefixBlock;  // from one slot's (max, sum) to the next one's

template <int D>
__device__ __forceinline__ RowParts row_parts(const OwnParams &p, const PrefixPlan &pl, int hkv, int row) {
  RowParts r;
  const int rr = row % (2 * kPrefixBlock), item = hkv * pl.pairs + row / (2 * kPrefixBlock);
  const int c0 = pl.owner((long long)item * pl.nt), c1 = pl.owner((long long)(item + 1) * pl.nt - 1);
  const size_t at = (size_t(c0) + item) * 2 + rr / kPrefixBlock;
  r.ml = p.parts.ml + at * kPrefixBlock + rr % kPrefixBlock;
  r.o = p.parts.o + (at * (D / 4) * kPrefixBlock + rr % kPrefixBlock) * 4;
  r.n = c1 - c0 + 1;
  return r;
}

// A softmax state of one row, C channels per lane.
template <int C>
struct LaneState {
  float m = -INFINITY, l = 0.f, o[C];
  __device__ __forceinline__ LaneState() {
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] = 0.f;
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

// Adds partials first, first + step, .. of the row to the state (four loads in
// flight).  Lane l holds channels C*l .. (C = D / 32): in a partial's
// [D/4][128][4] layout, C floats of group C*l/4.
template <int D>
__device__ __forceinline__ void add_parts(const RowParts &rp, int first, int step, int lane, LaneState<D / 32> &st) {
  constexpr int C = D / 32;
  const size_t o_step = size_t(D) * 2 * kPrefixBlock;
  const float *o = rp.o + size_t(C * lane / 4) * kPrefixBlock * 4 + (C * lane) % 4;
  for (int s0 = first; s0 < rp.n; s0 += 4 * step) {
    float2 ml[4];
    float x[4][C];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int s = s0 + u * step;
      if (s < rp.n) {
        ml[u] = rp.ml[s * kMlStep];
        load_c<C>(o + s * o_step, x[u]);
      } else {
        ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int i = 0; i < C; ++i) x[u][i] = 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) st.add(ml[u].x, ml[u].y, x[u]);
  }
}

template <int C>
__device__ __forceinline__ void write_out(const OwnParams &p, size_t row, int lane, const LaneState<C> &st) {
  const float inv = st.l > 0.f ? 1.f / st.l : 0.f;
  uint16_t *out = p.out + row * (32 * C) + C * lane;
  if constexpr (C == 4)
    *reinterpret_cast<uint2 *>(out) = make_uint2(pack_bf16x2(st.o[0] * inv, st.o[1] * inv),
                                                 pack_bf16x2(st.o[2] * inv, st.o[3] * inv));
  else
    *reinterpret_cast<uint32_t *>(out) = pack_bf16x2(st.o[0] * inv, st.o[1] * inv);
  if (lane == 0 && p.lse) p.lse[row] = st.l > 0.f ? (st.m + __log2f(st.l)) * 0.6931471805599453f : -INFINITY;
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

  pdl_wait();

  // ---- copies: a cursor (unit, step) that runs ST - 1 steps ahead
  struct {
    int unit, step, n, first;  // first: the unit's first virtual slot of this warp
    size_t own, pre;           // row of the pair's (head's) slot 0
  } at;
  auto steps_of = [&](int unit, int &first) {
    const int v0 = (unit % p.n_split) * p.slots_per_unit, v1 = min(v0 + p.slots_per_unit, v_all);
    first = v0 + warp * kStep;
    return v1 > first ? (v1 - first + NW * kStep - 1) / (NW * kStep) : 0;
  };
  auto enter = [&](int unit) {
    at.unit = unit;
    at.step = 0;
    while (at.unit < p.n_units && (at.n = steps_of(at.unit, at.first)) == 0) at.unit += gridDim.x;
    if (at.unit < p.n_units) {
      const int pair = at.unit / p.n_split;
      at.own = size_t(pair) * nslot;
      at.pre = size_t(pair % Hkv) * pslot;
    }
  };
  enter(blockIdx.x);
  int in = 0, out = 0;  // stage filled next, stage read next
  constexpr int kPerLane = kStep * D / 16 / 32, kRowStride = 32 * 16 / D;
  const int my_row0 = lane / (D / 16), my_ch = lane % (D / 16);
  auto issue = [&]() {
    if (at.unit < p.n_units) {
      const int v = at.first + at.step * NW * kStep;
      const bool pre = kInline && v < v_inline;
      const nd_kv_cache &src = pre ? p.pre : c;
      // slots past the region's end read its last one (and are masked)
      const int base = pre ? v : v - v_inline, last = (pre ? p.pre.sink_cap : nslot) - 1;
      const size_t row = pre ? at.pre : at.own;
      const uint32_t st = my_stages + in * S::kBytes;
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) {
        const int r = my_row0 + k * kRowStride;
        const uint32_t off = swz(uint32_t(r * D + my_ch * 16));
        const size_t goff = (row + min(base + r, last)) * D + my_ch * 16;
        cp_async16(st + off, src.k_codes + goff);
        cp_async16(st + S::kCodes + off, src.v_codes + goff);
      }
      const int r = lane & 15, which = lane >> 4;
      const uint32_t dst = st + 2 * S::kCodes + which * S::kScales + r * NG * 4;
      const float *sc = (which ? src.v_scale : src.k_scale) + (row + min(base + r, last)) * NG;
      if constexpr (NG == 4) cp_async16(dst, sc);
      else cp_async8(dst, sc);
      if (++in == ST) in = 0;
      if (++at.step == at.n) enter(at.unit + gridDim.x);
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
    pl = prefix_plan(p.pre.sink_len[0], p.pre.sink_cap, Hkv, c.batch * G, p.prefix_grid);

  for (int unit = blockIdx.x; unit < p.n_units; unit += gridDim.x) {
    const int pair = unit / p.n_split, b = pair / Hkv, hkv = pair % Hkv;
    int first;
    const int n = steps_of(unit, first);
    // ---- the unit's query and metadata
    HeadQ<D> hq;
    {
      uint4 w[NG];
      const uint16_t *qh = p.q + (size_t(b) * p.Hq + hkv * G + (g < G ? g : 0)) * D;
#pragma unroll
      for (int grp = 0; grp < NG; ++grp)
        w[grp] = g < G ? *reinterpret_cast<const uint4 *>(qh + 32 * grp + 8 * t) : make_uint4(0, 0, 0, 0);
      make_q<D>(w, hq);
    }
    int sl = c.sink_len[b], rl = c.ring_len[b], rs = c.ring_start[b];
    const bool sane = sl >= 0 && sl <= c.sink_cap && rl >= 0 && rl <= c.ring_cap && rs >= 0 &&
                      (c.ring_cap == 0 || rs < c.ring_cap);
    if (!sane) {
      if (threadIdx.x == 0) raise_device_error(p.err, ND_DEVERR_METADATA);
      sl = rl = rs = 0;
    }
    const int n_vis = min(rl, p.window);
    const int rs_eff = c.ring_cap ? (rs + rl - n_vis) % c.ring_cap : 0;  // oldest visible entry

    RunState<D> run;
    for (int s = 0; s < n; ++s) {
      issue();
      cp_async_wait<ST - 1>();
      __syncwarp();
      const int v = first + s * NW * kStep;
      const bool pre = kInline && v < v_inline;
      const int base = pre ? v : v - v_inline;
      const bool all_vis = pre ? base + kStep <= pre_vis
                               : base + kStep <= nslot &&
                                     (base + kStep <= sl || (base >= c.sink_cap && n_vis == c.ring_cap));
      bool vis[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ps = base + 2 * t + (i & 1) + 8 * (i >> 1);
        if (all_vis) vis[i] = true;
        else if (pre) vis[i] = ps < pre_vis;
        else if (ps < c.sink_cap) vis[i] = ps < sl;
        else {
          int age = ps - c.sink_cap - rs_eff;
          if (age < 0) age += c.ring_cap;
          vis[i] = ps < nslot && age < n_vis;
        }
      }
      attend_step<D>(my_stages + out * S::kBytes, hq, vis, g < G, lane, run);
      __syncwarp();  // every lane is done with this stage before it is refilled
      if (++out == ST) out = 0;
    }

    // ---- merge.  The stage that the next copy will fill is free until then.
    float *state = reinterpret_cast<float *>(smem + (warp * ST + in) * S::kBytes);  // [8][D], max [8], sum [8]
    if (lane == 0) s_state[warp] = state;
    store_state<D>(run, lane, state, state + 8 * D, state + 8 * D + 8);
    __syncthreads();
    for (int h = warp; h < G; h += NW) {
      LaneState<C> st;
#pragma unroll 4
      for (int w = 0; w < NW; ++w) {
        const float *sw = s_state[w];
        float x[C];
        load_c<C>(sw + h * D + C * lane, x);
        st.add(sw[8 * D + h], sw[8 * D + 8 + h], x);
      }
      if (p.n_split > 1) {
        const size_t part = size_t(unit) * G + h;
        store_c<C>(p.ws_o + part * D + C * lane, st.o);
        if (lane == 0) {
          p.ws_ml[2 * part] = st.m;
          p.ws_ml[2 * part + 1] = st.l;
        }
      } else {
        if (pl.nt > 0) add_parts<D>(row_parts<D>(p, pl, hkv, b * G + h), 0, 1, lane, st);
        write_out<C>(p, size_t(b) * p.Hq + hkv * G + h, lane, st);
      }
    }
    __syncthreads();  // the states are read before their stages are filled again
  }
  cp_async_wait<0>();
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
  for (int h = 0; h < G; ++h) {
    LaneState<C> st;
    for (int s = warp; s < p.n_split; s += kMergeWarps) {
      const size_t part = (size_t(pair) * p.n_split + s) * G + h;
      float x[C];
      load_c<C>(p.ws_o + part * D + C * lane, x);
      st.add(p.ws_ml[2 * part], p.ws_ml[2 * part + 1], x);
    }
    // (the first sources go to the warps that the parts left out)
    if (pl.nt > 0)
      add_parts<D>(row_parts<D>(p, pl, hkv, b * G + h), (warp + kMergeWarps - p.n_split % kMergeWarps) % kMergeWarps,
                   kMergeWarps, lane, st);
    store_c<C>(&s_o[h][warp][C * lane], st.o);
    if (lane == 0) s_ml[h][warp][0] = st.m, s_ml[h][warp][1] = st.l;
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
cudaError_t launch_own(const OwnParams &p, cudaStream_t stream) {
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
  const int most = kPrefixCtas * kCtas;
  return launch_pdl(kern, dim3(unsigned(p.n_units < most ? p.n_units : most)), dim3(NW * 32), smem, stream, p);
}

// How a call is carried out; the workspace query and the launch agree on it.
struct SharedPlan {
  bool inline_prefix;
  int n_split, slots_per_unit, inline_slots;
  bool wide;  // more warps per unit: few units
};

SharedPlan shared_plan(int batch, int n_kv_heads, int head_dim, int prefix_cap, int max_slots) {
  SharedPlan s;
  const long long pairs = (long long)batch * n_kv_heads;
  // A prefix of up to 256 slots for up to 152 pairs is read again by each.
  s.inline_prefix = pairs <= kPrefixCtas && prefix_cap <= 256;
  s.inline_slots = s.inline_prefix ? (prefix_cap + kStep - 1) / kStep * kStep : 0;
  s.wide = pairs <= kPrefixCtas;
  const int warps = s.wide ? (head_dim == 64 ? 16 : 8) : 4;
  const int steps = (s.inline_slots + max_slots + kStep - 1) / kStep;
  // parts of a pair where the pairs leave SMs idle, each at least two steps
  // of each of its warps
  const long long want = pairs * 2 > kPrefixCtas ? 1 : kPrefixCtas / pairs, cap = steps / (2 * warps);
  const long long n = want < cap ? want : cap;
  s.n_split = n > 1 ? int(n) : 1;
  s.slots_per_unit = (steps + s.n_split - 1) / s.n_split * kStep;
  s.n_split = (steps * kStep + s.slots_per_unit - 1) / s.slots_per_unit;
  return s;
}

}  // namespace

size_t shared_decode_workspace_bytes(int batch, int n_q_heads, int n_kv_heads, int head_dim, int prefix_cap,
                                     int max_slots) {
  const SharedPlan s = shared_plan(batch, n_kv_heads, head_dim, prefix_cap, max_slots);
  size_t rows = s.n_split > 1 ? size_t(batch) * n_q_heads * s.n_split : 0;
  if (!s.inline_prefix) rows += prefix_slots(prefix_cap, n_kv_heads, batch * (n_q_heads / n_kv_heads)) * 2 * kPrefixBlock;
  return rows * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_shared_decode(const void *q, const nd_kv_cache &prefix, const nd_kv_cache &c, int n_q_heads,
                                 int window, void *out, float *lse, void *ws, int *err, cudaStream_t stream) {
  const int d = c.head_dim, G = n_q_heads / c.n_kv_heads, rows = c.batch * G;
  const SharedPlan s = shared_plan(c.batch, c.n_kv_heads, d, prefix.sink_cap, c.sink_cap + c.ring_cap);
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
  float *w = static_cast<float *>(ws);
  cudaError_t e;
  if (!s.inline_prefix) {
    const size_t pre_rows = prefix_slots(prefix.sink_cap, c.n_kv_heads, rows) * 2 * kPrefixBlock;
    p.parts.o = w;
    p.parts.ml = reinterpret_cast<float2 *>(w + pre_rows * d);
    p.prefix_grid = prefix_grid(prefix.sink_cap, c.n_kv_heads, rows);
    w += pre_rows * (d + 2);
    e = launch_shared_prefix(q, prefix, c.batch, n_q_heads, p.parts, err, stream);
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
