// tree_decode.cu -- attention of a tree of drafted tokens: every node against
// its sequence's int8 cache and the nodes its mask names, in one softmax.
//
//   s_j = (q . k_j) log2(e) / sqrt(D),  out = sum_j 2^(s_j - m) v_j / l,
//   m = max_j s_j,  l = sum_j 2^(s_j - m)
//
// over the filled sinks, the ring entries whose position is less than `window`
// below the node's, and the mask's nodes, in one pass with a running m, l and
// sum.  One warp to a (node, query head), a lane to D/32 channels.
#include "nd_common.cuh"
#include "nd_internal.h"

namespace nd {

namespace {

struct TreeParams {
  const uint16_t *q, *k, *v;
  int64_t k_stride, v_stride;
  nd_kv_cache c;
  const int32_t *depth;
  const uint32_t *mask;
  int n, Hq, G, window;
  uint16_t *out;
  float *lse;
  int *err;
};

template <int D>
__global__ void __launch_bounds__(128) tree_rows_kernel(const __grid_constant__ TreeParams p) {
  constexpr int CPL = D / 32;
  const nd_kv_cache &c = p.c;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  const int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);  // (b * n + i) * Hq + h
  if (row >= int64_t(c.batch) * p.n * p.Hq) return;
  const int h = int(row % p.Hq);
  const int64_t node = row / p.Hq;
  const int b = int(node / p.n), i = int(node % p.n), hk = h / p.G, words = (p.n + 31) / 32;
  const int sl = c.sink_len[b], rs = c.ring_start[b], rl = c.ring_len[b], depth = p.depth[node];
  const bool sane = sl >= 0 && sl <= c.sink_cap && rl >= 0 && rl <= c.ring_cap && rs >= 0 && (c.ring_cap == 0 || rs < c.ring_cap);
  if (!sane && lane == 0) raise_device_error(p.err, ND_DEVERR_METADATA);
  float q[CPL], o[CPL], m = -INFINITY, l = 0.f;
  bool finite = true;
#pragma unroll
  for (int e = 0; e < CPL; ++e) {
    q[e] = __uint_as_float(uint32_t(p.q[row * D + lane * CPL + e]) << 16) * (1.4426950408889634f * rsqrtf(float(D)));
    o[e] = 0.f;
    finite = finite && fabsf(q[e]) < INFINITY;
  }
  finite = __all_sync(0xffffffffu, finite);
  auto take = [&](const float *k, const float *v) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < CPL; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const float mn = fmaxf(m, s), a = ex2(m - mn), w = ex2(s - mn);
    m = mn;
    l = fmaf(l, a, w);
#pragma unroll
    for (int e = 0; e < CPL; ++e) o[e] = fmaf(o[e], a, w * v[e]);
  };
  auto slot = [&](int s) {
    const int64_t at = (int64_t(b) * c.n_kv_heads + hk) * (int64_t(c.sink_cap) + c.ring_cap) + s;
    const int grp = lane * CPL / 32;
    const float ks = c.k_scale[at * (D / 32) + grp], vs = c.v_scale[at * (D / 32) + grp];
    float k[CPL], v[CPL];
#pragma unroll
    for (int e = 0; e < CPL; ++e) {
      k[e] = float(c.k_codes[at * D + lane * CPL + e]) * ks;
      v[e] = float(c.v_codes[at * D + lane * CPL + e]) * vs;
    }
    take(k, v);
  };
  if (sane && finite && depth >= 0) {
    for (int s = 0; s < sl; ++s) slot(s);
    const int reach = max(0, min(rl, p.window - 1 - depth));
    for (int e = rl - reach; e < rl; ++e) slot(c.sink_cap + int((int64_t(rs) + e) % c.ring_cap));
    for (int j = 0; j < p.n; ++j) {
      if (!(p.mask[node * words + j / 32] >> (j % 32) & 1u) || p.depth[int64_t(b) * p.n + j] < 0) continue;
      const int64_t at = int64_t(b) * p.n + j;
      float k[CPL], v[CPL];
#pragma unroll
      for (int e = 0; e < CPL; ++e) {
        k[e] = __uint_as_float(uint32_t(p.k[at * p.k_stride + hk * D + lane * CPL + e]) << 16);
        v[e] = __uint_as_float(uint32_t(p.v[at * p.v_stride + hk * D + lane * CPL + e]) << 16);
      }
      take(k, v);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < CPL; ++e) p.out[row * D + lane * CPL + e] = __bfloat16_as_ushort(__float2bfloat16_rn(o[e] * inv));
  if (p.lse && lane == 0) p.lse[(int64_t(b) * p.Hq + h) * p.n + i] = l > 0.f ? 0.6931471805599453f * (m + log2f(l)) : -INFINITY;
}

}  // namespace

size_t tree_decode_workspace_bytes(int batch, int n, int n_q_heads, int n_kv_heads, int head_dim, int max_slots) { return 0; }

cudaError_t launch_tree_decode(const TreeDecodeArgs &a, const nd_kv_cache &c, void *ws, int *err, cudaStream_t stream) {
  TreeParams p;
  p.q = static_cast<const uint16_t *>(a.q);
  p.k = static_cast<const uint16_t *>(a.k);
  p.v = static_cast<const uint16_t *>(a.v);
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.c = c;
  p.depth = a.depth;
  p.mask = a.mask;
  p.n = a.n;
  p.Hq = a.n_q_heads;
  p.G = a.n_q_heads / c.n_kv_heads;
  p.window = a.window;
  p.out = static_cast<uint16_t *>(a.out);
  p.lse = a.lse;
  p.err = err;
  const int64_t rows = int64_t(c.batch) * a.n * a.n_q_heads;
  const dim3 grid(unsigned((rows + 3) / 4));
  return c.head_dim == 64 ? launch_pdl(tree_rows_kernel<64>, grid, dim3(128), 0, stream, p)
                          : launch_pdl(tree_rows_kernel<128>, grid, dim3(128), 0, stream, p);
}

}  // namespace nd
