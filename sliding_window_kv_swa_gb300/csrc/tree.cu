// tree.cu -- trees of drafted tokens: their layout from the parents, the
// longest path that the model agrees with, and that path's append to the ring.
//
// All three are chains of latencies over a few kilobytes per sequence, so a
// sequence is one CTA (the commit: up to a cluster of eight) and its nodes live in
// shared memory.
#include "nd_common.cuh"
#include "nd_internal.h"

namespace nd {

namespace {

constexpr int kMaxNodes = ND_TREE_MAX_NODES;

// The sequence's nodes, 0 when n_nodes is out of range.
__device__ __forceinline__ int node_count(const int32_t *n_nodes, int b, int n, int *err) {
  const int m = n_nodes ? n_nodes[b] : n;
  if (m >= 0 && m <= n) return m;
  if (threadIdx.x == 0) raise_device_error(err, ND_DEVERR_METADATA);
  return 0;
}

// A thread per node walks up to its root: the steps are the depth, the first
// `window` nodes on the way the mask.  One sequence of 8 nodes 1.8 us, 512 of 256
// nodes (depths to 80; 5.2 MB written) 8.7 to 9.4: 5.2 without the mask's words,
// 5.8 without the walk.  The words are indexed by node, so they lie in local memory,
// and every step within the window loads and stores one there.
struct LayoutParams {
  const int32_t *parents, *n_nodes, *seq_len, *pos_base;
  int n, window;
  int32_t *depth, *positions;
  uint32_t *mask;
  int *err;
};

__global__ void __launch_bounds__(kMaxNodes) tree_layout_kernel(const __grid_constant__ LayoutParams p) {
  __shared__ int s_parent[kMaxNodes];
  const int b = blockIdx.x, i = threadIdx.x, n = p.n, words = (n + 31) / 32;
  pdl_wait();
  const int live = node_count(p.n_nodes, b, n, p.err);
  if (i < live) {
    const int up = p.parents[size_t(b) * n + i];
    const bool ok = up >= -1 && up < i;
    if (!ok) raise_device_error(p.err, ND_DEVERR_METADATA);
    s_parent[i] = ok ? up : -2;
  }
  __syncthreads();
  if (i >= n) return;
  const size_t at = size_t(b) * n + i;
  int depth = -1;
  uint32_t w[kMaxNodes / 32];
  for (int k = 0; k < words; ++k) w[k] = 0;
  if (i < live) {
    int j = i;
    for (; j >= 0; j = s_parent[j]) {
      if (++depth < p.window) w[j / 32] |= 1u << (j % 32);
    }
    if (j != -1) {
      depth = -1;
      for (int k = 0; k < words; ++k) w[k] = 0;
    }
  }
  p.depth[at] = depth;
  if (p.positions)
    p.positions[at] = depth < 0 ? -1 : (p.seq_len ? p.seq_len[b] : 0) + (p.pos_base ? *p.pos_base : 0) + depth;
  for (int k = 0; k < words; ++k) p.mask[at * words + k] = w[k];
}

// The same walk, ended at the first node that does not hold; the deepest that
// reaches its root wins by one atomic maximum.  512 trees of 256 nodes 3.4 us.
struct AcceptParams {
  const int32_t *parents, *n_nodes, *tokens, *target, *root_target;
  int n, max_path;
  int32_t *path, *path_len, *next;
  int *err;
};

__global__ void __launch_bounds__(kMaxNodes) tree_accept_kernel(const __grid_constant__ AcceptParams p) {
  __shared__ int s_up[kMaxNodes];    // the parent where the node agrees with it, -2 where it does not
  __shared__ int s_best;
  const int b = blockIdx.x, i = threadIdx.x, n = p.n;
  pdl_wait();
  const int live = node_count(p.n_nodes, b, n, p.err);
  const size_t row = size_t(b) * n;
  if (i == 0) s_best = 0;
  if (i < live) {
    const int up = p.parents[row + i];
    const bool ok = up >= -1 && up < i;
    if (!ok) raise_device_error(p.err, ND_DEVERR_METADATA);
    bool right = ok;
    if (ok && up >= 0) right = p.tokens[row + i] == p.target[row + up];
    if (ok && up < 0 && p.root_target) right = p.tokens[row + i] == p.root_target[b];
    s_up[i] = right ? up : -2;
  }
  __syncthreads();
  if (i < live) {
    int j = i, depth = -1;
    for (; j >= 0; j = s_up[j]) ++depth;
    // deepest first, then the lowest number
    if (j == -1 && depth < p.max_path) atomicMax(&s_best, (depth + 1) * kMaxNodes + (kMaxNodes - 1 - i));
  }
  __syncthreads();
  const int len = s_best / kMaxNodes, last = kMaxNodes - 1 - s_best % kMaxNodes;
  int32_t *path = p.path + size_t(b) * p.max_path;
  for (int k = len + i; k < p.max_path; k += blockDim.x) path[k] = -1;
  if (i == 0) {
    p.path_len[b] = len;
    if (p.next) p.next[b] = len ? p.target[row + last] : p.root_target ? p.root_target[b] : -1;
    for (int k = len - 1, j = last; k >= 0; --k, j = s_up[j]) path[k] = j;
  }
}

struct CommitParams {
  nd_kv_cache c;
  const uint16_t *k, *v;
  int64_t k_stride, v_stride;
  int n, max_path;
  const int32_t *path, *path_len;
  int *err;
  int parts;  // CTAs of a sequence
};

// The path's rows (token, head, K or V), D / 8 lanes to a row, kU rows of a lane's
// loads in flight: a chain of three latencies (metadata and path, rows, stores)
// with as many bytes behind each as there are.  A sequence with many rows and
// few neighbours is a cluster of CTAs; its metadata advance once all of them have
// read them.
// 512 sequences of up to 16 tokens of 8 heads of 128 (26 MB on average): 21 us,
// 64 of up to 6 of 2 heads of 64: 3.6.  80 registers a thread are three CTAs an SM,
// so 512 sequences are a second round for 56 of them, and the codec costs more
// instructions than so few warps' latencies hide: with its exact division tried per
// value instead of once for a lane's eight, 26 and 5.5 us; a row to a warp, 55 and 4.2.
template <int D>
__global__ void __launch_bounds__(256) tree_commit_kernel(const __grid_constant__ CommitParams p) {
  constexpr int kL = D / 8, kU = 4;
  const nd_kv_cache &c = p.c;
  const int parts = p.parts, b = blockIdx.x / parts, part = blockIdx.x % parts, cap = c.ring_cap;
  const int sub = threadIdx.x / kL, ch = threadIdx.x % kL, per = blockDim.x / kL;
  pdl_wait();
  const int rs = c.ring_start[b], rl = c.ring_len[b], sl = c.sink_len[b], sq = c.seq_len[b], len = p.path_len[b];
  const int32_t *path = p.path + int64_t(b) * p.max_path;
  bool ok = sl >= 0 && sl <= c.sink_cap && rl >= 0 && rl <= cap && rs >= 0 && rs < cap && len >= 0 && len <= p.max_path;
  if (ok)
    for (int t = threadIdx.x; t < len; t += blockDim.x) ok = ok && path[t] >= 0 && path[t] < p.n;
  ok = __syncthreads_and(ok);  // the same in all CTAs of the sequence
  if (parts > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  if (ok) {
    const int first = max(0, len - cap);  // tokens before it are overwritten within the path
    const int Hkv = c.n_kv_heads, per_token = 2 * Hkv, rows = (len - first) * per_token, step = per * parts;
    const unsigned slot0 = unsigned((int64_t(rs) + rl + first) % cap);
#pragma unroll 1
    for (int r0 = part * per; r0 < rows; r0 += kU * step) {
      uint4 w[kU];
      size_t at[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        // (K's rows of a token, then V's; past the end: the last row, not stored)
        const int r = min(r0 + u * step + sub, rows - 1), t = r / per_token, k = r - t * per_token, is_v = k >= Hkv, h = is_v ? k - Hkv : k;
        const int64_t node = int64_t(b) * p.n + path[first + t];
        const uint16_t *src = (is_v ? p.v + node * p.v_stride : p.k + node * p.k_stride) + h * D + ch * 8;
        w[u] = *reinterpret_cast<const uint4 *>(src);
        const unsigned ring = slot0 + t;  // t < cap
        const int slot = c.sink_cap + int(ring >= unsigned(cap) ? ring - cap : ring);
        at[u] = ((size_t(b) * Hkv + h) * (size_t(c.sink_cap) + cap) + slot) * 2 + is_v;
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (r0 + u * step >= rows) break;  // (the same for the CTA)
        const uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
        float y[8], amax = 0.f;
        bool finite = true;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          finite = finite && (x[i] & 0x7f80u) != 0x7f80u && (x[i] & 0x7f800000u) != 0x7f800000u;
          y[2 * i] = bf16_lo(x[i]), y[2 * i + 1] = bf16_hi(x[i]);
          amax = fmaxf(amax, fmaxf(fabsf(y[2 * i]), fabsf(y[2 * i + 1])));
        }
        // a group of 32 channels is four neighbouring lanes'
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const float scale = __fdiv_rn(amax, 127.0f), inv = __frcp_rn(scale);
        // the codec (nd_common.cuh): the nearest integer to x * inv is the code
        // unless one of the lane's eight lies near a half, the scale is tiny or a value
        // not finite.  1.5 * 2^23 added leaves the integer in the low bits.
        uint32_t m[8];
        float near = 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float q = y[i] * inv, big = q + 12582912.f;
          near = fminf(near, fabsf(fabsf(q - (big - 12582912.f)) - 0.5f));
          m[i] = __float_as_uint(big);
        }
        if (!(near > 1e-4f && scale >= 1e-30f && scale < INFINITY && finite)) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float q = 0.f;
            if (amax != 0.f) q = fminf(fmaxf(codec_rint(y[i], scale, inv), -127.f), 127.f);
            m[i] = uint32_t(int(q));
          }
        }
        uint32_t o[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          o[i] = prmt(prmt(m[4 * i], m[4 * i + 1], 0x0040u), prmt(m[4 * i + 2], m[4 * i + 3], 0x0040u), 0x5410u);
        if (r0 + u * step + sub < rows) {
          const size_t row = at[u] >> 1;
          const bool is_v = at[u] & 1;
          *reinterpret_cast<uint2 *>((is_v ? c.v_codes : c.k_codes) + row * D + ch * 8) = make_uint2(o[0], o[1]);
          if (ch % 4 == 0) ((is_v ? c.v_scale : c.k_scale) + row * (D / 32))[ch / 4] = scale;
        }
      }
    }
  }
  if (parts > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  if (part != 0 || threadIdx.x != 0) return;
  if (!ok) {
    raise_device_error(p.err, ND_DEVERR_METADATA);
    return;
  }
  const int64_t over = int64_t(rl) + len - cap;
  c.ring_len[b] = over > 0 ? cap : rl + len;
  if (over > 0) c.ring_start[b] = int((rs + over) % cap);
  c.seq_len[b] = sq + len;
}

template <int D>
cudaError_t launch_commit(CommitParams p, cudaStream_t stream) {
  // 16 rows (D = 128) to a CTA and pass, four passes in flight: more CTAs where a
  // path has more rows than that and the sequences leave room
  const int64_t rows = int64_t(p.max_path) * p.c.n_kv_heads * 2, at_once = 4 * (256 / (D / 8));
  p.parts = 1;
  while (p.parts < 8 && rows > at_once * p.parts && int64_t(p.c.batch) * p.parts < 304) p.parts *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.c.batch * p.parts);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.parts;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.parts > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, tree_commit_kernel<D>, p);
}

int threads_for(int n) { return n > 0 ? (n + 31) / 32 * 32 : 32; }

}  // namespace

cudaError_t launch_tree_layout(const int32_t *parents, const int32_t *n_nodes, const int32_t *seq_len,
                               const int32_t *pos_base, int batch, int n, int window, int32_t *depth,
                               int32_t *positions, uint32_t *mask, int *err, cudaStream_t stream) {
  const LayoutParams p = {parents, n_nodes, seq_len, pos_base, n, window, depth, positions, mask, err};
  return launch_pdl(tree_layout_kernel, dim3(batch), dim3(threads_for(n)), 0, stream, p);
}

cudaError_t launch_tree_accept(const int32_t *parents, const int32_t *n_nodes, const int32_t *tokens,
                               const int32_t *target, const int32_t *root_target, int batch, int n, int max_path,
                               int32_t *path, int32_t *path_len, int32_t *next, int *err, cudaStream_t stream) {
  const AcceptParams p = {parents, n_nodes, tokens, target, root_target, n, max_path, path, path_len, next, err};
  return launch_pdl(tree_accept_kernel, dim3(batch), dim3(threads_for(n)), 0, stream, p);
}

cudaError_t launch_tree_commit(const nd_kv_cache &c, const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                               int n, const int32_t *path, const int32_t *path_len, int max_path, int *err,
                               cudaStream_t stream) {
  const CommitParams p = {c, static_cast<const uint16_t *>(k), static_cast<const uint16_t *>(v), k_stride, v_stride, n,
                          max_path, path, path_len, err, 1};
  switch (c.head_dim) {
    case 32: return launch_commit<32>(p, stream);
    case 64: return launch_commit<64>(p, stream);
    case 128: return launch_commit<128>(p, stream);
    case 256: return launch_commit<256>(p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace nd
