// tree.cu -- trees of drafted tokens: their layout from the parents, the
// longest path that the model agrees with, and that path's append to the ring.
//
// All three are chains of latencies over a few kilobytes per sequence, so a
// sequence is one CTA (the commit: a few) and its nodes live in shared memory.
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
};

// One warp to a (token, head, K or V) row; lane l holds channels l * CPL ...
template <int D>
__global__ void __launch_bounds__(256) tree_commit_kernel(const __grid_constant__ CommitParams p) {
  constexpr int CPL = D / 32;
  const nd_kv_cache &c = p.c;
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cap = c.ring_cap;
  pdl_wait();
  const int rs = c.ring_start[b], rl = c.ring_len[b], sl = c.sink_len[b], len = p.path_len[b];
  const int32_t *path = p.path + size_t(b) * p.max_path;
  bool ok = sl >= 0 && sl <= c.sink_cap && rl >= 0 && rl <= cap && rs >= 0 && rs < cap && len >= 0 && len <= p.max_path;
  if (ok)
    for (int t = threadIdx.x; t < len; t += blockDim.x) ok = ok && path[t] >= 0 && path[t] < p.n;
  if (!__syncthreads_and(ok)) {  // (every thread has read the metadata)
    if (threadIdx.x == 0) raise_device_error(p.err, ND_DEVERR_METADATA);
    return;
  }
  const int first = max(0, len - cap);  // tokens before it are overwritten within the path
  const int rows = (len - first) * c.n_kv_heads * 2;
  for (int r = warp; r < rows; r += blockDim.x >> 5) {
    const int t = first + r / (2 * c.n_kv_heads), h = (r >> 1) % c.n_kv_heads, is_v = r & 1;
    const int slot = c.sink_cap + int((int64_t(rs) + rl + t) % cap);
    const int64_t node = int64_t(b) * p.n + path[t];
    const uint16_t *src = (is_v ? p.v + node * p.v_stride : p.k + node * p.k_stride) + h * D + lane * CPL;
    float x[CPL];
    int code[CPL];
#pragma unroll
    for (int i = 0; i < CPL; ++i) x[i] = __uint_as_float(uint32_t(src[i]) << 16);
    const float scale = quant_lanes<CPL>(x, code);
    const size_t at = (size_t(b) * c.n_kv_heads + h) * (c.sink_cap + cap) + slot;
    int8_t *dst = (is_v ? c.v_codes : c.k_codes) + at * D + lane * CPL;
#pragma unroll
    for (int i = 0; i < CPL; ++i) dst[i] = int8_t(code[i]);
    if (lane % (32 / CPL) == 0) ((is_v ? c.v_scale : c.k_scale) + at * (D / 32))[lane / (32 / CPL)] = scale;
  }
  if (threadIdx.x == 0) {
    const int64_t over = int64_t(rl) + len - cap;
    c.ring_len[b] = over > 0 ? cap : rl + len;
    if (over > 0) c.ring_start[b] = int((rs + over) % cap);
    c.seq_len[b] += len;
  }
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
                          max_path, path, path_len, err};
  const dim3 grid(c.batch), block(256);
  switch (c.head_dim) {
    case 32: return launch_pdl(tree_commit_kernel<32>, grid, block, 0, stream, p);
    case 64: return launch_pdl(tree_commit_kernel<64>, grid, block, 0, stream, p);
    case 128: return launch_pdl(tree_commit_kernel<128>, grid, block, 0, stream, p);
    case 256: return launch_pdl(tree_commit_kernel<256>, grid, block, 0, stream, p);
  }
  return cudaErrorInvalidValue;
}

}  // namespace nd
