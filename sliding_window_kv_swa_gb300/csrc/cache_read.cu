// cache_read.cu -- reads a bounded int8 cache back into keys and values, in
// the layout a prefill has them ([batch][rows][heads][channels]) and in
// position order: the sinks, then the ring entries that the window reaches,
// oldest first.  The inverse of the handoff from a prefill.
//
// value = code * scale, one fp32 product, rounded once to the output type.
// HBM-bound: per (row, KV head) 2 (D + D/8) bytes in, 2 D elements out, most
// of it the output's writes: a lane moves 8 channels, so that a warp's store
// of bf16 covers whole lines (with 16 channels to a lane, two stores of half a
// sector each: 18.9 us against 15.7 for 36 rows of 384 slots, 8 heads, D =
// 128; the bytes take 13 us).  fp32 still has such halves, a lane's 8 channels
// being 32 bytes in two stores: 30.6 us for the same rows, the bytes 21.4.
#include "nd_common.cuh"
#include "nd_internal.h"

namespace nd {

namespace {

struct ReadParams {
  nd_kv_cache c;
  int window, n_rows;
  void *k, *v;           // [B][n_rows][Hkv][D]
  int32_t *pos, *len;    // [B][n_rows], [B]; may be NULL
  int *err;
};

__device__ __forceinline__ void store8(uint16_t *dst, const uint2 &w, float s) {
  const uint32_t u[2] = {w.x, w.y};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    o[2 * i] = pack_bf16x2(float(int8_t(u[i])) * s, float(int8_t(u[i] >> 8)) * s);
    o[2 * i + 1] = pack_bf16x2(float(int8_t(u[i] >> 16)) * s, float(int8_t(u[i] >> 24)) * s);
  }
  *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ void store8(float *dst, const uint2 &w, float s) {
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 2; ++i)
    reinterpret_cast<float4 *>(dst)[i] = make_float4(float(int8_t(u[i])) * s, float(int8_t(u[i] >> 8)) * s,
                                                     float(int8_t(u[i] >> 16)) * s, float(int8_t(u[i] >> 24)) * s);
}

constexpr int kTile = 8;  // output rows per CTA (16: 16.4 us; 32: 18.5)

// grid (row tiles, B).  A warp takes a (head, K or V) and its kTile rows: the
// slots of neighbouring rows are neighbours (but for the ring's wrap), so its
// loads cover 8 D bytes of codes in one piece, all of them in flight before the
// first is converted.
template <typename E, int D>
__global__ void __launch_bounds__(256) cache_read_kernel(const ReadParams p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kU = kTile / kRows;  // rows per load of the warp, loads
  const nd_kv_cache &c = p.c;
  const int b = blockIdx.y, row0 = blockIdx.x * kTile;
  const int Hkv = c.n_kv_heads, nslot = c.sink_cap + c.ring_cap;
  pdl_wait();
  const int sl = c.sink_len[b], rs = c.ring_start[b], rl = c.ring_len[b], sq = c.seq_len[b];
  const bool sane = sl >= 0 && sl <= c.sink_cap && rl >= 0 && rl <= c.ring_cap && rs >= 0 &&
                    rs < (c.ring_cap > 0 ? c.ring_cap : 1);
  const int n = sane ? min(rl, p.window) : 0, live = sane ? sl + n : 0;
  if (row0 == 0 && threadIdx.x == 0) {
    if (!sane) raise_device_error(p.err, ND_DEVERR_METADATA);
    if (p.len) p.len[b] = live;
  }
  if (p.pos && threadIdx.x < kTile && row0 + threadIdx.x < p.n_rows) {
    const int r = row0 + threadIdx.x;
    p.pos[size_t(b) * p.n_rows + r] = r >= live ? -1 : (r < sl ? r : sq - n + (r - sl));
  }
  if (row0 >= live) return;
  int oldest = rs + rl - n;  // ring slot of the oldest visible entry
  if (oldest >= c.ring_cap) oldest -= c.ring_cap;
  const int lane = threadIdx.x & 31, sub = lane / kLanes, ch = (lane % kLanes) * 8;
  const int r0 = row0 + sub;
  for (int pair = threadIdx.x >> 5; pair < 2 * Hkv; pair += blockDim.x >> 5) {
    const int h = pair >> 1;
    const size_t base = (size_t(b) * Hkv + h) * nslot;
    const int8_t *codes = ((pair & 1) ? c.v_codes : c.k_codes) + base * D + ch;
    const float *scale = ((pair & 1) ? c.v_scale : c.k_scale) + base * (D / 32) + ch / 32;
    uint2 w[kU];
    float s[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int r = r0 + u * kRows;
      if (r >= live) continue;
      int ring = oldest + r - sl;
      if (ring >= c.ring_cap) ring -= c.ring_cap;
      const int slot = r < sl ? r : c.sink_cap + ring;
      w[u] = *reinterpret_cast<const uint2 *>(codes + size_t(slot) * D);
      s[u] = scale[size_t(slot) * (D / 32)];
    }
    E *out = static_cast<E *>((pair & 1) ? p.v : p.k) + ((size_t(b) * p.n_rows + r0) * Hkv + h) * D + ch;
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (r0 + u * kRows < live) store8(out + size_t(u * kRows) * Hkv * D, w[u], s[u]);
  }
}

template <typename E>
cudaError_t launch_read_t(const ReadParams &p, dim3 grid, cudaStream_t stream) {
  switch (p.c.head_dim) {
    case 32: return launch_pdl(cache_read_kernel<E, 32>, grid, dim3(256), 0, stream, p);
    case 64: return launch_pdl(cache_read_kernel<E, 64>, grid, dim3(256), 0, stream, p);
    case 128: return launch_pdl(cache_read_kernel<E, 128>, grid, dim3(256), 0, stream, p);
    case 256: return launch_pdl(cache_read_kernel<E, 256>, grid, dim3(256), 0, stream, p);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_cache_read(const nd_kv_cache &c, int window, bool f32, int n_rows, void *k, void *v,
                              int32_t *positions, int32_t *lengths, int *err, cudaStream_t stream) {
  ReadParams p;
  p.c = c;
  p.window = window;
  p.n_rows = n_rows;
  p.k = k;
  p.v = v;
  p.pos = positions;
  p.len = lengths;
  p.err = err;
  const dim3 grid(unsigned((n_rows - 1) / kTile + 1), unsigned(c.batch));  // (n_rows may be the largest int)
  return f32 ? launch_read_t<float>(p, grid, stream) : launch_read_t<uint16_t>(p, grid, stream);
}

}  // namespace nd
