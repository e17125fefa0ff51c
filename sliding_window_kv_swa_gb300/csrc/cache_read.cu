// cache_read.cu -- reads a bounded int8 cache back into keys and values, in
// the layout a prefill has them ([batch][rows][heads][channels]) and in
// position order: the sinks, then the ring entries that the window reaches,
// oldest first.  The inverse of the handoff from a prefill.
//
// value = code * scale, one fp32 product, rounded once to the output type.
// HBM-bound: per (row, KV head) 2 (D + D/8) bytes in, 2 D elements out.
// A lane moves 16 channels (one 16-byte load of codes); kU rows' loads go out
// before any is converted.
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

__device__ __forceinline__ void store16(uint16_t *dst, const uint4 &w, float s) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = pack_bf16x2(float(int8_t(u[i])) * s, float(int8_t(u[i] >> 8)) * s);
    o[2 * i + 1] = pack_bf16x2(float(int8_t(u[i] >> 16)) * s, float(int8_t(u[i] >> 24)) * s);
  }
  reinterpret_cast<uint4 *>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
  reinterpret_cast<uint4 *>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
}
__device__ __forceinline__ void store16(float *dst, const uint4 &w, float s) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4 *>(dst)[i] = make_float4(float(int8_t(u[i])) * s, float(int8_t(u[i] >> 8)) * s,
                                                     float(int8_t(u[i] >> 16)) * s, float(int8_t(u[i] >> 24)) * s);
}

constexpr int kRowsPerCta = 8;

// grid (row blocks, B): (row, head, K or V) triples of kRowsPerCta output rows.
template <typename E, int D>
__global__ void __launch_bounds__(256) cache_read_kernel(const ReadParams p) {
  constexpr int kLanes = D / 16, kU = 4;
  const nd_kv_cache &c = p.c;
  const int b = blockIdx.y, row0 = blockIdx.x * kRowsPerCta;
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
  if (p.pos && threadIdx.x < kRowsPerCta && row0 + threadIdx.x < p.n_rows) {
    const int r = row0 + threadIdx.x;
    p.pos[size_t(b) * p.n_rows + r] = r >= live ? -1 : (r < sl ? r : sq - n + (r - sl));
  }
  const int sub = threadIdx.x / kLanes, ch = (threadIdx.x % kLanes) * 16, per = blockDim.x / kLanes;
  const int rows = min(kRowsPerCta, live - row0), n_items = rows * Hkv * 2;  // none for a block behind the sequence
  for (int t0 = sub; t0 < n_items; t0 += per * kU) {
    uint4 w[kU];
    float s[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int t = t0 + u * per;
      if (t >= n_items) continue;
      const int r = row0 + t / (2 * Hkv), h = (t >> 1) % Hkv;
      const int slot = r < sl ? r : c.sink_cap + (rs + rl - n + (r - sl)) % c.ring_cap;
      const size_t row = (size_t(b) * Hkv + h) * nslot + slot;
      w[u] = *reinterpret_cast<const uint4 *>(((t & 1) ? c.v_codes : c.k_codes) + row * D + ch);
      s[u] = ((t & 1) ? c.v_scale : c.k_scale)[row * (D / 32) + ch / 32];
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int t = t0 + u * per;
      if (t >= n_items) continue;
      const int r = row0 + t / (2 * Hkv), h = (t >> 1) % Hkv;
      E *out = static_cast<E *>((t & 1) ? p.v : p.k);
      store16(out + ((size_t(b) * p.n_rows + r) * Hkv + h) * D + ch, w[u], s[u]);
    }
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
  const dim3 grid(unsigned((n_rows + kRowsPerCta - 1) / kRowsPerCta), unsigned(c.batch));
  return f32 ? launch_read_t<float>(p, grid, stream) : launch_read_t<uint16_t>(p, grid, stream);
}

}  // namespace nd
