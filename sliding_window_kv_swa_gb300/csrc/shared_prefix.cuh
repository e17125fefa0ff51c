// shared_prefix.cuh -- how the shared prefix's work is split, and where its
// partial results lie: used by the kernel that makes them (shared_prefix.cu)
// and by the ones that merge them (shared_decode.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "nd.h"

namespace nd {

constexpr int kPrefixTile = 64;    // keys per tile
constexpr int kPrefixBlock = 128;  // rows per block; a CTA holds two (a pair)
constexpr int kPrefixCtas = 152;   // one per SM
constexpr int kPrefixMinTiles = 2; // fewest tiles worth a CTA

// Up to 64 rows: a CTA takes every other key tile with either half of its
// softmax warps, and each half has partials of its own.
__host__ __device__ inline int prefix_streams(int rows) { return rows <= kPrefixBlock / 2 ? 2 : 1; }

// Partials: slot s holds a row pair's O [2][32][D/4][4 rows][4] and (max, sum)
// [2][128], maxima in log2 units; with two streams, theirs of the one block.
// (The prefix kernel has a row per thread and stores four channels of 32 rows
// at once, the merge reads all channels of the four heads of a group: in this
// order both touch whole sectors.  With O [D/4][128][4] the merge's loads went
// to 32 lines each.)
struct PrefixParts {
  float *o;
  float2 *ml;
};

__host__ __device__ inline int prefix_pairs(int rows) { return (rows + 2 * kPrefixBlock - 1) / (2 * kPrefixBlock); }

// Fewer than 2^30 tiles (checked by the entry point).
// The line of (item, tile): an item is a (KV head, row pair), its nt key tiles
// lie side by side.  CTA c has tiles [start(c), start(c + 1)); the segment of
// item i in CTA c has partial slot c + i, unique because a segment follows the
// one before it in the same CTA with the next item, or in the next CTA.
struct PrefixPlan {
  int len, nt, pairs, items, ctas;
  int per_item;  // CTAs of each item where they are the same number, else 0
  bool sane;
  int even, odd;  // tiles / ctas and tiles % ctas
  __host__ __device__ int tiles() const { return items * nt; }
  // = tiles * c / ctas, in 32 bits
  __host__ __device__ int start(int c) const { return even * c + odd * c / ctas; }
  // the CTAs of an item's first and last tile
  __host__ __device__ int first_cta(int item) const { return per_item ? item * per_item : owner(item * nt); }
  __host__ __device__ int last_cta(int item) const {
    return per_item ? (item + 1) * per_item - 1 : owner((item + 1) * nt - 1);
  }
  // the CTA whose stretch holds tile x
  __host__ __device__ int owner(int x) const {
    const long long y = (long long)(x + 1) * ctas - 1;
    return y < (1ll << 31) ? int(y) / tiles() : int(y / tiles());  // (a 32-bit division where it suffices)
  }
};

__host__ __device__ inline PrefixPlan prefix_plan(int sink_len, int sink_cap, int n_kv_heads, int rows, int grid) {
  PrefixPlan p;
  p.sane = sink_len >= 0 && sink_len <= sink_cap;
  p.len = p.sane ? sink_len : 0;
  p.nt = (p.len + kPrefixTile - 1) / kPrefixTile;
  p.pairs = prefix_pairs(rows);
  p.items = n_kv_heads * p.pairs;
  const int want = (p.tiles() + kPrefixMinTiles - 1) / kPrefixMinTiles;
  p.ctas = want < grid ? want : grid;
  // A multiple of the items cuts each item into equal parts, one segment per
  // CTA; worth up to a sixth of the CTAs (64 items: 128 CTAs of one segment
  // each, 22 us, against 152 of two and more, 26 us).
  const int equal = p.items > 0 ? p.ctas / p.items * p.items : 0;
  if (equal * 6 >= p.ctas * 5) p.ctas = equal;
  p.per_item = equal > 0 && p.ctas == equal ? equal / p.items : 0;
  p.even = p.ctas > 0 ? p.tiles() / p.ctas : 0;
  p.odd = p.tiles() - p.even * p.ctas;
  return p;
}

// Blocks to launch (up to `most`) for a prefix of up to sink_cap slots, and
// partial slots.
inline int prefix_grid(int sink_cap, int n_kv_heads, int rows, int most) {
  const int c = prefix_plan(sink_cap, sink_cap, n_kv_heads, rows, most).ctas;
  return c > 0 ? c : 1;
}
inline size_t prefix_slots(int sink_cap, int n_kv_heads, int rows, int most) {
  return size_t(prefix_grid(sink_cap, n_kv_heads, rows, most)) + size_t(n_kv_heads) * prefix_pairs(rows);
}

cudaError_t launch_shared_prefix(const void *q, const nd_kv_cache &prefix, int batch, int n_q_heads, int grid,
                                 const PrefixParts &out, int *err, cudaStream_t stream);

}  // namespace nd
