// tree_decode.cu -- attention of a tree of drafted tokens: every node against
// its sequence's int8 cache and the nodes its mask names, in one softmax, on
// the 5th-generation tensor cores.
//
// Mathematics.  A (sequence, KV head)'s rows are the R = n * G queries that read
// it (row r: node r / G, head r % G of the group).  Over any part of its keys a
// row's softmax is the triple
//   m = max_j s_j,  l = sum_j 2^(s_j - m),  O = sum_j 2^(s_j - m) v_j,
//   s_j = (q . k_j) log2(e) / sqrt(D),
// and triples of different parts merge exactly.  The keys are taken in tiles of
// up to 128: filled sinks; ring entries in their order, the newest window - 1
// of them, of which a row at depth t sees those from entry nv + t - window + 1
// on; and nodes by 64, of which a row sees what its mask's bits say.
//
// Types.  Cached keys and values become fp16 after power-of-two scalings, as in
// shared_prefix.cu: code * fp16(scale * 2^e), e per tile for K and following
// the largest scale seen for V (at most 64, see kMostUp); q (bf16) becomes fp16
// exactly after one per row (channels 2^-28 below the row's largest lose bits).
// A node's key gets a power of two of its own and is then exact in the same
// way; its values stay bf16, and their weights are bf16 (2^-9 of themselves)
// with the power of two that O holds V in, which bf16's range has room for.
// Cached keys' weights are fp16 with the running maximum up to 2^8 behind and
// all of it scaled by 2^7.  Sums, maxima and partials are fp32.
//
// Masked places.  A weight of 0 times a NaN or an infinity would be NaN, so
// slots and nodes that nothing may see are 0 in the operands; a node whose key
// or value is not finite is 0 too and makes NaN of the scores of the rows that
// see it.  A row that sees nothing (or whose query is not finite) keeps m =
// -inf and l = 0 and comes out 0.
//
// Lanes.  The products have 128 rows whatever R is.  With R <= 64 (32) the rows
// stand two (four) times in Q, and each copy takes its own half (quarter) of a
// tile's columns, with a maximum, sum and O of its own, so that all four
// softmax warps work; the copies merge at the end like any triples.
//
// Work split.  The ((sequence, KV head), tile) pairs, tiles fastest, form one
// line that is cut into equal stretches, one per CTA and row block (one CTA per
// SM); row blocks of one stretch run side by side and share their codes in L2.
// A stretch is one or more segments (tiles of one (sequence, KV head)); one
// that has all of its tiles writes the output, others write their triple for
// tree_merge_kernel.  The line counts the tiles that the caches have room for;
// those that hold nothing are skipped.
//
// Roles (16 warps):
//   warps 0-3   : softmax (thread = TMEM lane): stage Q; per tile read S, write
//                 P over it; at a segment's end read O and write it
//   warps 4-11  : codes (or nodes' bf16) of the staged tile -> K, V operands in
//                 shared memory, half of them K, half V
//   warp 12     : copies the tiles ahead
//   warp 15     : the staged tile's scales -> exponents, fp16 scales
//   warps 13, 14: MMA issuers: S = Q K^T; O += P V
// Every wait is bounded: one that gives up raises the device error flag and the
// abort flag, and all roles leave through the common exit.
#include <atomic>
#include <climits>

#include "nd_common.cuh"
#include "nd_internal.h"
#include "tc_ptx.cuh"

namespace nd {

namespace {

constexpr int BM = 128;        // rows of a product = TMEM lanes
constexpr int BN = 128;        // cached keys per tile
constexpr int kNodes = 64;     // nodes per tile
constexpr int kThreads = 16 * 32;
constexpr int kWarpTurn = 4, kWarpLoad = 12, kWarpS = 13, kWarpPV = 14, kWarpScan = 15;
// Register split (setmaxnreg, per warpgroup) of the 128 a thread at launch: a
// softmax thread holds up to 128 scores.
constexpr int kRegsSoftmax = 232, kRegsOther = 88;
static_assert(128 * kRegsSoftmax + 3 * 128 * kRegsOther <= kThreads * 128, "register split");
constexpr float kLazyLog2 = 8.f;  // the maximum used may lag the true one by 2^8
constexpr float kPBias = 7.f;     // P is scaled by 2^7
constexpr int kInfo = 16;         // tile records in flight: more than the tiles between copy and softmax
constexpr int kMostUp = 64;       // V's largest exponent: a node's value times 2^(64 + 15) stays finite up to 2^48
constexpr int kCtas = 152;        // one per SM

// ------------------------------------------------------------ the split
struct TreePlan {
  int ts, tr, tn, t;   // tiles of the sinks, the ring and the nodes, and all
  int pairs;           // (sequence, KV head)
  int nb, rb;          // row blocks, rows of each
  int ctas;            // stretches
  int even, odd;       // units / ctas and units % ctas
  bool whole;          // a unit is a pair (nothing is split), else a tile
  __host__ __device__ int start(int c) const {
    const int u = even * c + int((long long)odd * c / ctas);
    return whole ? u * t : u;
  }
  // the stretch that holds tile x of the line
  __host__ __device__ int owner(int x) const {
    return int(((long long)(x + 1) * ctas - 1) / ((long long)pairs * t));
  }
  int rows_of_lanes() const { return rb <= 32 ? 32 : rb <= 64 ? 64 : 128; }
};

TreePlan tree_plan(int batch, int n, int n_q_heads, int n_kv_heads, int sink_cap, int ring_cap) {
  TreePlan p;
  const int R = n * (n_q_heads / n_kv_heads);
  p.nb = (R + BM - 1) / BM;
  p.rb = (R + p.nb - 1) / p.nb;
  p.ts = (sink_cap + BN - 1) / BN;
  p.tr = (ring_cap + BN - 1) / BN;
  p.tn = (n + kNodes - 1) / kNodes;
  p.t = p.ts + p.tr + p.tn;
  p.pairs = batch * n_kv_heads;
  const long long tiles = (long long)p.pairs * p.t;
  const int most = kCtas / p.nb;
  // whole pairs where that leaves at most a sixteenth of the CTAs' time idle
  p.whole = (long long)((p.pairs + most - 1) / most) * most * 16 <= (long long)p.pairs * 17;
  const long long units = p.whole ? p.pairs : tiles;
  p.ctas = int(units < most ? units : most);
  p.even = int(units / p.ctas);
  p.odd = int(units - (long long)p.even * p.ctas);
  return p;
}

// Partials of a stretch: which = 0 for its first segment, 1 for a later one.
// O [D/4][128 lanes][4], (max, sum) [128]; maxima in log2 units.
template <int D>
__host__ __device__ constexpr size_t part_floats() {
  return size_t(BM) * (D + 2);
}

// ------------------------------------------------------------ the kernel
template <int D>
struct Lay {
  static constexpr int NG = D / 32, kBoxes = D / 64;
  static constexpr int kKV = kBoxes * BN * 128;          // one K or V operand tile
  static constexpr int kCodes = BN * D, kScales = BN * NG * 4;
  static constexpr int kRaw = 2 * kCodes + 2 * kScales;  // K codes, V codes, K scales, V scales; or nodes' K, V
  static_assert(kNodes * D * 2 == kCodes, "a node tile's rows take the codes' place");
  static constexpr int NK = D == 128 ? 2 : 3, NV = NK, NR = D == 128 ? 2 : 5;
  static constexpr int kRow = 144, kT = 4 * 32 * kRow;   // a softmax warp's 32 rows of 64 channels, padded
  static constexpr int oK = 0, oV = oK + NK * kKV, oR = oV + NV * kKV, oT = oR + NR * kRaw;
  static constexpr int kBytes = oT + kT + 1024;          // + alignment slack
  static_assert(kBytes + 6 * 1024 <= 227 * 1024, "shared memory");
  // TMEM columns: S[2], O, Q
  static constexpr int cO = 2 * BN, cQ = cO + D, kTmemCols = 512;
  static_assert(cQ + D / 2 <= kTmemCols, "TMEM");
};

struct TreeParams {
  const uint16_t *q, *k, *v;
  int64_t k_stride, v_stride;
  nd_kv_cache c;
  const int32_t *depth;
  const uint32_t *mask;
  int n, Hq, G, window;
  unsigned g_magic;  // ceil(2^32 / G): r / G for G >= 2 and r < 2^24
  uint16_t *out;
  float *lse;
  float *parts;
  TreePlan plan;
  int *err;
};

__device__ __forceinline__ int ilog2(float x) { return int((__float_as_uint(x) >> 23) & 0xffu) - 127; }
__device__ __forceinline__ float pow2i(int e) {  // e in [-126, 127]
  return __uint_as_float(uint32_t(e + 127) << 23);
}
__device__ __forceinline__ int clamp_exp(int e) { return max(-120, min(120, e)); }

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ float lds_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int N>
struct Ring {
  int i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++i == N) {
      i = 0;
      phase ^= 1u;
    }
  }
};

// A bounded wait of a whole warp that sleeps between polls (up to 2 us each).
__device__ __forceinline__ bool ring_wait(uint64_t *bar, uint32_t parity, int *err, volatile int *abort_flag) {
  bool ok = mbar_test_wait(bar, parity);
  for (uint32_t i = 0; i < kWaitLimit / 64 && !ok; ++i) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(r)
        : "r"(smem_u32(bar)), "r"(parity), "n"(2000)
        : "memory");
    ok = r != 0;
    if (!ok && *abort_flag) break;
  }
  if (!ok && !*abort_flag) {
    raise_device_error(err, ND_DEVERR_TIMEOUT);
    *abort_flag = 1;
  }
  return __all_sync(0xffffffffu, ok);
}

// Whether any thread of the four softmax warps says so; a barrier of theirs.
__device__ __forceinline__ bool softmax_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(uint32_t(x))
      : "memory");
  return r != 0;
}

// A segment: tiles [t0, t1) of one pair, and what its metadata say.
struct Seg {
  int pair, b, t0, t1;
  int sl, nv, ring0;  // filled sinks; ring entries that a node at depth 0 sees; ring slot of the oldest of them
  int ts, tr;         // tiles that they fill
  bool sane, all;     // all: the pair has no other segment
};

__device__ __forceinline__ Seg seg_at(const TreeParams &p, int x, int x1) {
  const TreePlan &pl = p.plan;
  const nd_kv_cache &c = p.c;
  Seg s;
  s.pair = x / pl.t;
  s.t0 = x - s.pair * pl.t;
  s.t1 = min(pl.t, s.t0 + x1 - x);
  s.all = s.t0 == 0 && s.t1 == pl.t;
  s.b = s.pair / c.n_kv_heads;
  const int sl = c.sink_len[s.b], rs = c.ring_start[s.b], rl = c.ring_len[s.b];
  s.sane = sl >= 0 && sl <= c.sink_cap && rl >= 0 && rl <= c.ring_cap && rs >= 0 && (c.ring_cap == 0 || rs < c.ring_cap);
  s.sl = s.sane ? sl : 0;
  s.nv = s.sane ? min(rl, p.window - 1) : 0;
  const unsigned first = unsigned(rs) + unsigned(rl - s.nv);  // below 2^32
  s.ring0 = s.nv > 0 ? int(first >= unsigned(c.ring_cap) ? first - unsigned(c.ring_cap) : first) : 0;
  s.ts = (s.sl + BN - 1) / BN;
  s.tr = (s.nv + BN - 1) / BN;
  return s;
}
// the first tile from t on that holds something
__device__ __forceinline__ int live_tile(const TreePlan &pl, const Seg &s, int t) {
  if (t >= s.ts && t < pl.ts) t = pl.ts;
  if (t >= pl.ts + s.tr && t < pl.ts + pl.tr) t = pl.ts + pl.tr;
  return t;
}

template <int D, int REP>
__global__ void __launch_bounds__(kThreads, 1) tree_decode_kernel(const __grid_constant__ TreeParams p) {
  using Y = Lay<D>;
  constexpr int NK = Y::NK, NV = Y::NV, NR = Y::NR, NG = Y::NG;
  constexpr int kLanes = BM / REP;  // rows, and lanes of a copy of them
  constexpr int kCols = BN / REP;   // a thread's columns of a tile
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t raw_full[NR], raw_empty[NR], scan_full[NR], k_full[NK], k_empty[NK], v_full[NV], v_empty[NV],
      s_full[2], p_full[2], pv_done[2], q_full;
  __shared__ float4 s_info[kInfo];           // per tile, for the softmax
  __shared__ uint2 s_live[kInfo];            // node tiles: nodes that are not padding
  __shared__ uint32_t s_bad[kInfo][2];       // and those that are not finite
  __shared__ float s_kf[kInfo][kNodes];      // and 2^-e of their keys
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ float2 s_ml[BM];

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the same in the warp
  volatile int *abort_flag = &s_abort;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sK = base + Y::oK, sV = base + Y::oV, sT = base + Y::oT;
  auto sR = [&](int st) { return base + Y::oR + st * Y::kRaw; };

  if (tid == 0) {
    for (int s = 0; s < NR; ++s) {
      mbar_init(&raw_full[s], 33);  // the bulk copies' transaction and 32 lanes' scale copies
      mbar_init(&raw_empty[s], 9);  // the warps that turn the tile, and the scan
      mbar_init(&scan_full[s], 1);
    }
    for (int s = 0; s < NK; ++s) {
      mbar_init(&k_full[s], 4);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 4);
      mbar_init(&v_empty[s], 1);
    }
    for (int u = 0; u < 2; ++u) {
      mbar_init(&s_full[u], 1);
      mbar_init(&p_full[u], 4);
      mbar_init(&pv_done[u], 1);
    }
    mbar_init(&q_full, 4);
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == kWarpS) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                 "r"(Y::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  pdl_wait();
  pdl_trigger();  // the merge reads nothing of this kernel's before it waits
  const uint32_t tO = tmem + Y::cO, tQ = tmem + Y::cQ;

  const TreePlan &pl = p.plan;
  const int stretch = blockIdx.x / pl.nb, blk = blockIdx.x % pl.nb;
  const int x0 = pl.start(stretch), x1 = pl.start(stretch + 1);
  bool fail = false;

  // (each side of the split has its setmaxnreg to itself: behind a common one the
  // compiler takes the smaller bound for all roles)
  if (warp >= 4) {
  regs_dec<kRegsOther>();
  if (warp == kWarpLoad) {
    // -------------------------------------------------- loader
    const uint32_t leader = elect_one();
    const int nslot = p.c.sink_cap + p.c.ring_cap;
    Ring<NR> raw;
    raw.phase = 1;  // the first round of an empty ring does not wait
    for (int x = x0; x < x1 && !fail;) {
      const Seg s = seg_at(p, x, x1);
      x += s.t1 - s.t0;
      if (!s.sane && lane == 0) raise_device_error(p.err, ND_DEVERR_METADATA);
      const size_t slot0 = size_t(s.pair) * nslot;
      const int hk = s.pair - s.b * p.c.n_kv_heads;
#pragma unroll 1
      for (int t = live_tile(pl, s, s.t0); t < s.t1; t = live_tile(pl, s, t + 1), raw.next()) {
        if (!ring_wait(&raw_empty[raw.i], raw.phase, p.err, abort_flag)) {
          fail = true;
          break;
        }
        uint64_t *bar = &raw_full[raw.i];
        const uint32_t dst = sR(raw.i);
        if (t < pl.ts + pl.tr) {
          // up to two pieces: a ring tile may wrap
          const bool ring = t >= pl.ts;
          const int first = (ring ? t - pl.ts : t) * BN;
          const int cnt = min(BN, (ring ? s.nv : s.sl) - first);
          int at = first, c1 = cnt;
          if (ring) {
            unsigned w = unsigned(s.ring0) + unsigned(first);
            if (w >= unsigned(p.c.ring_cap)) w -= unsigned(p.c.ring_cap);
            c1 = min(cnt, p.c.ring_cap - int(w));
            at = p.c.sink_cap + int(w);
          }
          expect_tx(bar, 2 * cnt * D, leader);
          if (leader) {
            const size_t a = (slot0 + at) * D;
            bulk_copy(dst, p.c.k_codes + a, c1 * D, bar);
            bulk_copy(dst + Y::kCodes, p.c.v_codes + a, c1 * D, bar);
            if (c1 < cnt) {
              const size_t w = (slot0 + p.c.sink_cap) * D;
              bulk_copy(dst + c1 * D, p.c.k_codes + w, (cnt - c1) * D, bar);
              bulk_copy(dst + Y::kCodes + c1 * D, p.c.v_codes + w, (cnt - c1) * D, bar);
            }
          }
          __syncwarp();
          // scales: a slot's row is 16 (D = 128) or 8 bytes, and a head's first
          // one aligned to no more than that
#pragma unroll
          for (int i = 0; i < BN / 32; ++i) {
            const int r = lane + 32 * i;
            if (r < cnt) {
              const size_t w = (slot0 + (r < c1 ? at + r : p.c.sink_cap + r - c1)) * NG;
              const uint32_t sd = dst + 2 * Y::kCodes + r * (NG * 4);
              if constexpr (NG == 4) {
                cp_async16(sd, p.c.k_scale + w);
                cp_async16(sd + Y::kScales, p.c.v_scale + w);
              } else {
                cp_async8(sd, p.c.k_scale + w);
                cp_async8(sd + Y::kScales, p.c.v_scale + w);
              }
            }
          }
        } else {
          const int j0 = (t - pl.ts - pl.tr) * kNodes, cnt = min(kNodes, p.n - j0);
          expect_tx(bar, 2 * cnt * (2 * D), leader);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < kNodes / 32; ++i) {
            const int r = lane + 32 * i;
            if (r < cnt) {
              const int64_t node = int64_t(s.b) * p.n + j0 + r;
              bulk_copy(dst + r * (2 * D), p.k + node * p.k_stride + hk * D, 2 * D, bar);
              bulk_copy(dst + Y::kCodes + r * (2 * D), p.v + node * p.v_stride + hk * D, 2 * D, bar);
            }
          }
        }
        cp_async_arrive(bar);
        __syncwarp();
      }
    }
  } else if (warp >= kWarpTurn && warp < kWarpLoad) {
    // -------------------------------------------------- operands
    const int turn = warp - kWarpTurn;
    const bool is_v = turn & 1;
    constexpr int kTurnRows = BN / 4;
    const int row_w = (turn >> 1) * kTurnRows;  // the warp's first row
    constexpr int kPieces = D / 16, kRowsIt = 32 / kPieces, kIts = kTurnRows / kRowsIt, kU = 2;
    static_assert(kIts % kU == 0, "rows of a warp");
    const int piece = lane % kPieces, row_l = lane / kPieces;
    // K-major (and for V MN-major) 128-byte swizzle: row * 128 + 16-byte chunk ^
    // (row & 7) inside a box of 64 channels; a lane's two chunks.  The upper
    // box's lanes store their odd chunk first, so the eight lanes of a row cover
    // the eight chunk positions (all banks) at once.
    const int box = piece / 4, c0 = (2 * piece) & 7;
    const uint32_t odd_first = box == 1 ? 1u : 0u;
    uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
    const uint32_t codes_off = (is_v ? Y::kCodes : 0) + (row_w + row_l) * D + piece * 16 + 8 * odd_first;
    const uint32_t scale_off = 2 * Y::kCodes + (is_v ? Y::kScales : 0) + 4 * ((row_w + row_l) * NG + piece / 2);
    const uint32_t operand = is_v ? sV : sK;
    const uint32_t row_off = operand + (row_w + row_l) * 128 + box * (BN * 128);
    const uint32_t first_c = ((c0 + odd_first) ^ (row_l & 7)) << 4;  // and the other chunk: ^ 16
    Ring<NR> raw;
    Ring<NK> op;
    op.phase = 1;
    int g = 0;
    for (int x = x0; x < x1 && !fail;) {
      const Seg s = seg_at(p, x, x1);
      x += s.t1 - s.t0;
#pragma unroll 1
      for (int t = live_tile(pl, s, s.t0); t < s.t1; t = live_tile(pl, s, t + 1), ++g, raw.next(), op.next()) {
        // the scan waited for the tile's copies before it arrived
        if (!ring_wait(&scan_full[raw.i], raw.phase, p.err, abort_flag) ||
            !ring_wait(&empty[op.i], op.phase, p.err, abort_flag)) {
          fail = true;
          break;
        }
        if (t < pl.ts + pl.tr) {
          const uint32_t raw_at = sR(raw.i) + codes_off, sc_at = sR(raw.i) + scale_off;
          const uint32_t dst = row_off + op.i * Y::kKV;
#pragma unroll 1
          for (int i0 = 0; i0 < kIts; i0 += kU) {
            uint2 w[kU][2];
            uint32_t s2[kU];
#pragma unroll
            for (int i = 0; i < kU; ++i) {
              w[i][0] = lds64(raw_at + (i0 + i) * kRowsIt * D);
              w[i][1] = lds64((raw_at ^ 8u) + (i0 + i) * kRowsIt * D);
              s2[i] = lds32(sc_at + (i0 + i) * kRowsIt * NG * 4);
            }
#pragma unroll
            for (int i = 0; i < kU; ++i) {
              // a lane's rows are kRowsIt (4 or 8) apart: the swizzle of the
              // second of a pair differs from the first's in one bit at most
              const uint32_t at = dst + (i0 + i) * kRowsIt * 128 + (first_c ^ ((i * kRowsIt & 4) << 4));
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const uint32_t wa = w[i][q].x ^ 0x80808080u, wb = w[i][q].y ^ 0x80808080u;
                st_shared_v4(q ? at ^ 16u : at, hmul2(codes_to_half2(wa, kSelBytes01), s2[i]),
                             hmul2(codes_to_half2(wa, kSelBytes23), s2[i]), hmul2(codes_to_half2(wb, kSelBytes01), s2[i]),
                             hmul2(codes_to_half2(wb, kSelBytes23), s2[i]));
              }
            }
          }
        } else {
          // nodes: D/8 lanes to a row, a sixteenth of the tile's rows per warp
          // and iteration
          constexpr int kL = D / 8, kR = 32 / kL;
          const int sub = lane / kL, ch = lane % kL;
          const int cnt = min(kNodes, p.n - (t - pl.ts - pl.tr) * kNodes);
          const uint2 alive = s_live[g % kInfo];
          const uint32_t src = sR(raw.i) + (is_v ? Y::kCodes : 0), dst = operand + op.i * Y::kKV;
#pragma unroll 1
          for (int r0 = (turn >> 1) * (kNodes / 4); r0 < (turn >> 1) * (kNodes / 4) + kNodes / 4; r0 += kR) {
            const int r = r0 + sub;
            const bool use = r < cnt && ((r < 32 ? alive.x : alive.y) >> (r & 31) & 1u);
            uint32_t w[4] = {0u, 0u, 0u, 0u};
            if (use) ld_shared_v4(src + r * (2 * D) + ch * 16, w[0], w[1], w[2], w[3]);
            float mx = 0.f;
            bool bad = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a = fabsf(bf16_lo(w[e])), b = fabsf(bf16_hi(w[e]));
              bad = bad || !(a < INFINITY) || !(b < INFINITY);
              mx = fmaxf(mx, fmaxf(a, b));
            }
            const uint32_t row_lanes = (kL == 32 ? 0xffffffffu : ((1u << kL) - 1u)) << (sub * kL);
            bad = (__ballot_sync(0xffffffffu, bad) & row_lanes) != 0;
#pragma unroll
            for (int off = kL / 2; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            if (!is_v) {
              const int e = clamp_exp(14 - ilog2(mx));
              const float up = pow2i(e);
#pragma unroll
              for (int i = 0; i < 4; ++i) w[i] = pack_half2(bf16_lo(w[i]) * up, bf16_hi(w[i]) * up);
              if (ch == 0) s_kf[g % kInfo][r] = pow2i(-e);
            }
            if (bad) {
#pragma unroll
              for (int i = 0; i < 4; ++i) w[i] = 0u;
              if (ch == 0) atomicOr(&s_bad[g % kInfo][r / 32], 1u << (r & 31));
            }
            st_shared_v4(dst + (ch / 8) * (BN * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4), w[0], w[1], w[2], w[3]);
          }
        }
        // the MMA reads the tile through the async proxy
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[op.i]);
          mbar_arrive(&raw_empty[raw.i]);
        }
      }
    }
  } else if (warp == kWarpScan) {
    // -------------------------------------------------- scales' exponents
    // ahead of the conversion: a tile's largest scales fix the powers of two
    // that its keys and values are taken with, and the scales become the fp16
    // pairs that multiply the codes, in place
    Ring<NR> raw;
    int g = 0;
    for (int x = x0; x < x1 && !fail;) {
      const Seg s = seg_at(p, x, x1);
      x += s.t1 - s.t0;
      int e_v = INT_MAX;  // the exponent that V's operands have in O (unset)
#pragma unroll 1
      for (int t = live_tile(pl, s, s.t0); t < s.t1; t = live_tile(pl, s, t + 1), ++g, raw.next()) {
        const int st = raw.i;
        float4 info = make_float4(1.f, 1.f, 1.f, 0.f);
        if (t < pl.ts + pl.tr) {
          if (!ring_wait(&raw_full[st], raw.phase, p.err, abort_flag)) {
            fail = true;
            break;
          }
          const int left = (t >= pl.ts ? s.nv - (t - pl.ts) * BN : s.sl - t * BN);
          const uint32_t rks = sR(st) + 2 * Y::kCodes, rvs = rks + Y::kScales;
          constexpr int kPer = BN * NG / 32;
          float ksc[kPer], vsc[kPer], km = 0.f, vm = 0.f;
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int idx = lane + 32 * i;
            // a slot behind the last: whatever is staged counts 0
            ksc[i] = idx / NG < left ? lds_f32(rks + 4 * idx) : 0.f;
            vsc[i] = idx / NG < left ? lds_f32(rvs + 4 * idx) : 0.f;
            km = fmaxf(km, fabsf(ksc[i]));
            vm = fmaxf(vm, fabsf(vsc[i]));
          }
          // (of values >= 0 the bits order as the values do)
          km = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(km)));
          vm = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vm)));
          // |code * scale| < 2^(ilog2 + 8): K below 2^15, V first below 2^12
          const int e_k = clamp_exp(7 - ilog2(km));
          if (vm > 0.f) {
            const int want = min(kMostUp, clamp_exp(4 - ilog2(vm)));
            if (e_v == INT_MAX) {
              e_v = want;  // every value so far was 0, and so is O
            } else if (want + 3 < e_v) {
              info.y = pow2i(max(want - e_v, -126));
              e_v = want;
            }
          }
          const float up_k = pow2i(e_k), up_v = e_v == INT_MAX ? 1.f : pow2i(e_v);
          info.x = pow2i(-e_k);
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int idx = lane + 32 * i;
            const float a = ksc[i] * up_k, b = vsc[i] * up_v;
            sts32(rks + 4 * idx, pack_half2(a, a));
            sts32(rvs + 4 * idx, pack_half2(b, b));
          }
        } else {
          const int j0 = (t - pl.ts - pl.tr) * kNodes + lane;
          const int32_t *depth = p.depth + int64_t(s.b) * p.n;
          const uint32_t lo = __ballot_sync(0xffffffffu, j0 < p.n && depth[min(j0, p.n - 1)] >= 0);
          const uint32_t hi = __ballot_sync(0xffffffffu, j0 + 32 < p.n && depth[min(j0 + 32, p.n - 1)] >= 0);
          if (lane == 0) {
            s_live[g % kInfo] = make_uint2(lo, hi);
            s_bad[g % kInfo][0] = s_bad[g % kInfo][1] = 0u;
          }
          if (!ring_wait(&raw_full[st], raw.phase, p.err, abort_flag)) {
            fail = true;
            break;
          }
          // nodes follow the segment's cached tiles: from here on O stays in this scale
          if (e_v == INT_MAX) e_v = 0;
        }
        __syncwarp();
        if (lane == 0) {
          // 2^-e of K; the factor that O needs before this tile's V; 2^-e of V; e of V
          info.z = e_v == INT_MAX ? 1.f : pow2i(-e_v);
          info.w = e_v == INT_MAX ? 0.f : float(e_v);
          s_info[g % kInfo] = info;
          mbar_arrive(&scan_full[st]);
          mbar_arrive(&raw_empty[st]);
        }
      }
    }
  } else if (warp == kWarpS) {
    // -------------------------------------------------- S(g) = Q K(g)^T
    const uint32_t leader = elect_one();
    constexpr uint32_t kId = idesc_f16(BM, BN, 0), kIdNodes = idesc_f16(BM, kNodes, 0);
    Ring<NK> kr;
    Ring<2> sr;  // a buffer is free once PV has read the P in it
    sr.phase = 1;
    uint32_t q_phase = 0;
    const uint64_t dk = sdesc_sw128(sK, 16, 1024);
    for (int x = x0; x < x1 && !fail;) {
      const Seg s = seg_at(p, x, x1);
      x += s.t1 - s.t0;
      fail = !ring_wait(&q_full, q_phase, p.err, abort_flag);
      q_phase ^= 1u;
#pragma unroll 1
      for (int t = live_tile(pl, s, s.t0); t < s.t1 && !fail; t = live_tile(pl, s, t + 1), kr.next(), sr.next()) {
        if (!ring_wait(&k_full[kr.i], kr.phase, p.err, abort_flag) ||
            !ring_wait(&pv_done[sr.i], sr.phase, p.err, abort_flag)) {
          fail = true;
          break;
        }
        tc_fence_after();
        const uint64_t kd = dk + uint64_t(kr.i * (Y::kKV >> 4));
        const uint32_t id = t < pl.ts + pl.tr ? kId : kIdNodes;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)  // 16 channels = 8 TMEM columns of Q's fp16 pairs
          mma_ts(tmem + sr.i * BN, tQ + kk * 8, kd + (kk >> 2) * (BN * 128 >> 4) + (kk & 3) * 2, id, kk > 0 ? 1u : 0u, leader);
        mma_commit(&s_full[sr.i], leader);
        mma_commit(&k_empty[kr.i], leader);
      }
    }
  } else if (warp == kWarpPV) {
    // -------------------------------------------------- O += P(g) V(g)
    // (a segment's first product overwrites O: its P exists only once the
    // softmax warps have read the segment before out of it)
    const uint32_t leader = elect_one();
    constexpr uint32_t kId = idesc_f16(BM, D, 1), kIdNodes = idesc_bf16(BM, D, 1);
    Ring<NV> vr;
    Ring<2> pr;
    const uint64_t dv = sdesc_sw128(sV, BN * 128, 1024);
    for (int x = x0; x < x1 && !fail;) {
      const Seg s = seg_at(p, x, x1);
      x += s.t1 - s.t0;
      uint32_t more = 0;
#pragma unroll 1
      for (int t = live_tile(pl, s, s.t0); t < s.t1 && !fail; t = live_tile(pl, s, t + 1), vr.next(), pr.next(), more = 1) {
        if (!ring_wait(&v_full[vr.i], vr.phase, p.err, abort_flag) ||
            !ring_wait(&p_full[pr.i], pr.phase, p.err, abort_flag)) {
          fail = true;
          break;
        }
        tc_fence_after();
        const uint64_t vd = dv + uint64_t(vr.i * (Y::kKV >> 4));
        const uint32_t tP = tmem + pr.i * BN;
        if (t < pl.ts + pl.tr) {
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            mma_ts(tO, tP + kk * 8, vd + kk * (16 * 128 >> 4), kId, kk > 0 ? 1u : more, leader);
        } else {
#pragma unroll
          for (int kk = 0; kk < kNodes / 16; ++kk)
            mma_ts(tO, tP + kk * 8, vd + kk * (16 * 128 >> 4), kIdNodes, kk > 0 ? 1u : more, leader);
        }
        mma_commit(&pv_done[pr.i], leader);
        mma_commit(&v_empty[vr.i], leader);
      }
    }
  }
  } else {
    // -------------------------------------------------- softmax warps
    regs_inc<kRegsSoftmax>();
    const uint32_t lane_base = uint32_t(warp * 32) << 16;
    const int r_blk = tid & (kLanes - 1), copy = tid / kLanes;  // row of the block; which copy of it
    const int col0 = copy * kCols;
    const int R = p.n * p.G, r = blk * pl.rb + r_blk;
    const bool exists = r_blk < pl.rb && r < R;
    auto node_of = [&](int row) { return p.G == 1 ? row : int(__umulhi(unsigned(row), p.g_magic)); };
    const int node = exists ? node_of(r) : 0;
    const uint32_t my_t = sT + warp * (32 * Y::kRow);
    Ring<2> sr;
    Ring<NV> vr;
    int g = 0;
    for (int x = x0; x < x1 && !fail;) {
      const Seg s = seg_at(p, x, x1);
      const bool first_seg = x == x0;
      x += s.t1 - s.t0;
      const int hk = s.pair - s.b * p.c.n_kv_heads;
      const int depth = exists ? p.depth[int64_t(s.b) * p.n + node] : -1;
      // ---- Q: the warp's 32 rows, D / 8 lanes to a row, turned over to a row
      // per lane in shared memory, as fp16 times 2^eq of the row
      float c_row;
      bool dead = !s.sane || depth < 0;
      {
        constexpr int kL = D / 8, kRows = 32 / kL, kIt = 32 / kRows;
        const int sub = lane / kL, ch = lane % kL;
        uint4 w[kIt];
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
          const int rb_ = (warp * 32 + i * kRows + sub) & (kLanes - 1), rw = blk * pl.rb + rb_;
          const bool ok = rb_ < pl.rb && rw < R;
          const int nd = ok ? node_of(rw) : 0;
          const uint16_t *src = p.q + ((int64_t(s.b) * p.n + nd) * p.Hq + hk * p.G + (ok ? rw - nd * p.G : 0)) * D + 8 * ch;
          w[i] = ok ? *reinterpret_cast<const uint4 *>(src) : make_uint4(0u, 0u, 0u, 0u);
        }
        uint32_t row[D / 2];
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          __syncwarp();
          if (D == 64 || ch / 8 == h) {
#pragma unroll
            for (int i = 0; i < kIt; ++i)
              st_shared_v4(my_t + (i * kRows + sub) * Y::kRow + (ch & 7) * 16, w[i].x, w[i].y, w[i].z, w[i].w);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            ld_shared_v4(my_t + lane * Y::kRow + i * 16, row[h * 32 + 4 * i], row[h * 32 + 4 * i + 1], row[h * 32 + 4 * i + 2],
                         row[h * 32 + 4 * i + 3]);
        }
        float qm = 0.f;
        bool finite = true;
#pragma unroll
        for (int i = 0; i < D / 2; ++i) {
          const float a = fabsf(bf16_lo(row[i])), b = fabsf(bf16_hi(row[i]));
          finite = finite && a < INFINITY && b < INFINITY;
          qm = fmaxf(qm, fmaxf(a, b));
        }
        dead = dead || !finite;
        const int eq = clamp_exp(14 - ilog2(qm));
        const float up = pow2i(eq);
#pragma unroll
        for (int i = 0; i < D / 2; ++i) row[i] = dead ? 0u : pack_half2(bf16_lo(row[i]) * up, bf16_hi(row[i]) * up);
        c_row = pow2i(-eq) * (1.4426950408889634f * rsqrtf(float(D)));
        // (the products that read the Q before are done: the warp waited for its last S)
#pragma unroll
        for (int h = 0; h < D / 64; ++h) tmem_st32(tQ + lane_base + 32 * h, row + 32 * h);
        tmem_st_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full);

      // ring entries below `low` are outside the row's window
      // (a dead row takes what comes and is put to 0 at the end)
      const int low = dead ? 0 : int(min((long long)INT_MAX, max(0ll, (long long)depth + s.nv - p.window + 1)));
      float m_used = -INFINITY, l = 0.f, down = 1.f;
      bool any = false;
      uint64_t *pv_last = nullptr;  // PV of the tile before: its barrier and parity
      uint32_t pv_phase = 0;
#pragma unroll 1
      for (int t = live_tile(pl, s, s.t0); t < s.t1; t = live_tile(pl, s, t + 1), ++g, sr.next(), vr.next()) {
        const int u = sr.i;
        const bool nodes = t >= pl.ts + pl.tr;
        if (!fail) fail = !ring_wait(&s_full[u], sr.phase, p.err, abort_flag);
        // what the warps that turn a node tile say of it: K's were done before S
        if (nodes && !fail) fail = !ring_wait(&v_full[vr.i], vr.phase, p.err, abort_flag);
        tc_fence_after();
        uint64_t *const pv_prev = pv_last;
        const uint32_t pv_prev_phase = pv_phase;
        pv_last = &pv_done[u];
        pv_phase = sr.phase;
        const float4 info = s_info[g % kInfo];
        down = info.z;
        uint32_t v[kCols];
        // never 0, which would make NaN of a masked column's -inf: |S| < 2^37, so at
        // 2^-126 and below a score is 2^-89 at most and its weight 1 to every bit
        float ct = fmaxf(c_row * info.x, 1.1754943508222875e-38f);
        const uint32_t tS = tmem + u * BN + lane_base;
        if (!nodes) {
#pragma unroll
          for (int i = 0; i < kCols; i += 32) tmem_ld32(tS + col0 + i, v + i);
          tmem_ld_wait();
          // columns [lo, hi) are seen
          const bool ring = t >= pl.ts;
          const int first = (ring ? t - pl.ts : t) * BN + col0;
          const int hi = (ring ? s.nv : s.sl) - first;
          const int lo = ring ? max(low, first) - first : 0;
          if (__any_sync(0xffffffffu, lo > 0 || hi < kCols)) {
#pragma unroll
            for (int i = 0; i < kCols; ++i) v[i] = i >= lo && i < hi ? v[i] : 0xff800000u;
          }
        } else if (col0 < kNodes) {
          // 64 columns: the copies behind them see nothing of a node tile
          const int t_n = t - pl.ts - pl.tr, words = (p.n + 31) / 32;
          constexpr int kC = kCols < kNodes ? kCols : kNodes;
#pragma unroll
          for (int i = 0; i < kC; i += 32) tmem_ld32(tS + col0 + i, v + i);
          tmem_ld_wait();
          const uint32_t *mk = p.mask + (int64_t(s.b) * p.n + node) * words;
          const uint2 alive = s_live[g % kInfo];
#pragma unroll
          for (int i = 0; i < kC; i += 32) {
            const int wd = (col0 + i) / 32;
            const uint32_t bad = s_bad[g % kInfo][wd];
            uint32_t see = 0u;
            if (!dead && 2 * t_n + wd < words) see = mk[2 * t_n + wd] & (wd ? alive.y : alive.x);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float sc = __uint_as_float(v[i + e]) * s_kf[g % kInfo][col0 + i + e];
              v[i + e] = see >> e & 1u ? (bad >> e & 1u ? 0x7fffffffu : __float_as_uint(sc)) : 0xff800000u;
            }
          }
#pragma unroll
          for (int i = kC; i < kCols; ++i) v[i] = 0xff800000u;
        } else {
#pragma unroll
          for (int i = 0; i < kCols; ++i) v[i] = 0xff800000u;
        }
        float mxp[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mxp[i] = __uint_as_float(v[i]);
#pragma unroll
        for (int j = 8; j + 16 <= kCols; j += 16)
#pragma unroll
          for (int i = 0; i < 8; ++i) mxp[i] = max3(mxp[i], __uint_as_float(v[j + i]), __uint_as_float(v[j + 8 + i]));
#pragma unroll
        for (int i = 0; i < 8; ++i) mxp[i] = fmaxf(mxp[i], __uint_as_float(v[kCols - 8 + i]));
        const float mx = ct * max3(max3(mxp[0], mxp[1], mxp[2]), max3(mxp[3], mxp[4], mxp[5]), fmaxf(mxp[6], mxp[7]));
        const bool need = mx > m_used + kLazyLog2;  // the first tile with a key included
        float alpha = info.y;  // what V's new exponent asks of O
        if (need) {
          const float a = ex2(m_used - mx);  // 0 at the first
          alpha *= a;
          l *= a;
          m_used = mx;
        }
        // nodes' weights carry V's exponent
        const float shift = kPBias - (m_used == -INFINITY ? 0.f : m_used) + (nodes ? info.w : 0.f);
        const uint64_t c2 = pack_f32x2(ct, ct), nmc2 = pack_f32x2(shift, shift);
        float rsp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kCols; i += 2) {
          float a, b;
          fma_f32x2(a, b, __uint_as_float(v[i]), __uint_as_float(v[i + 1]), c2, nmc2);
          a = ex2(a);
          b = ex2(b);
          add_f32x2(rsp[(i >> 1) & 1 ? 2 : 0], rsp[(i >> 1) & 1 ? 3 : 1], a, b);
          v[i / 2] = nodes ? pack_bf16x2(a, b) : pack_half2(a, b);
        }
        const float sum = (rsp[0] + rsp[1]) + (rsp[2] + rsp[3]);
        l += nodes ? sum * info.z : sum;
        if (any && __any_sync(0xffffffffu, alpha != 1.f)) {
          // O once the PV before has landed
          if (!fail) fail = !ring_wait(pv_prev, pv_prev_phase, p.err, abort_flag);
          tc_fence_after();
#pragma unroll 1
          for (int ch = 0; ch < D; ch += 32) {
            uint32_t ov[32];
            tmem_ld32(tO + lane_base + ch, ov);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tmem_st32(tO + lane_base + ch, ov);
          }
        }
        any = true;
        // P over S: this copy's columns, zeros in the others'
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t out[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if constexpr (REP == 1) out[i] = v[h * 32 + i];
            else if constexpr (REP == 2) out[i] = copy == h ? v[i] : 0u;
            else out[i] = copy == 2 * h + i / 16 ? v[i % 16] : 0u;
          }
          tmem_st32(tS + 32 * h, out);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[u]);
      }
      // ---- the segment's end
      if (any && !fail) fail = !ring_wait(pv_last, pv_phase, p.err, abort_flag);
      tc_fence_after();
      if constexpr (REP > 1) fail = softmax_any(fail);  // (the barriers below want all four warps)
      if (dead) m_used = -INFINITY, l = 0.f;
      if (s.all) {
        // copies merge: the row's weight of each, then the sum through shared memory
        float scale = l > 0.f || !(l <= 0.f) ? down / l : 0.f;
        float m_all = m_used, l_all = l;
        if constexpr (REP > 1) {
          s_ml[tid] = make_float2(m_used, l);
          asm volatile("bar.sync 1, 128;" ::: "memory");
          float mm = -INFINITY;
#pragma unroll
          for (int c = 0; c < REP; ++c) mm = fmaxf(mm, s_ml[c * kLanes + r_blk].x);
          l_all = 0.f;
#pragma unroll
          for (int c = 0; c < REP; ++c) {
            const float2 o = s_ml[c * kLanes + r_blk];
            l_all += o.x == -INFINITY && o.y == 0.f ? 0.f : o.y * ex2(o.x - mm);
          }
          m_all = mm;
          scale = m_used == -INFINITY && l == 0.f ? 0.f : (l_all != 0.f ? ex2(m_used - mm) * down / l_all : 0.f);
        }
        const int64_t row = ((int64_t(s.b) * p.n + node) * p.Hq + hk * p.G + (r - node * p.G));
        uint16_t *dst = p.out + row * D;
        // 32 channels at a time; of several copies the first adds the others'
#pragma unroll 1
        for (int ch = 0; ch < D; ch += 32) {
          uint32_t ov[32];
          if (any) {
            tmem_ld32(tO + lane_base + ch, ov);
            tmem_ld_wait();
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) ov[i] = any && scale != 0.f ? __float_as_uint(__uint_as_float(ov[i]) * scale) : 0u;
          if constexpr (REP > 1) {
            // a lane's 32 floats in its warp's buffer: 132 bytes would not keep 16-byte stores aligned, 144 does
            if (copy > 0) {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                st_shared_v4(my_t + lane * Y::kRow + 4 * i, ov[i], ov[i + 1], ov[i + 2], ov[i + 3]);
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (copy == 0) {
#pragma unroll
              for (int c = 1; c < REP; ++c) {
                const uint32_t src = sT + (c * kLanes / 32 + warp) * (32 * Y::kRow) + lane * Y::kRow;
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                  uint32_t a0, a1, a2, a3;
                  ld_shared_v4(src + 4 * i, a0, a1, a2, a3);
                  ov[i] = __float_as_uint(__uint_as_float(ov[i]) + __uint_as_float(a0));
                  ov[i + 1] = __float_as_uint(__uint_as_float(ov[i + 1]) + __uint_as_float(a1));
                  ov[i + 2] = __float_as_uint(__uint_as_float(ov[i + 2]) + __uint_as_float(a2));
                  ov[i + 3] = __float_as_uint(__uint_as_float(ov[i + 3]) + __uint_as_float(a3));
                }
              }
            }
          }
          if (copy == 0 && exists && !fail) {
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              st_global_v4(dst + ch + i, pack_bf16x2(__uint_as_float(ov[i]), __uint_as_float(ov[i + 1])),
                           pack_bf16x2(__uint_as_float(ov[i + 2]), __uint_as_float(ov[i + 3])),
                           pack_bf16x2(__uint_as_float(ov[i + 4]), __uint_as_float(ov[i + 5])),
                           pack_bf16x2(__uint_as_float(ov[i + 6]), __uint_as_float(ov[i + 7])));
          }
          if constexpr (REP > 1) asm volatile("bar.sync 1, 128;" ::: "memory");
        }
        if (copy == 0 && exists && p.lse && !fail)
          p.lse[(int64_t(s.b) * p.Hq + hk * p.G + (r - node * p.G)) * p.n + node] =
              l_all != 0.f ? 0.6931471805599453f * (m_all - kPBias + log2f(l_all)) : -INFINITY;
      } else if (!fail) {
        float *part = p.parts + (size_t(blockIdx.x) * 2 + (first_seg ? 0 : 1)) * part_floats<D>();
        if (any) {
#pragma unroll 1
          for (int ch = 0; ch < D; ch += 32) {
            uint32_t ov[32];
            tmem_ld32(tO + lane_base + ch, ov);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4 *>(part + ((ch + i) / 4 * BM + tid) * 4) =
                  make_float4(__uint_as_float(ov[i]) * down, __uint_as_float(ov[i + 1]) * down,
                              __uint_as_float(ov[i + 2]) * down, __uint_as_float(ov[i + 3]) * down);
          }
        }
        *reinterpret_cast<float2 *>(part + BM * D + 2 * tid) = make_float2(m_used, l);
      }
      tc_fence_before();
    }
  }

  // ---- common exit: on the error path give copies and MMAs still in flight a
  //      bounded time (about 2 ms) to land before shared memory and TMEM go
  tc_fence_before();
  if (__syncthreads_or(fail || *abort_flag))
    for (int i = 0; i < 2000; ++i) __nanosleep(1000);
  __syncthreads();
  if (warp == kWarpS) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Y::kTmemCols) : "memory");
  }
}

// ------------------------------------------------------------ the merge
struct MergeParams {
  const float *parts;
  TreePlan plan;
  int n, Hq, Hkv, G, lanes;  // lanes: of a copy of the rows
  uint16_t *out;
  float *lse;
};

// grid (pairs that may be split, row blocks, channels by 16); a warp has 8 rows
// and 4 groups of 4 channels, so its loads take 128 bytes in a piece and its
// stores a sector.
template <int D>
__global__ void __launch_bounds__(512) tree_merge_kernel(const __grid_constant__ MergeParams p) {
  const TreePlan &pl = p.plan;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();  // (also where nothing is to merge: the next kernel waits for this one alone)
  int pair = blockIdx.x;
  if (pl.pairs > pl.ctas) {
    // the pair that the cut behind stretch blockIdx.x goes through, if it is
    // the first such cut
    const int x = pl.start(blockIdx.x + 1);
    pair = x / pl.t;
    if (x == pair * pl.t || pl.start(blockIdx.x) > pair * pl.t) return;
  }
  const int c0 = pl.owner(pair * pl.t), c1 = pl.owner((pair + 1) * pl.t - 1);
  if (c0 == c1) return;  // its one segment wrote the output
  const int blk = blockIdx.y, r_blk = warp * 8 + lane / 4, r = blk * pl.rb + r_blk, R = p.n * p.G;
  const int quad = blockIdx.z * 4 + lane % 4, copies = BM / p.lanes;
  if (r_blk >= pl.rb || r >= R) return;
  auto part = [&](int c) {
    const int which = c == c0 && pl.start(c) < pair * pl.t ? 1 : 0;
    return p.parts + ((size_t(c) * pl.nb + blk) * 2 + which) * part_floats<D>();
  };
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = c0; c <= c1; ++c) {
    const float *src = part(c);
    for (int k = 0; k < copies; ++k) {
      const int at = k * p.lanes + r_blk;
      const float2 ml = *reinterpret_cast<const float2 *>(src + BM * D + 2 * at);
      if (ml.x == -INFINITY && ml.y == 0.f) continue;  // saw nothing
      const float4 v = *reinterpret_cast<const float4 *>(src + (quad * BM + at) * 4);
      const float mn = fmaxf(m, ml.x), a = mn == -INFINITY ? 0.f : ex2(m - mn), b = mn == -INFINITY ? 1.f : ex2(ml.x - mn);
      m = mn;
      l = l * a + ml.y * b;
      o = make_float4(o.x * a + v.x * b, o.y * a + v.y * b, o.z * a + v.z * b, o.w * a + v.w * b);
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  const int node = r / p.G, h = pair % p.Hkv * p.G + r % p.G, b = pair / p.Hkv;
  *reinterpret_cast<uint2 *>(p.out + ((int64_t(b) * p.n + node) * p.Hq + h) * D + quad * 4) =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (p.lse && quad == 0)
    p.lse[(int64_t(b) * p.Hq + h) * p.n + node] = l != 0.f ? 0.6931471805599453f * (m - kPBias + log2f(l)) : -INFINITY;
}

template <int D, int REP>
cudaError_t launch_main(const TreeParams &p, cudaStream_t stream) {
  auto kern = tree_decode_kernel<D, REP>;
  static std::atomic<unsigned long long> smem_set{0};  // the opt-in, once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
  if (!bit || !(smem_set.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::kBytes);
    if (e != cudaSuccess) return e;
    smem_set.fetch_or(bit, std::memory_order_release);
  }
  return launch_pdl(kern, dim3(p.plan.ctas * p.plan.nb), dim3(kThreads), size_t(Lay<D>::kBytes), stream, p);
}

template <int D>
cudaError_t launch_d(const TreeParams &p, cudaStream_t stream) {
  const TreePlan &pl = p.plan;
  const int lanes = pl.rows_of_lanes();
  const cudaError_t e = lanes == 32 ? launch_main<D, 4>(p, stream) : lanes == 64 ? launch_main<D, 2>(p, stream)
                                                                                 : launch_main<D, 1>(p, stream);
  if (e != cudaSuccess || pl.whole) return e;
  const MergeParams m = {p.parts, pl, p.n, p.Hq, p.c.n_kv_heads, p.G, lanes, p.out, p.lse};
  const dim3 grid(pl.pairs > pl.ctas ? pl.ctas - 1 : pl.pairs, pl.nb, D / 16);
  return launch_pdl(tree_merge_kernel<D>, grid, dim3((pl.rb + 7) / 8 * 32), 0, stream, m);
}

}  // namespace

bool tree_decode_fits(int batch, int n, int n_kv_heads, int sink_cap, int ring_cap) {
  const long long t = (sink_cap + (long long)BN - 1) / BN + (ring_cap + (long long)BN - 1) / BN + (n + kNodes - 1) / kNodes;
  return (long long)batch * n_kv_heads * t < (1 << 30);
}

// For any sink_cap + ring_cap = max_slots: one may leave a tile more than the other.
size_t tree_decode_workspace_bytes(int batch, int n, int n_q_heads, int n_kv_heads, int head_dim, int max_slots) {
  const TreePlan p = tree_plan(batch, n, n_q_heads, n_kv_heads, max_slots, 1);
  if (p.whole) return 0;
  return size_t(p.ctas) * p.nb * 2 * (head_dim == 128 ? part_floats<128>() : part_floats<64>()) * sizeof(float);
}

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
  p.g_magic = p.G > 1 ? unsigned((0x100000000ull + p.G - 1) / p.G) : 0u;
  p.window = a.window;
  p.out = static_cast<uint16_t *>(a.out);
  p.lse = a.lse;
  p.parts = static_cast<float *>(ws);
  p.plan = tree_plan(c.batch, a.n, a.n_q_heads, c.n_kv_heads, c.sink_cap, c.ring_cap);
  p.err = err;
  return c.head_dim == 64 ? launch_d<64>(p, stream) : launch_d<128>(p, stream);
}

}  // namespace nd
