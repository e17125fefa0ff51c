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
// Types.  Cached keys and values become fp16: code * fp16(scale * 2^e) * 2^-24,
// rounded once, e per 32 keys, with the largest scale in [2^14, 2^15).  (The
// 2^-24 lets one fused multiply and add turn a pair of codes, see scaled_codes;
// operands 2^-21 below the largest of the 32 keys are subnormal.)  K's e is a
// factor of its columns' scores, V's of their weights, which are brought to the
// power of two that O holds V in, the lowest e so far: O is rescaled where a tile
// lowers it.  q (bf16) becomes fp16 exactly after a power of two per row (channels
// 2^-28 below the row's largest lose bits).  A node's key gets a power of two of
// its own and is then exact in the same way; its values stay bf16, and their
// weights are bf16 (2^-8 of themselves) with O's power of two, which bf16's range
// has room for.  Cached keys' weights are fp16 with the running maximum up to 2^8
// behind and all of it scaled by 2^7.  Sums, maxima and partials are fp32.
//
// Masked places.  A weight of 0 times a NaN or an infinity would be NaN, so
// slots and nodes that nothing may see are 0 in the operands.  A node whose key
// or value is not finite is 0 too and makes NaN of the scores of the rows that
// see it; so is a cached slot with a scale that is not finite, which counts nothing
// for its keys' exponent and makes NaN of the sums of the rows that see it (the
// window may hide it from deeper ones).  A row that sees nothing (or whose query
// is not finite) ends with m = -inf and l = 0 and comes out 0.
//
// Lanes.  The products have 128 rows whatever R is.  With R <= 64 (32) the rows
// stand two (four) times in Q, and each copy takes its own half (quarter) of a
// tile's columns, with a maximum, sum and O of its own, so that all lanes' warps
// work; the copies merge at the end like any triples.
//
// Work split.  The ((sequence, KV head), tile) pairs, tiles fastest, form one
// line that is cut into equal stretches, one per CTA and row block (one CTA per
// SM); row blocks of one stretch run side by side and share their codes in L2.
// A stretch is one or more segments (tiles of one (sequence, KV head)); one
// that has all of its tiles writes the output, others write their triple for
// tree_merge_kernel.  The line counts the tiles that the caches have room for;
// those that hold nothing are skipped.
//
// Roles (20 warps):
//   warps 0-7   : softmax: two threads to a TMEM lane, on alternate tiles: read S,
//                 write P; between segments write the output and stage Q
//   warps 8-15  : codes (or nodes' bf16) of the staged tile -> K, V operands in
//                 shared memory, half of them K, half V, and their exponents
//   warps 16, 17: note the tiles of K and V ahead, copy them
//   warps 18, 19: MMA issuers: S = Q K^T; O += P V
// Every wait is bounded: one that gives up sets the abort flag, all roles leave
// through the common exit, and that raises the device error flag.
//
// What bounds it.  Below about 150 rows the read of the codes, above the
// products.  Measured (D = 128): 128 sessions of 16 nodes (64 rows) over 1280
// slots of 8 heads 129 us, the bytes 62 (48 % of the copy rate); 8 sessions of 64
// nodes (256 rows) over 33024 slots 270 to 275 us in a graph, 283 to 287 call by
// call, the products 142 (50 to 53 %).  No unit is busy for much more than half of
// that: with conversion, exponentials and products all left out, the roles' waits
// and bookkeeping alone took 111 (of 139) and 208 (of 366) us.  A warp issues an instruction every five cycles, held up by
// latencies, by the others and by instruction fetches: code that is not needed for
// most tiles costs all of them (see tile() and ring_wait()).  Without effect on
// these two: 16 warps that convert, four that stage Q beside the softmax, three
// staged tiles and one operand; asking codes into L2 cost 5 %.
#include <atomic>
#include <climits>
#include <type_traits>

#include "nd_common.cuh"
#include "nd_internal.h"
#include "tc_ptx.cuh"

namespace nd {

namespace {

constexpr int BM = 128;        // rows of a product = TMEM lanes
constexpr int BN = 128;        // cached keys per tile
constexpr int kNodes = 64;     // nodes per tile
constexpr int kThreads = 20 * 32;
constexpr int kWarpTurn = 8, kWarpFeedK = 16, kWarpFeedV = 17, kWarpS = 18;
// Register split (setmaxnreg, per warpgroup) of the 96 a thread at launch: a
// softmax thread holds up to 64 scores.
constexpr int kRegsLaunch = 96, kRegsSoftmax = 144, kRegsOther = 64;
static_assert(2 * 128 * kRegsSoftmax + 3 * 128 * kRegsOther <= kThreads * kRegsLaunch, "register split");
constexpr int kBatch = 8;         // tiles that are noted at once
constexpr int kKf = 8;            // node tiles' key factors in flight: more than the tiles between operand and softmax
constexpr float kLazyLog2 = 8.f;  // the maximum used may lag the true one by 2^8
constexpr float kPBias = 7.f;     // P is scaled by 2^7
constexpr int kCodeBits = 24;     // operands made of codes hold 2^-24 of code * scale * 2^e
constexpr int kMostUp = 88;       // V's largest e: a node's value times 2^(88 - 24 + 15) stays finite up to 2^48
constexpr float kUnits = 16777216.f;  // 2^24
constexpr int kCtas = 152;        // one per SM
// A pair of so few tiles is not split while every pair has a CTA: whole against
// split, 3 and 4 tiles (cached ones and nodes) of 2 to 128 pairs took 8.6 to 10 us
// against 11 to 19 with heads of 64 (8 nodes, 4 query heads per KV head), 11.3 to
// 13.3 against 13.2 to 24.7 with heads of 128 (16 nodes).  At 8 tiles 20 pairs are as
// fast either way (11.8 against 13.3, 16.7 against 15.4), 64 and more faster whole
// (12.0 against 20.5, 17.1 against 24.4).
constexpr int kFewTiles = 4;

// ------------------------------------------------------------ the split
struct TreePlan {
  int ts, tr, tn, t;   // tiles of the sinks, the ring and the nodes, and all
  int pairs;           // (sequence, KV head)
  int nb, rb;          // row blocks, rows of each
  int ctas;            // stretches
  int even, odd;       // units / ctas and units % ctas
  bool whole;          // a unit is a pair (nothing is split), else a tile
  __host__ __device__ int start(int c) const {
    const int u = even * c + odd * c / ctas;  // = units * c / ctas
    return whole ? u * t : u;
  }
  // the stretch that holds tile x of the line
  __device__ int owner(int x) const {
    int c = min(ctas - 1, int(float(x) * float(ctas) / (float(pairs) * float(t))));
    while (start(c) > x) --c;
    while (start(c + 1) <= x) ++c;
    return c;
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
  // whole pairs where that leaves at most a sixteenth of the CTAs' time idle, or
  // the parts would be shorter than their merge; else two tiles a stretch at least
  p.whole = (long long)((p.pairs + most - 1) / most) * most * 16 <= (long long)p.pairs * 17 ||
            (p.t <= kFewTiles && p.pairs <= most);
  const long long units = p.whole ? p.pairs : tiles, ctas = p.whole ? units : (units + 1) / 2;
  p.ctas = int(ctas < most ? ctas : most);
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
// A tile's record: whether it is nodes, whether its segment begins and the stretch
// ends with it, keys (bits 8-15) and those in the first piece (16-23).
constexpr int kKindNodes = 1, kFresh = 2, kLast = 4;

template <int D>
struct Lay {
  static constexpr int NG = D / 32, kBoxes = D / 64;
  static constexpr int kKV = kBoxes * BN * 128;          // one K or V operand tile
  static constexpr int kCodes = BN * D, kScales = BN * NG * 4;
  static_assert(kNodes * D * 2 == kCodes, "a node tile's rows take the codes' place");
  // stages: operands of K and of V; staged codes and scales (or nodes' rows) of either
  static constexpr int NK = D == 128 ? 2 : 3, NR = D == 128 ? 2 : 5;
  static constexpr int kRaw = kCodes + kScales;
  static constexpr int kRec = 32, kInfo = 16;            // tiles noted; tiles between operand and softmax
  static_assert(kRec >= 2 * kBatch + NR + NK + 2 && kInfo > NK + 3, "tile records");
  static constexpr int kT1 = 2048, kT = 8 * kT1;         // a softmax warp's turning buffer
  static constexpr int oK = 0, oV = oK + NK * kKV, oR = oV + NK * kKV, oT = oR + 2 * NR * kRaw, oSmall = oT + kT;
  // barriers; [2]: K, V
  struct Small {
    uint64_t raw_full[2][NR], raw_empty[2][NR], op_full[2][NK], op_empty[2][NK];
    uint64_t s_full[2], s_empty[2], p_full[2], pv_done[2], q_full, v_known[4];  // s_: score buffers
    int4 rec[2][kRec];           // tiles, as the feeders note them: flags (kFresh ...), first key, pair, slot
    // for the softmax
    int e[2][kInfo][4];          // exponents of each 32 keys
    uint16_t live[kInfo][4];     // node tiles: nodes that are not padding, 16 to a word
    uint16_t bad[2][kInfo][4];   // and those whose key, value is not finite
    float kf[kKf][kNodes];       // and 2^-e of their keys
    float m[2][BM];              // the rows' maxima, from a tile's softmax threads to the next one's
    float2 ml[BM];               // and what their copies have
    uint32_t tmem;
    int abort;
    int any_bad;                 // a slot so far has a scale that is not finite
  };
  static constexpr int kBytes = oSmall + int(sizeof(Small));
  static_assert(kBytes <= 227 * 1024, "shared memory");
  // TMEM columns: S[2], O, Q, P
  static constexpr int cO = 2 * BN, cQ = cO + D, cP = cQ + D / 2, kTmemCols = 512;
  static_assert(cP + BN / 2 <= kTmemCols, "TMEM");
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
// Asks a line into L2.
__device__ __forceinline__ void prefetch_l2(const void *src) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// A predicated store, not a branch: with one among the codes' warps the compiler
// spills in every role (128 sessions of 16 nodes 136 us against 129, 8 of 64 over
// 33024 slots 309 against 272).
__device__ __forceinline__ void set_if(int *flag, bool x) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %0, 0;\n @p st.shared.u32 [%1], 1;\n}\n" ::"r"(uint32_t(x)),
               "r"(smem_u32(flag))
               : "memory");
}
// A row's NG scales; and put back as pairs of fp16, times a power of two.
template <int NG>
__device__ __forceinline__ void lds_row(uint32_t a, float *x) {
  if constexpr (NG == 4)
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(a) : "memory");
  else
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x[0]), "=f"(x[1]) : "r"(a) : "memory");
}
template <int NG>
__device__ __forceinline__ void sts_row(uint32_t a, const float *x, float up) {
  uint32_t h[NG];
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const float y = x[i] * up;
    h[i] = pack_half2(y, y);
  }
  if constexpr (NG == 4) st_shared_v4(a, h[0], h[1], h[2], h[3]);
  else asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(h[0]), "r"(h[1]) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
// Two codes times a scale, in fp16 and rounded once.  A code biased to unsigned
// (xor 0x80) in the low byte of an fp16 is the subnormal (code + 128) 2^-24, and
// code * s 2^-24 = (code + 128) 2^-24 * s - s 2^-17, a fused multiply and add of
// exact operands (off = s * -2^-17 is exact down to s = 2^3, below that off by
// 2^-25).  One instruction less per pair than subtracting the bias first.
constexpr uint32_t kMinus128 = 0x80808080u;  // two fp16 -2^-17
constexpr uint32_t kBytes01 = 0x4140u, kBytes23 = 0x4342u;  // [b0, 0, b1, 0], [b2, 0, b3, 0]
__device__ __forceinline__ uint32_t scaled_codes(uint32_t biased, uint32_t sel, uint32_t s, uint32_t off) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(prmt(biased, 0u, sel)), "r"(s), "r"(off));
  return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
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

// A bounded wait of a whole warp that sleeps between polls (up to 2 us each).  One
// that gives up sets the abort flag, and the common exit raises the device's.
// All roles' loops together have to stay small enough for the SM's instruction
// cache: with 160 KB of code, a walk over the tiles in every role, the fetches
// from the cache behind it bounded the kernel (85 % of their rate; 210 us at 128
// sessions of 16 nodes).
__device__ __forceinline__ bool ring_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
  bool ok = mbar_test_wait(bar, parity);
#pragma unroll 1
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
  if (!ok) *abort_flag = 1;
  return __all_sync(0xffffffffu, ok);
}

// Whether any thread of the eight softmax warps says so; a barrier of theirs.
__device__ __forceinline__ bool softmax_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, 256, p;\n selp.u32 %0, 1, 0, q;\n}\n"
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

// The newest of a segment's ring entries with a scale that is not finite, INT_MAX
// where a sink has one, -1 where none has; a walk over the segment's scales by each
// warp, taken only by CTAs that have met such a slot.
template <int NG>
__device__ __noinline__ int bad_slots(const nd_kv_cache &c, int pair, int sink0, int sink1, int e0, int e1, int ring0) {
  const size_t base = pair * (size_t(c.sink_cap) + c.ring_cap);
  int newest = -1;
#pragma unroll 1
  for (int i = e0 - (sink1 - sink0) + int(threadIdx.x & 31); i < e1; i += 32) {  // sinks, as it were, before the entries
    const bool sink = i < e0;
    unsigned w = unsigned(ring0) + unsigned(max(i, 0));
    if (w >= unsigned(c.ring_cap)) w -= unsigned(c.ring_cap);
    const size_t at = (base + (sink ? size_t(sink1 - (e0 - i)) : size_t(c.sink_cap) + w)) * NG;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < NG; ++j) bad = bad || !(fabsf(c.k_scale[at + j]) < INFINITY) || !(fabsf(c.v_scale[at + j]) < INFINITY);
    if (bad) newest = sink ? INT_MAX : max(newest, i);
  }
  return __reduce_max_sync(0xffffffffu, newest);
}

template <int D, int REP>
__global__ void __launch_bounds__(kThreads, 1) tree_decode_kernel(const __grid_constant__ TreeParams p) {
  using Y = Lay<D>;
  constexpr int NK = Y::NK, NR = Y::NR, NG = Y::NG, kInfo = Y::kInfo, kRec = Y::kRec;
  constexpr int kLanes = BM / REP;     // rows, and lanes of a copy of them
  constexpr int kCols = BN / REP;      // a thread's columns of a tile
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  typename Y::Small &sm = *reinterpret_cast<typename Y::Small *>(smem_raw + Y::oSmall);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the same in the warp
  volatile int *abort_flag = &sm.abort;
  const uint32_t base = smem_u32(smem_raw);
  const uint32_t sK = base + Y::oK, sV = base + Y::oV, sT = base + Y::oT;
  auto sR = [&](int kv, int st) { return base + Y::oR + (kv * NR + st) * Y::kRaw; };

  if (tid == 0) {
    for (int kv = 0; kv < 2; ++kv) {
      for (int s = 0; s < NR; ++s) {
        mbar_init(&sm.raw_full[kv][s], NG == 4 ? 1 : 33);  // the bulk copies' transaction (D = 64: and the lanes' copies)
        mbar_init(&sm.raw_empty[kv][s], 4);                // the warps that turn it
      }
      for (int s = 0; s < NK; ++s) {
        mbar_init(&sm.op_full[kv][s], 4);
        mbar_init(&sm.op_empty[kv][s], 1);
      }
      mbar_init(&sm.s_full[kv], 1);
      mbar_init(&sm.s_empty[kv], 4);
      mbar_init(&sm.p_full[kv], 4);
      mbar_init(&sm.pv_done[kv], 1);
    }
    mbar_init(&sm.q_full, 8);
    for (int s = 0; s < 4; ++s) mbar_init(&sm.v_known[s], 4);
    sm.abort = 0;
    sm.any_bad = 0;
    fence_barrier_init();
  }
  if (warp == kWarpS) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem)),
                 "r"(Y::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);
  pdl_wait();
  pdl_trigger();  // the merge reads nothing of this kernel's before it waits
  const uint32_t tO = tmem + Y::cO, tQ = tmem + Y::cQ, tP = tmem + Y::cP;

  const TreePlan &pl = p.plan;
  const int stretch = blockIdx.x / pl.nb, blk = blockIdx.x % pl.nb;
  const int x0 = pl.start(stretch), x1 = pl.start(stretch + 1);
  bool fail = false;

  // (each side of the split has its setmaxnreg to itself: behind a common one the
  // compiler takes the smaller bound for all roles)
  if (warp >= kWarpTurn) {
    regs_dec<kRegsOther>();
    if (warp == kWarpFeedK || warp == kWarpFeedV) {
      // -------------------------------------------------- feeders, one for K and one for V
      // Ahead of the copies tiles are noted, kBatch at a time, a lane to a tile, and
      // queries and nodes asked into L2.  (Asking the codes too costs more than it
      // gives: 140 against 133 us at 128 sessions of 16 nodes.)
      const int kv = warp == kWarpFeedV;
      const uint32_t leader = elect_one();
      const int8_t *const codes = kv ? p.c.v_codes : p.c.k_codes;
      const float *const scales = kv ? p.c.v_scale : p.c.k_scale;
      const size_t nslot = size_t(p.c.sink_cap) + p.c.ring_cap;
      auto node_row = [&](int pair, int j) {
        const int b = pair / p.c.n_kv_heads;
        return (kv ? p.v : p.k) + (int64_t(b) * p.n + j) * (kv ? p.v_stride : p.k_stride) + (pair - b * p.c.n_kv_heads) * D;
      };
      Ring<NR> raw;
      raw.phase = 1;  // the first round of an empty ring does not wait
      int noted = 0, x = x0, t = 0;
      bool fresh = true;
      Seg s = {};
#pragma unroll 1
      for (int i = -1;; ++i) {
        if (i >= 0) {
          if (i >= noted) break;
          const int4 rec = sm.rec[kv][i % kRec];
          const int cnt = rec.x >> 8 & 255;
          if (!ring_wait(&sm.raw_empty[kv][raw.i], raw.phase, abort_flag)) {
            fail = true;
            break;
          }
          uint64_t *bar = &sm.raw_full[kv][raw.i];
          const uint32_t dst = sR(kv, raw.i);
          expect_tx(bar, rec.x & kKindNodes ? cnt * (2 * D) : cnt * (NG == 4 ? D + NG * 4 : D), leader);
          __syncwarp();
          if (!(rec.x & kKindNodes)) {
            const int c1 = rec.x >> 16 & 255;
            const size_t at = rec.z * nslot + rec.w, wrap = rec.z * nslot + p.c.sink_cap;
            if (leader && c1 > 0) {
              bulk_copy(dst, codes + at * D, c1 * D, bar);
              if (NG == 4) bulk_copy(dst + Y::kCodes, scales + at * NG, c1 * (NG * 4), bar);
              if (c1 < cnt) {
                bulk_copy(dst + c1 * D, codes + wrap * D, (cnt - c1) * D, bar);
                if (NG == 4) bulk_copy(dst + Y::kCodes + c1 * (NG * 4), scales + wrap * NG, (cnt - c1) * (NG * 4), bar);
              }
            }
            if constexpr (NG != 4) {
              // 8 bytes a slot: a head's first ones aligned to no more than that
#pragma unroll
              for (int k = 0; k < BN / 32; ++k) {
                const int r = lane + 32 * k;
                if (r < cnt) cp_async8(dst + Y::kCodes + r * (NG * 4), scales + (r < c1 ? at + r : wrap + (r - c1)) * NG);
              }
            }
          } else {
#pragma unroll 1
            for (int r = lane; r < cnt; r += 32) bulk_copy(dst + r * (2 * D), node_row(rec.z, rec.y + r), 2 * D, bar);
          }
          if constexpr (NG != 4) cp_async_arrive(bar);
          __syncwarp();
          raw.next();
        }
        if (noted - i <= kBatch && (!fresh || x < x1)) {
          if (fresh) {
            s = seg_at(p, x, x1);
            x += s.t1 - s.t0;
            // at least one tile, though it may hold nothing
            t = min(live_tile(pl, s, s.t0), s.t1 - 1);
            if (!kv && !s.sane && lane == 0) raise_device_error(p.err, ND_DEVERR_METADATA);
            if (kv) {  // ask for its queries
              const int hk = s.pair - s.b * p.c.n_kv_heads, r1 = min(p.n * p.G, (blk + 1) * pl.rb);
              constexpr int kLines = D * 2 / 128;
#pragma unroll 1
              for (int k = lane; k < (r1 - blk * pl.rb) * kLines; k += 32) {
                const int r = blk * pl.rb + k / kLines, nd = p.G == 1 ? r : int(__umulhi(unsigned(r), p.g_magic));
                prefetch_l2(p.q + ((int64_t(s.b) * p.n + nd) * p.Hq + hk * p.G + (r - nd * p.G)) * D + k % kLines * 64);
              }
            }
          }
          // lane j: the j-th live tile from t on
          auto nth = [&](int j) {
            int u = t + j;
            if (t < pl.ts && u >= s.ts && j > 0) u += pl.ts - max(s.ts, t + 1) ;
            if (t < pl.ts + pl.tr && u >= pl.ts + s.tr && j > 0) u += pl.tr - max(s.tr, t < pl.ts ? 0 : t + 1 - pl.ts);
            return u;
          };
          const int u = nth(lane);
          const bool mine = lane < kBatch && u < s.t1;
          const int count = __popc(__ballot_sync(0xffffffffu, mine));
          const bool end = nth(lane + 1) >= s.t1;
          if (mine) {
            int4 rec = make_int4((fresh && lane == 0 ? kFresh : 0) | (end && x >= x1 ? kLast : 0), 0, s.pair, 0);
            if (u < pl.ts + pl.tr) {
              const bool ring = u >= pl.ts;
              rec.y = (ring ? u - pl.ts : u) * BN;
              const int cnt = max(0, min(BN, (ring ? s.nv : s.sl) - rec.y));
              int c1 = cnt;
              rec.w = rec.y;
              if (ring) {
                // two pieces where it wraps
                unsigned w = unsigned(s.ring0) + unsigned(rec.y);
                if (w >= unsigned(p.c.ring_cap)) w -= unsigned(p.c.ring_cap);
                c1 = min(cnt, p.c.ring_cap - int(w));
                rec.w = p.c.sink_cap + int(w);
              }
              rec.x |= cnt << 8 | c1 << 16;
            } else {
              rec.y = (u - pl.ts - pl.tr) * kNodes;
              const int cnt = min(kNodes, p.n - rec.y);
              rec.x |= kKindNodes | cnt << 8;
#pragma unroll 1
              for (int r = 0; r < cnt; ++r) prefetch_l2(node_row(s.pair, rec.y + r));
            }
            sm.rec[kv][(noted + lane) % kRec] = rec;
          }
          noted += count;
          t = nth(count);
          fresh = t >= s.t1;
          __syncwarp();
        }
      }
    } else if (warp < kWarpFeedK) {
      // -------------------------------------------------- operands
      const int turn = warp - kWarpTurn, kv = turn & 1;
      constexpr int kTurnRows = BN / 4;
      const int row_w = (turn >> 1) * kTurnRows;  // the warp's first row
      constexpr int kPieces = D / 16, kRowsIt = 32 / kPieces, kIts = kTurnRows / kRowsIt, kU = 4;
      static_assert(kIts % kU == 0, "rows of a warp");
      // A lane takes 16 codes of a row, which become two 16-byte chunks.  K-major
      // (and for V MN-major) 128-byte swizzle: row * 128 + chunk ^ (row & 7) inside
      // a box of 64 channels.  Of eight neighbouring lanes the four in the upper
      // box (D = 128) have the other row of a pair: its swizzle differs in the
      // lowest bit, so the eight cover all chunk positions, that is all banks, at
      // once, as their 16-byte loads do.
      const int piece = lane % kPieces, box = piece / 4, c0 = (2 * piece) & 7;
      const int row_l = D == 128 ? (lane / kPieces) ^ box : lane / kPieces;
      const uint32_t codes_off = (row_w + row_l) * D + piece * 16, scale_off = Y::kCodes + 4 * ((row_w + row_l) * NG + piece / 2);
      const uint32_t operand = kv ? sV : sK;
      const uint32_t row_off = operand + (row_w + row_l) * 128 + box * (BN * 128);
      const uint32_t first_c = (c0 ^ (row_l & 7)) << 4;  // and the other chunk: ^ 16
      Ring<NR> raw;
      Ring<NK> op;
      op.phase = 1;
      int flags = 0;
#pragma unroll 1
      for (int g = 0; !(flags & kLast); ++g, raw.next(), op.next()) {
        if (!ring_wait(&sm.raw_full[kv][raw.i], raw.phase, abort_flag)) {
          fail = true;
          break;
        }
        const int4 rec = sm.rec[kv][g % kRec];
        flags = rec.x;
        const int cnt = flags >> 8 & 255;
        const uint32_t stage = sR(kv, raw.i);
        if (!(flags & kKindNodes)) {
          // the exponent of the warp's 32 keys, a lane to a key, and their scales as
          // pairs of fp16, in place: the largest scale goes to 2^14 .. 2^15
          const uint32_t at = stage + Y::kCodes + (row_w + lane) * (NG * 4);
          float y[NG], most = 0.f;
          lds_row<NG>(at, y);
          // a slot behind the last, whatever is staged, and one that is not finite count 0
          const bool held = row_w + lane < cnt;
          bool ok = held;
#pragma unroll
          for (int j = 0; j < NG; ++j) ok = ok & (fabsf(y[j]) < INFINITY);
#pragma unroll
          for (int j = 0; j < NG; ++j) {
            if (!ok) y[j] = 0.f;
            most = fmaxf(most, fabsf(y[j]));
          }
          set_if(&sm.any_bad, held & !ok);
          // (of values >= 0 the bits order as the values do)
          most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
          const int e = min(kMostUp, clamp_exp(14 - ilog2(most)));
          sts_row<NG>(at, y, pow2i(e));
          if (lane == 0) sm.e[kv][g % kInfo][turn >> 1] = e;
        }
        __syncwarp();
        if (kv && lane == 0) mbar_arrive(&sm.v_known[g & 3]);
        if (!ring_wait(&sm.op_empty[kv][op.i], op.phase, abort_flag)) {
          fail = true;
          break;
        }
        if (!(flags & kKindNodes)) {
          const uint32_t raw_at = stage + codes_off, sc_at = stage + scale_off;
          const uint32_t dst = row_off + op.i * Y::kKV;
          uint32_t ahead[kU][4], ahead_s[kU];  // the next group's loads run ahead of this one's stores
          auto load = [&](int i0) {
#pragma unroll
            for (int i = 0; i < kU; ++i) {
              ld_shared_v4(raw_at + (i0 + i) * kRowsIt * D, ahead[i][0], ahead[i][1], ahead[i][2], ahead[i][3]);
              ahead_s[i] = lds32(sc_at + (i0 + i) * kRowsIt * NG * 4);
            }
          };
          load(0);
#pragma unroll 1
          for (int i0 = 0; i0 < kIts; i0 += kU) {
            uint32_t x[kU][4], s2[kU];
#pragma unroll
            for (int i = 0; i < kU; ++i) {
#pragma unroll
              for (int j = 0; j < 4; ++j) x[i][j] = ahead[i][j] ^ 0x80808080u;
              s2[i] = ahead_s[i];
            }
            if (i0 + kU < kIts) load(i0 + kU);
#pragma unroll
            for (int i = 0; i < kU; ++i) {
              // a lane's rows are kRowsIt (4 or 8) apart: their swizzles differ in
              // one bit at most
              const uint32_t at = dst + (i0 + i) * kRowsIt * 128 + (first_c ^ ((i * kRowsIt & 4) << 4));
              const uint32_t off = hmul2(s2[i], kMinus128);
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const uint32_t wa = x[i][2 * q], wb = x[i][2 * q + 1];
                st_shared_v4(q ? at ^ 16u : at, scaled_codes(wa, kBytes01, s2[i], off), scaled_codes(wa, kBytes23, s2[i], off),
                             scaled_codes(wb, kBytes01, s2[i], off), scaled_codes(wb, kBytes23, s2[i], off));
              }
            }
          }
        } else {
          // nodes: D/8 lanes to a row, 16 of the tile's rows per warp
          constexpr int kL = D / 8, kR = 32 / kL;
          const int sub = lane / kL, ch = lane % kL, first = (turn >> 1) * 16;
          const int32_t *depth = p.depth + int64_t(rec.z / p.c.n_kv_heads) * p.n + rec.y;
          const uint32_t alive = __ballot_sync(0xffffffffu, lane < 16 && first + lane < cnt && depth[min(first + lane, cnt - 1)] >= 0);
          uint32_t bads = 0u;
          const uint32_t dst = operand + op.i * Y::kKV;
#pragma unroll 1
          for (int r0 = 0; r0 < 16; r0 += kR) {
            const int r = first + r0 + sub;
            uint32_t x[4] = {0u, 0u, 0u, 0u};
            if (alive >> (r0 + sub) & 1u) ld_shared_v4(stage + r * (2 * D) + ch * 16, x[0], x[1], x[2], x[3]);
            uint32_t m2 = 0u;  // of magnitudes the bits order as the values do, infinities and NaN above all
#pragma unroll
            for (int e = 0; e < 4; ++e) m2 = max_u16x2(m2, x[e] & 0x7fff7fffu);
            uint32_t most = max(m2 << 16, m2 & 0xffff0000u);
#pragma unroll
            for (int off = kL / 2; off >= 1; off >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
            const bool bad = most >= 0x7f800000u;
            if (!kv) {
              const int e = clamp_exp(14 - ilog2(__uint_as_float(most)));
              const float up = pow2i(e);
#pragma unroll
              for (int i = 0; i < 4; ++i) x[i] = pack_half2(bf16_lo(x[i]) * up, bf16_hi(x[i]) * up);
              if (ch == 0) sm.kf[g % kKf][r] = pow2i(-e);
            }
            if (bad) {
#pragma unroll
              for (int i = 0; i < 4; ++i) x[i] = 0u;
            }
            const uint32_t who = __ballot_sync(0xffffffffu, bad);
#pragma unroll
            for (int k = 0; k < kR; ++k) bads |= (who >> (k * kL) & 1u) << (r0 + k);
            st_shared_v4(dst + (ch / 8) * (BN * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4), x[0], x[1], x[2], x[3]);
          }
          if (lane == 0) {
            sm.bad[kv][g % kInfo][turn >> 1] = uint16_t(bads);
            if (!kv) sm.live[g % kInfo][turn >> 1] = uint16_t(alive);
          }
        }
        // the MMA reads the tile through the async proxy
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.op_full[kv][op.i]);
          mbar_arrive(&sm.raw_empty[kv][raw.i]);
        }
      }
    } else if (warp == kWarpS) {
      // -------------------------------------------------- S(g) = Q K(g)^T
      const uint32_t leader = elect_one();
      constexpr uint32_t kId = idesc_f16(BM, BN, 0), kIdNodes = idesc_f16(BM, kNodes, 0);
      Ring<NK> kr;
      Ring<2> sr;  // a buffer is free once the softmax has read it
      sr.phase = 1;
      uint32_t q_phase = 0;
      const uint64_t dk = sdesc_sw128(sK, 16, 1024);
      int flags = 0;
#pragma unroll 1
      for (int g = 0; !(flags & kLast); ++g, kr.next(), sr.next()) {
        bool ok = ring_wait(&sm.op_full[0][kr.i], kr.phase, abort_flag) &&
                  ring_wait(&sm.s_empty[sr.i], sr.phase, abort_flag);
        flags = sm.rec[0][g % kRec].x;
        if (ok && (flags & kFresh)) {
          ok = ring_wait(&sm.q_full, q_phase, abort_flag);
          q_phase ^= 1u;
        }
        if (!ok) {
          fail = true;
          break;
        }
        tc_fence_after();
        const uint64_t kd = dk + uint64_t(kr.i * (Y::kKV >> 4));
        const uint32_t id = flags & kKindNodes ? kIdNodes : kId;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)  // 16 channels = 8 TMEM columns of Q's fp16 pairs
          mma_ts(tmem + sr.i * BN, tQ + kk * 8, kd + (kk >> 2) * (BN * 128 >> 4) + (kk & 3) * 2, id, kk > 0 ? 1u : 0u, leader);
        mma_commit(&sm.s_full[sr.i], leader);
        mma_commit(&sm.op_empty[0][kr.i], leader);
      }
    } else {
      // -------------------------------------------------- O += P(g) V(g)
      // (a segment's first product overwrites O: its P exists only once the
      // softmax warps have read the segment before out of it)
      const uint32_t leader = elect_one();
      constexpr uint32_t kId = idesc_f16(BM, D, 1), kIdNodes = idesc_bf16(BM, D, 1);
      Ring<NK> vr;
      Ring<2> pr;
      const uint64_t dv = sdesc_sw128(sV, BN * 128, 1024);
      int flags = 0;
#pragma unroll 1
      for (int g = 0; !(flags & kLast); ++g, vr.next(), pr.next()) {
        if (!ring_wait(&sm.op_full[1][vr.i], vr.phase, abort_flag) || !ring_wait(&sm.p_full[pr.i], pr.phase, abort_flag)) {
          fail = true;
          break;
        }
        flags = sm.rec[1][g % kRec].x;
        tc_fence_after();
        const uint64_t vd = dv + uint64_t(vr.i * (Y::kKV >> 4));
        const uint32_t id = flags & kKindNodes ? kIdNodes : kId, more = flags & kFresh ? 0u : 1u;
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)  // (nodes: half as many keys)
          mma_ts(tO, tP + kk * 8, vd + kk * (16 * 128 >> 4), id, kk > 0 ? 1u : more,
                 kk >= kNodes / 16 && (flags & kKindNodes) ? 0u : leader);
        mma_commit(&sm.pv_done[pr.i], leader);
        mma_commit(&sm.op_empty[1][vr.i], leader);
      }
    }
  } else {
    // -------------------------------------------------- softmax warps
    regs_inc<kRegsSoftmax>();
    // A lane has two threads, one in either warpgroup: for every other tile, and
    // for half of its channels of Q and of the output.  A tile's thread gets the
    // row's maximum from the one of the tile before as soon as that has it, so
    // the two warpgroups work on neighbouring tiles side by side.
    const int wg = warp >> 2, quad = warp & 3, tl = tid & (BM - 1);
    const uint32_t lane_base = uint32_t(quad * 32) << 16;
    const int r_blk = tl & (kLanes - 1), copy = tl / kLanes;  // row of the block; which copy of it
    const int col0 = copy * kCols;
    const int R = p.n * p.G, r = blk * pl.rb + r_blk, words = (p.n + 31) / 32;
    const bool exists = r_blk < pl.rb && r < R;
    const int node = exists ? (p.G == 1 ? r : int(__umulhi(unsigned(r), p.g_magic))) : 0, head = exists ? r - node * p.G : 0;
    const uint32_t my_t = sT + warp * Y::kT1;
    // what the lane's other thread says
    auto other = [&](float x, float y) {
      float2 *half = reinterpret_cast<float2 *>(smem_raw + Y::oT);  // (what the copies send comes later)
      half[wg * BM + tl] = make_float2(x, y);
      asm volatile("bar.sync %0, 64;" ::"r"(2 + quad) : "memory");
      const float2 o = half[(wg ^ 1) * BM + tl];
      asm volatile("bar.sync %0, 64;" ::"r"(2 + quad) : "memory");
      return o;
    };
    if constexpr (REP > 1) {
      // P's columns of other copies stay 0
      uint32_t zero[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) zero[i] = 0u;
      tmem_st32(tP + lane_base + 32 * wg, zero);
      tmem_st_wait();
    }
    struct Row {
      float c;    // 2^-eq log2(e) / sqrt(D)
      int depth;
      bool dead;  // padding, or not finite
    };
    // ring entries below it are outside the row's window
    // (a dead row takes what comes and is put to 0 at the end)
    auto first_seen = [&](const Row &row, const Seg &seg) {
      return row.dead ? 0 : int(min((long long)INT_MAX, max(0ll, (long long)row.depth + seg.nv - p.window + 1)));
    };
    Ring<NK> vr;
    int g = 0, x = x0;
    bool first_seg = true;
    Seg s = {}, next = {};
    Row me = {}, next_row = {};
    float m_own = -INFINITY, l = 0.f;
    int e_o = INT_MAX;  // O holds 2^(e_o - 24) V (unset: every V so far was 0); as of this thread's last tile
    // Rounds of: the next segment's queries, so that its products start while
    // the one's before are written; the output of the one before; its tiles.
    for (int round = 0;; ++round) {
      const bool more = x < x1;
      // the products that read the Q before are done once the last S is; the other
      // warpgroup may have been the one to see it
      if (round > 0) {
        if (!fail) fail = !ring_wait(&sm.s_full[(g - 1) & 1], ((g - 1) >> 1) & 1, abort_flag);
        tc_fence_after();  // Q is overwritten behind those products' reads
      }
      if (more) {
        // ---- Q: half a row, as fp16 times 2^eq of the row (its lines were asked
        // into L2; a row per lane reads each of them eight times, from L1 but once)
        next = seg_at(p, x, x1);
        x += next.t1 - next.t0;
        const int64_t at = int64_t(next.b) * p.n + node;
        const uint4 *src = reinterpret_cast<const uint4 *>(
            p.q + (at * p.Hq + (next.pair - next.b * p.c.n_kv_heads) * p.G + head) * D + wg * (D / 2));
        uint32_t row[D / 4];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint4 w = exists ? src[i] : make_uint4(0u, 0u, 0u, 0u);
          row[4 * i] = w.x, row[4 * i + 1] = w.y, row[4 * i + 2] = w.z, row[4 * i + 3] = w.w;
        }
        next_row.depth = exists ? p.depth[at] : -1;
        uint32_t most = 0u;  // of magnitudes the bits order as the values do, infinities and NaN above all
#pragma unroll
        for (int i = 0; i < D / 4; ++i) most = max_u16x2(most, row[i] & 0x7fff7fffu);
        most = max(most << 16, most & 0xffff0000u);
        const float2 o = other(__uint_as_float(min(most, 0x7f800000u)), 0.f);
        const float qa = fmaxf(__uint_as_float(min(most, 0x7f800000u)), o.x);
        next_row.dead = !next.sane || next_row.depth < 0 || !(qa < INFINITY);
        const int eq = clamp_exp(14 - ilog2(qa));
        const float up = next_row.dead ? 0.f : pow2i(eq);
#pragma unroll
        for (int i = 0; i < D / 4; ++i) row[i] = next_row.dead ? 0u : pack_half2(bf16_lo(row[i]) * up, bf16_hi(row[i]) * up);
        next_row.c = pow2i(-eq) * (1.4426950408889634f * rsqrtf(float(D)));
        if constexpr (D == 128) tmem_st32(tQ + lane_base + 32 * wg, row);
        else tmem_st16(tQ + lane_base + 16 * wg, row);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_full);
      }
      if (round > 0) {
        // ---- the output of the segment before
        const int last = g - 1;
        if (!fail) fail = !ring_wait(&sm.pv_done[last & 1], (last >> 1) & 1, abort_flag);
        tc_fence_after();
        if (__any_sync(0xffffffffu, *(volatile int *)&sm.any_bad)) {
          // the rows that see a slot that is not finite
          const int newest = bad_slots<NG>(p.c, s.pair, min(s.sl, s.t0 * BN), min(s.sl, min(s.t1, pl.ts) * BN),
                                           min(s.nv, max(0, s.t0 - pl.ts) * BN), min(s.nv, max(0, s.t1 - pl.ts) * BN), s.ring0);
          if (newest >= first_seen(me, s)) l = __uint_as_float(0x7fffffffu);
        }
        const float2 o = other(m_own, l);
        const float m_used = me.dead ? -INFINITY : fmaxf(m_own, o.x);
        // (a half that saw nothing has l = 0)
        l = (l == 0.f ? 0.f : l * ex2(m_own - m_used)) + (o.y == 0.f ? 0.f : o.y * ex2(o.x - m_used));
        if (me.dead) l = 0.f;
        fail = softmax_any(fail);  // (the barriers below want all their warps)
        const int h = (s.pair - s.b * p.c.n_kv_heads) * p.G + head;
        // (e_o only falls)
        const float2 o_e = other(e_o == INT_MAX ? 0.f : 1.f, float(e_o == INT_MAX ? kCodeBits : e_o));
        if (o_e.x != 0.f) e_o = e_o == INT_MAX ? int(o_e.y) : min(e_o, int(o_e.y));
        const float down = e_o == INT_MAX ? pow2i(-kCodeBits) : pow2i(-e_o);
        if (s.all) {
          // copies merge: the row's weight of each, then the sum through shared memory
          float m_all = m_used, l_all = l, scale;
          if constexpr (REP > 1) {
            if (wg == 0) sm.ml[tl] = make_float2(m_used, l);
            asm volatile("bar.sync 1, 256;" ::: "memory");
            m_all = -INFINITY;
#pragma unroll
            for (int c = 0; c < REP; ++c) m_all = fmaxf(m_all, sm.ml[c * kLanes + r_blk].x);
            l_all = 0.f;
#pragma unroll
            for (int c = 0; c < REP; ++c) {
              const float2 part = sm.ml[c * kLanes + r_blk];
              l_all += part.x == -INFINITY && part.y == 0.f ? 0.f : part.y * ex2(part.x - m_all);
            }
            scale = m_used == -INFINITY && l == 0.f ? 0.f : (l_all != 0.f ? ex2(m_used - m_all) * kUnits * down / l_all : 0.f);
          } else {
            scale = l != 0.f ? kUnits * down / l : 0.f;
          }
          uint16_t *dst = p.out + ((int64_t(s.b) * p.n + node) * p.Hq + h) * D + wg * (D / 2);
          // every copy finishes its part of the half row's channels, kC at a time,
          // with what the others send it
          constexpr int kPart = D / 2 / REP, kC = kPart < 16 ? kPart : 16;
          auto send_at = [&](int chunk) { return uint32_t(lane * 64 + ((chunk ^ (lane >> 1 & 3)) << 4)); };
          const uint32_t tO_half = tO + lane_base + wg * (D / 2);
#pragma unroll 1
          for (int ch = 0; ch < kPart; ch += kC) {
            float sum[kC];
#pragma unroll
            for (int i = 0; i < kC; ++i) sum[i] = 0.f;
#pragma unroll 1
            for (int k = 0; k < REP; ++k) {
              // send copy + k's channels of this round, take the own ones from copy - k
              uint32_t ov[kC];
              const int to = ((copy + k) & (REP - 1)) * kPart + ch;
              if constexpr (kC == 16) tmem_ld16(tO_half + to, ov);
              else tmem_ld8(tO_half + to, ov);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < kC; ++i) ov[i] = scale != 0.f ? __float_as_uint(__uint_as_float(ov[i]) * scale) : 0u;
              if (REP > 1 && k > 0) {
#pragma unroll
                for (int i = 0; i < kC; i += 4) st_shared_v4(my_t + send_at(i / 4), ov[i], ov[i + 1], ov[i + 2], ov[i + 3]);
                asm volatile("bar.sync %0, 128;" ::"r"(6 + wg) : "memory");
                const int from = (copy - k) & (REP - 1);
                const uint32_t at = sT + (wg * 4 + (from * kLanes + r_blk) / 32) * Y::kT1;
#pragma unroll
                for (int i = 0; i < kC; i += 4) ld_shared_v4(at + send_at(i / 4), ov[i], ov[i + 1], ov[i + 2], ov[i + 3]);
                asm volatile("bar.sync %0, 128;" ::"r"(6 + wg) : "memory");
              }
#pragma unroll
              for (int i = 0; i < kC; ++i) sum[i] += __uint_as_float(ov[i]);
            }
            if (exists && !fail) {
#pragma unroll
              for (int i = 0; i < kC; i += 8)
                st_global_v4(dst + copy * kPart + ch + i, pack_bf16x2(sum[i], sum[i + 1]), pack_bf16x2(sum[i + 2], sum[i + 3]),
                             pack_bf16x2(sum[i + 4], sum[i + 5]), pack_bf16x2(sum[i + 6], sum[i + 7]));
            }
          }
          if (wg == 0 && copy == 0 && exists && p.lse && !fail)
            p.lse[(int64_t(s.b) * p.Hq + h) * p.n + node] =
                l_all != 0.f ? 0.6931471805599453f * (m_all - kPBias + log2f(l_all)) : -INFINITY;
        } else if (!fail) {
          float *part = p.parts + (size_t(blockIdx.x) * 2 + (first_seg ? 0 : 1)) * part_floats<D>();
          const float by = kUnits * down;  // (first: O times 2^24 may be too large)
#pragma unroll 1
          for (int ch = wg * (D / 2); ch < (wg + 1) * (D / 2); ch += 16) {
            uint32_t ov[16];
            tmem_ld16(tO + lane_base + ch, ov);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<float4 *>(part + ((ch + i) / 4 * BM + tl) * 4) =
                  make_float4(__uint_as_float(ov[i]) * by, __uint_as_float(ov[i + 1]) * by,
                              __uint_as_float(ov[i + 2]) * by, __uint_as_float(ov[i + 3]) * by);
          }
          if (wg == 0) *reinterpret_cast<float2 *>(part + BM * D + 2 * tl) = make_float2(m_used, l);
        }
        tc_fence_before();
        // (no P of the next segment before all of this one's O has been read)
        asm volatile("bar.sync 1, 256;" ::: "memory");
        first_seg = false;
      }
      if (!more || fail) break;
      s = next;
      me = next_row;
      const bool dead = me.dead;
      const uint32_t *mask_row = p.mask + (int64_t(s.b) * p.n + node) * words;
      const int low = first_seen(me, s);
      m_own = -INFINITY, l = 0.f, e_o = INT_MAX;
      const int first_t = min(live_tile(pl, s, s.t0), s.t1 - 1);
      // a tile of cached keys, all of them seen by the warp's rows (0) or not (1), or of
      // nodes (2).  With 128 columns to a thread most tiles are of kind 0, which has
      // code of its own, the shortest (303 to 275 us at 8 sessions of 64 nodes); with
      // fewer, of short caches, one code for both is better (129 against 137 at 128 of
      // 16).
      auto tile = [&](auto kind, int t, bool last) {
        constexpr bool kN = decltype(kind)::value == 2, kMasked = decltype(kind)::value == 1;
        constexpr int kC = kCols < 64 ? kCols : 64;  // columns at a time
        const int u = g & 1;
        // what V's warps say of a node tile (K's were done before S)
        if (kN && !fail) fail = !ring_wait(&sm.op_full[1][vr.i], vr.phase, abort_flag);
        tc_fence_after();
        const uint32_t tS = tmem + u * BN + lane_base;
        uint32_t v[kC];
        // scores of columns col .. col + kC, -inf where the row does not see
        auto load = [&](int col) {
#pragma unroll
          for (int i = 0; i < kC; i += 32) tmem_ld32(tS + col + i, v + i);
          tmem_ld_wait();
          if constexpr (kMasked) {
            const bool ring = t >= pl.ts;
            const int first = (ring ? t - pl.ts : t) * BN + col;
            const int hi = (ring ? s.nv : s.sl) - first;
            const int lo = ring ? max(low, first) - first : 0;
            if (__any_sync(0xffffffffu, lo > 0 || hi < kC)) {
#pragma unroll
              for (int i = 0; i < kC; ++i) v[i] = i >= lo && i < hi ? v[i] : 0xff800000u;
            }
          } else if constexpr (kN) {
            // (64 columns: those behind them are not of this tile)
#pragma unroll
            for (int i = 0; i < kC; i += 32) {
              const int wd = (t - pl.ts - pl.tr) * 2 + (col + i) / 32, at = (col + i) & (kNodes - 1);
              uint32_t see = 0u, bad = 0u;
              if (!dead && col < kNodes && wd < words) {
                auto word = [&](const uint16_t *h) { return uint32_t(h[at / 16]) | uint32_t(h[at / 16 + 1]) << 16; };
                see = mask_row[wd] & word(sm.live[g % kInfo]);
                bad = word(sm.bad[0][g % kInfo]) | word(sm.bad[1][g % kInfo]);
              }
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float sc = __uint_as_float(v[i + e]) * sm.kf[g % kKf][at + e];
                v[i + e] = see >> e & 1u ? (bad >> e & 1u ? 0x7fffffffu : __float_as_uint(sc)) : 0xff800000u;
              }
            }
          }
        };
        // a score's factor, by 32 keys (nodes: all the same, and with 2^-e in the
        // scores); never 0, which would make NaN of a masked column's -inf: |S| <
        // 2^37, so at 2^-126 and below a score is 2^-89 at most and its weight 1 to
        // every bit
        auto factor = [&](int col) {
          return kN ? fmaxf(me.c, 1.1754943508222875e-38f)
                    : fmaxf(me.c * pow2i(-sm.e[0][g % kInfo][col / 32]) * kUnits, 1.1754943508222875e-38f);
        };
        float mx = -INFINITY;
#pragma unroll 1
        for (int col = col0; col < col0 + kCols; col += kC) {
          load(col);
#pragma unroll
          for (int h = 0; h < kC; h += 32) {
            float mxp[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mxp[i] = max3(__uint_as_float(v[h + i]), __uint_as_float(v[h + 4 + i]), __uint_as_float(v[h + 8 + i]));
#pragma unroll
            for (int j = 12; j < 28; j += 8)
#pragma unroll
              for (int i = 0; i < 4; ++i) mxp[i] = max3(mxp[i], __uint_as_float(v[h + j + i]), __uint_as_float(v[h + j + 4 + i]));
#pragma unroll
            for (int i = 0; i < 4; ++i) mxp[i] = fmaxf(mxp[i], __uint_as_float(v[h + 28 + i]));
            mx = fmaxf(mx, factor(col + h) * max3(mxp[0], mxp[1], fmaxf(mxp[2], mxp[3])));
          }
        }
        float m_used = -INFINITY, alpha = 1.f;
        if (t != first_t) {
          asm volatile("bar.sync %0, 64;" ::"r"(8 + 4 * wg + quad) : "memory");
          m_used = sm.m[u ^ 1][tl];
        }
        if (mx > m_used + kLazyLog2) {  // the first tile with a key included
          alpha = ex2(m_used - mx);     // 0 at the first
          m_used = mx;
        }
        if (!last) {
          sm.m[u][tl] = m_used;
          asm volatile("bar.arrive %0, 64;" ::"r"(8 + 4 * (wg ^ 1) + quad) : "memory");
        }
        if (m_own != m_used) {
          l *= ex2(m_own - m_used);  // (0 * 0 at the first)
          m_own = m_used;
        }
        // the power of two that O holds V in: it falls where a tile's values are
        // larger than those before, and with it O.  (V's warps know tiles in order,
        // so the tile before, the other warpgroup's, is known too.)
        if (!fail) fail = !ring_wait(&sm.v_known[g & 3], (g >> 2) & 1, abort_flag);
        auto e_of = [&](int tile) {
          const int4 e = *reinterpret_cast<const int4 *>(sm.e[1][tile % kInfo]);
          return min(min(e.x, e.y), min(e.z, e.w));
        };
        if (t != first_t) {
          if (!kN || t == pl.ts + pl.tr) e_o = min(e_o, e_of(g - 1));
          else if (e_o == INT_MAX) e_o = kCodeBits;  // (nodes alone so far)
        }
        const int e_now = kN ? (e_o == INT_MAX ? kCodeBits : e_o) : min(e_o, e_of(g));
        if (e_now < e_o && e_o != INT_MAX) alpha *= pow2i(max(e_now - e_o, -126));
        e_o = e_now;
        const float base_shift = kPBias - (m_used == -INFINITY ? 0.f : m_used);
        // P and O may change once the PV before has landed
        auto pv_before = [&]() {
          if (!fail) fail = !ring_wait(&sm.pv_done[u ^ 1], ((g - 1) >> 1) & 1, abort_flag);
          tc_fence_after();
        };
#pragma unroll
        for (int col = col0; col < col0 + kCols; col += kC) {
          if (REP == 1) load(col);
#pragma unroll
          for (int h = 0; h < kC; h += 32) {
            // weights carry what V's operand lacks of O's scale, never more than 1 for
            // codes: fp16 keeps them to 2^(-32-up) of the row's largest.  Below 2^-60
            // none is left of them (fp16 ends at 2^-25 of what is at most 2^15)
            const int up = kN ? e_now - kCodeBits : max(e_now - sm.e[1][g % kInfo][(col + h) / 32], -60);
            const float ct = factor(col + h), shift = base_shift + float(up);
            const uint64_t c2 = pack_f32x2(ct, ct), nmc2 = pack_f32x2(shift, shift);
            float rsp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = h; i < h + 32; i += 2) {
              float a, b;
              fma_f32x2(a, b, __uint_as_float(v[i]), __uint_as_float(v[i + 1]), c2, nmc2);
              a = ex2(a);
              b = ex2(b);
              add_f32x2(rsp[(i >> 1) & 1 ? 2 : 0], rsp[(i >> 1) & 1 ? 3 : 1], a, b);
              v[i / 2] = kN ? pack_bf16x2(a, b) : pack_half2(a, b);
            }
            const float sum = (rsp[0] + rsp[1]) + (rsp[2] + rsp[3]);
            l += kN ? sum * pow2i(-e_now) * kUnits : sum * pow2i(-up);
          }
          if (col + kC == col0 + kCols) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.s_empty[u]);
          }
          if (col == col0 && t != first_t) pv_before();
          if constexpr (kC == 64) tmem_st32(tP + lane_base + col / 2, v);
          else tmem_st16(tP + lane_base + col / 2, v);
        }
        if (t != first_t && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
          for (int ch = 0; ch < D; ch += 16) {
            uint32_t ov[16];
            tmem_ld16(tO + lane_base + ch, ov);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tmem_st16(tO + lane_base + ch, ov);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[u]);
      };
      // (which tiles, the warps know by themselves: after a wait that gave up they
      // still meet at the same barriers)
#pragma unroll 1
      for (int t = first_t; t < s.t1; ++g, vr.next()) {
        const int t_next = live_tile(pl, s, t + 1);
        if ((g & 1) == wg) {
          if (!fail) fail = !ring_wait(&sm.s_full[g & 1], (g >> 1) & 1, abort_flag);
          const bool ring = t >= pl.ts;
          const int first = (ring ? t - pl.ts : t) * BN + col0;
          if (t >= pl.ts + pl.tr) {
            tile(std::integral_constant<int, 2>{}, t, t_next >= s.t1);
          } else if (REP > 1 || __any_sync(0xffffffffu, (ring ? s.nv : s.sl) - first < kCols || (ring && low > first))) {
            tile(std::integral_constant<int, 1>{}, t, t_next >= s.t1);
          } else {
            if constexpr (REP == 1) tile(std::integral_constant<int, 0>{}, t, t_next >= s.t1);
          }
        }
        t = t_next;
      }
    }
  }

  // ---- common exit: on the error path give copies and MMAs still in flight a
  //      bounded time (about 2 ms) to land before shared memory and TMEM go
  tc_fence_before();
  if (__syncthreads_or(fail || *abort_flag)) {
    if (tid == 0) raise_device_error(p.err, ND_DEVERR_TIMEOUT);
#pragma unroll 1
    for (int i = 0; i < 2000; ++i) __nanosleep(1000);
  }
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
  // the i-th triple: stretch by stretch, copy by copy; four loads in flight
  const int total = (c1 - c0 + 1) * copies, low = p.lanes == 32 ? 2 : p.lanes == 64 ? 1 : 0;
  const bool later = pl.start(c0) < pair * pl.t;  // the pair is not the first of its first stretch
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int i0 = 0; i0 < total; i0 += 4) {
    float2 ml[4];
    float4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = min(i0 + j, total - 1), c = c0 + (i >> low), at = (i & (copies - 1)) * p.lanes + r_blk;
      const float *src = p.parts + ((size_t(c) * pl.nb + blk) * 2 + (c == c0 && later ? 1 : 0)) * part_floats<D>();
      ml[j] = *reinterpret_cast<const float2 *>(src + BM * D + 2 * at);
      v[j] = *reinterpret_cast<const float4 *>(src + (quad * BM + at) * 4);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (i0 + j >= total || (ml[j].x == -INFINITY && ml[j].y == 0.f)) continue;  // (saw nothing)
      const float mn = fmaxf(m, ml[j].x), a = mn == -INFINITY ? 0.f : ex2(m - mn), b = mn == -INFINITY ? 1.f : ex2(ml[j].x - mn);
      m = mn;
      l = l * a + ml[j].y * b;
      o = make_float4(o.x * a + v[j].x * b, o.y * a + v[j].y * b, o.z * a + v[j].z * b, o.w * a + v[j].w * b);
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
