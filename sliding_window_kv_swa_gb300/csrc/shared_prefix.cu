// shared_prefix.cu -- the shared part of a decode step whose sequences have one
// pinned prefix in common: every query of the batch against the prefix's int8
// keys and values, on the 5th-generation tensor cores.
//
// Mathematics.  A KV head's rows are the R = batch * G queries that read it
// (row r: sequence r / G, head of the group r % G).  With the prefix's keys
// k_j = code_j * scale_j the row's part of the softmax is the triple
//   m = max_j s_j,  l = sum_j 2^(s_j - m),  O = sum_j 2^(s_j - m) v_j,
//   s_j = (q . k_j) log2(e) / sqrt(D),
// taken in one pass over the keys; triples of different key ranges, and of the
// sequence's own slots, merge exactly (shared_decode.cu).
//
// Types.  The tensor cores multiply fp16 with fp32 sums.  q (bf16) becomes
// fp16 exactly after a power-of-two scaling per row (channels 2^-28 below the
// row's largest lose bits).  Keys and values are code * fp16(scale * 2^e),
// rounded to fp16: at most 2^-11 + 2^-11 of the value, an eighth of what bf16
// operands would cost.  e is chosen per 64-key tile for K (its inverse is one
// factor of the tile's scores) and follows the largest value scale seen for V,
// with 4 bits of headroom, so that O is rescaled for it only where scales grow
// by more than 2^3.  Far below the largest the operands are subnormal and off
// by 2^-25 in place of 2^-11 of themselves: with the tile's largest key scale
// in [2^7, 2^8), 127 * 2^-25 of a code's scale and 2^-25 of the product are
// below 2^-31 of the tile's largest key; with the largest value scale at 2^4
// or more, below 2^-28 of the largest value, under what an fp32 sum that holds
// both can tell apart.  P is fp16 with the running maximum up to 2^8 behind and
// all of it scaled by 2^7, so it stays below 2^15 and keys 2^-21 below the
// maximum still have all bits.  Sums, maxima and partials are fp32.
//
// What bounds it.  4 R D flops per key and KV head on the tensor cores, or
// below about 40 rows per KV head the read of the codes (2 (D + D/8) bytes per
// key); a CTA keeps two 128-row blocks and turns a tile's codes into fp16 once
// for both.  Measured (ncu, D = 128): 512 rows over 32768 keys of 8 heads 58
// us, the products' pipe 72 % active: S = Q K^T of 128 x 64 reads Q from shared
// memory for every tile and runs at half the rate (N = 128 would not, but the
// scores of two blocks and O are all of one CTA's TMEM with no second buffer;
// two CTAs with a block each would have the room, which has not been tried).
// 16 rows
// over 65536 keys: 42 us for 151 MB, 22 us of it the bytes; a tile costs 0.55
// us of the chain copy - scales - turn - S - softmax - PV, in which no role is
// busy for much more than half of it (Q from TMEM, other waits, deeper rings:
// no change), and 6 us go before the first product.
//
// Work split.  The (KV head, 256-row pair, 64-key tile) triples, key tiles
// fastest, form one line that is cut into equal stretches, one per CTA (one
// CTA per SM): the line's length comes from the prefix's sink_len on the
// device.  A stretch is one or more segments (a run of tiles of one row pair);
// each segment writes its rows' triples to its own slot, CTA + row pair, which
// both sides compute.
//
// Roles (16 warps):
//   warps 0-3, 4-7 : softmax of row block 0, 1 (thread = row = TMEM lane):
//                    stage Q; per tile read S, write P over it; at a segment's
//                    end read O and write the partials
//                    (fewer rows: see Mode)
//   warps 8-9, 10-11 : codes of the staged tile -> fp16 K, V operands in shared
//                    memory
//   warp 12        : copies codes (bulk) and scales of the tiles ahead
//   warp 15        : the staged tile's scales -> its exponents, fp16 scales
//   warps 13, 14   : MMA issuers: S(g) = Q K(g)^T; O += P(g) V(g).  (One issuer
//                    per block for both had to go through every wait of a tile
//                    one after the other, 1100 cycles with all of them met.)
// Every wait is bounded: one that gives up raises the device error flag and
// the abort flag, and all roles leave through the common exit.
#include <atomic>
#include <climits>

#include "nd_common.cuh"
#include "nd_internal.h"
#include "shared_prefix.cuh"
#include "tc_ptx.cuh"

namespace nd {

namespace {

constexpr int BM = kPrefixBlock;   // rows per block = TMEM lanes
constexpr int BN = kPrefixTile;    // keys per tile
constexpr int kThreads = 16 * 32;
constexpr int kWarpDeq0 = 8, kWarpLoad = 12, kWarpS = 13, kWarpPV = 14, kWarpScan = 15;
// Register split (setmaxnreg, per warpgroup) of the 128 a thread at launch:
// the softmax holds a 64-score row per thread.  (Four more warps for the
// conversion, on alternate tiles, measured slower -- 63 against 60 us at 4
// sequences over 65536 slots -- their share of the registers made the softmax
// spill.)
constexpr int kRegsSoftmax = 168, kRegsOther = 88;
static_assert(2 * 128 * kRegsSoftmax + 2 * 128 * kRegsOther == kThreads * 128, "register split");
constexpr float kLazyLog2 = 8.f;   // the maximum used may lag the true one by 2^8
constexpr float kPBias = 7.f;      // P is scaled by 2^7
constexpr int kInfo = 16;          // tile records in flight

// What a CTA's two softmax warpgroups hold:
//   kPair    two row blocks (more than 128 rows)
//   kSingle  one row block; the other warpgroup turns codes
//   kStreams one half block (up to 64 rows) twice: the warpgroups take every
//            other key tile each, with sums and an O of their own, so a tile
//            has two tiles' time for the latencies of its softmax, which
//            bound a single warp; the four idle warps turn codes
enum Mode { kPair, kSingle, kStreams };

template <int D, Mode M>
struct Lay {
  static constexpr int NB = M == kSingle ? 1 : 2;       // S and O sets
  static constexpr int NG = D / 32;
  static constexpr int kBoxes = D / 64;
  // Q, fp16: rows staged per set, and from one 64-channel box to the next.  (A
  // half block's MMA also reads the rows behind it, whatever they are, into
  // rows of S that nobody reads.)
  static constexpr int kQRows = M == kStreams ? 64 : BM;
  static constexpr int kQBox = kQRows * 128, kQ = kBoxes * kQBox;
  static constexpr int kKV = kBoxes * BN * 128;         // one K or V operand tile, fp16
  static constexpr int kCodes = BN * D, kScales = BN * NG * 4;
  static constexpr int kRaw = 2 * kCodes + 2 * kScales; // K codes, V codes, K scales, V scales
  static constexpr int NK = D == 128 && M == kPair ? 2 : 3, NV = 3, NR = D == 64 ? 6 : (M == kPair ? 4 : 5);
  static constexpr int oQ = 0, oK = NB * kQ, oV = oK + NK * kKV, oR = oV + NV * kKV;
  static constexpr int kBytes = oR + NR * kRaw + 1024;  // + alignment slack
  static_assert(kBytes <= 227 * 1024, "shared memory");
  static constexpr int NS = D == 64 ? 3 : 2;            // S buffers per set
  static constexpr int cO = 2 * NS * BN;                // TMEM columns: S[2][NS], O[2]
  static constexpr int kTmemCols = 512;
  static_assert(cO + 2 * D <= kTmemCols, "TMEM");
  static constexpr int kSoft = M == kStreams ? 2 : 4;   // softmax warps per set
  static constexpr int kTurn = M == kPair ? 2 : 4;      // warps that turn K, and V
};

struct PrefixParams {
  const uint16_t *q;
  nd_kv_cache c;     // the prefix: one row, its sink region
  int Hq, G, R;
  unsigned g_magic;  // ceil(2^32 / G): r / G for G >= 2 and r < 2^24
  PrefixParts out;
  int *err;
};

// exponent of the power of two at or below x (x >= 0; 0, subnormals and
// non-finite values included)
__device__ __forceinline__ int ilog2(float x) {
  return int((__float_as_uint(x) >> 23) & 0xffu) - 127;
}
__device__ __forceinline__ float pow2i(int e) {  // e in [-126, 127]
  return __uint_as_float(uint32_t(e + 127) << 23);
}
__device__ __forceinline__ int clamp_exp(int e) { return max(-120, min(120, e)); }

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar, uint32_t leader) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %4, 0;\n"
      " @e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar)), "r"(leader)
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

// A position in a ring of N stages and the parity of its current use (counters
// instead of divisions: every role's loop has to stay small, see the head of
// this file).
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

// A bounded wait of a whole warp that sleeps between polls (up to 2 us each):
// the polls of those that wait take issue slots from those
// that work (80 -> 70 us for 4 sequences over 65536 slots).
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

template <int D, Mode M>
__global__ void __launch_bounds__(kThreads, 1) shared_prefix_kernel(const __grid_constant__ PrefixParams p) {
  using Y = Lay<D, M>;
  constexpr int NB = Y::NB, kTurn = Y::kTurn, kTurnRows = BN / kTurn;
  constexpr int NK = Y::NK, NV = Y::NV, NR = Y::NR, NS = Y::NS, NG = Y::NG;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t raw_full[NR], raw_empty[NR], scan_full[NR], k_full[NK], k_empty[NK], v_full[NV], v_empty[NV],
      s_full[2][NS], p_full[2][NS], pv_done[2][NS], q_full[2];
  __shared__ float4 s_info[kInfo];  // per tile, for the softmax
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the same in the warp
  volatile int *abort_flag = &s_abort;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  auto sQ = [&](int rb) { return base + Y::oQ + rb * Y::kQ; };
  auto sK = [&](int st) { return base + Y::oK + st * Y::kKV; };
  auto sV = [&](int st) { return base + Y::oV + st * Y::kKV; };
  auto sR = [&](int st) { return base + Y::oR + st * Y::kRaw; };

  if (tid == 0) {
    for (int s = 0; s < NR; ++s) {
      mbar_init(&raw_full[s], 33);          // the bulk copies' transaction and 32 lanes' scale copies
      mbar_init(&raw_empty[s], 2 * kTurn + 1);  // the warps that turn the tile, and the scan
      mbar_init(&scan_full[s], 1);
    }
    for (int s = 0; s < NK; ++s) {
      mbar_init(&k_full[s], kTurn);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(&v_full[s], kTurn);
      mbar_init(&v_empty[s], 1);
    }
    for (int r = 0; r < 2; ++r) {
      for (int u = 0; u < NS; ++u) {
        mbar_init(&s_full[r][u], 1);
        mbar_init(&p_full[r][u], Y::kSoft);
        mbar_init(&pv_done[r][u], 1);
      }
      mbar_init(&q_full[r], Y::kSoft);
    }
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
  pdl_trigger();  // the own part reads nothing of this kernel's before it waits
  auto tS = [&](int rb, int buf) { return tmem + (NS * rb + buf) * BN; };
  auto tO = [&](int rb) { return tmem + Y::cO + rb * D; };

  // ---- this CTA's stretch of the line of tiles
  const PrefixPlan pl = prefix_plan(p.c.sink_len[0], p.c.sink_cap, p.c.n_kv_heads, p.R, gridDim.x);
  if (!pl.sane && blockIdx.x == 0 && tid == 0) raise_device_error(p.err, ND_DEVERR_METADATA);
  const bool has_work = int(blockIdx.x) < pl.ctas;
  const int x0 = has_work ? pl.start(blockIdx.x) : 0, x1 = has_work ? pl.start(blockIdx.x + 1) : 0;
  struct Seg {
    int item, t0, n, hk, r0, nb;  // nb: sets at work
  };
  auto seg_at = [&](int x) {
    Seg s;
    s.item = x / pl.nt;
    s.t0 = x - s.item * pl.nt;
    s.n = min(pl.nt - s.t0, x1 - x);
    s.hk = s.item / pl.pairs;
    s.r0 = M == kPair ? (s.item % pl.pairs) * 2 * BM : 0;
    s.nb = M == kSingle ? 1 : M == kStreams ? min(s.n, 2) : p.R - s.r0 > BM ? 2 : 1;
    return s;
  };
  bool fail = false;

  const bool soft = warp < 4 * NB && (warp & 3) < Y::kSoft;
  if (warp < 4 * NB) regs_inc<kRegsSoftmax>();
  else regs_dec<kRegsOther>();
  if (!soft) {
    if (warp == kWarpLoad) {
      // ------------------------------------------------ loader
      const uint32_t leader = elect_one();
      const size_t nslot = size_t(p.c.sink_cap) + p.c.ring_cap;
      Ring<NR> raw;
      raw.phase = 1;  // the first round of an empty ring does not wait
      for (int x = x0; x < x1 && !fail;) {
        const Seg s = seg_at(x);
        const size_t slot0 = s.hk * nslot + size_t(s.t0) * BN;
        const int8_t *kc = p.c.k_codes + slot0 * D, *vc = p.c.v_codes + slot0 * D;
        // scales: a slot's row is 16 (D = 128) or 8 bytes, and a head's first
        // one aligned to no more than that
        const float *ks = p.c.k_scale + (slot0 + lane) * NG, *vs = p.c.v_scale + (slot0 + lane) * NG;
        int left = pl.len - s.t0 * BN;
#pragma unroll 1
        for (int j = 0; j < s.n; ++j, raw.next(), left -= BN) {
          if (!ring_wait(&raw_empty[raw.i], raw.phase, p.err, abort_flag)) {
            fail = true;
            break;
          }
          uint64_t *bar = &raw_full[raw.i];
          const uint32_t dst = sR(raw.i), bytes = min(BN, left) * D;
          expect_tx(bar, 2 * bytes, leader);
          bulk_load(dst, kc, bytes, bar, leader);
          bulk_load(dst + Y::kCodes, vc, bytes, bar, leader);
          const uint32_t sd = dst + 2 * Y::kCodes + lane * (NG * 4);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (lane + 32 * i < left) {
              if constexpr (NG == 4) {
                cp_async16(sd + i * 32 * NG * 4, ks + i * 32 * NG);
                cp_async16(sd + i * 32 * NG * 4 + Y::kScales, vs + i * 32 * NG);
              } else {
                cp_async8(sd + i * 32 * NG * 4, ks + i * 32 * NG);
                cp_async8(sd + i * 32 * NG * 4 + Y::kScales, vs + i * 32 * NG);
              }
            }
          cp_async_arrive(bar);
          __syncwarp();
          kc += BN * D, vc += BN * D, ks += BN * NG, vs += BN * NG;
        }
        x += s.n;
      }
    } else if (warp < kWarpLoad) {
      // ------------------------------------------------ codes -> fp16 operands
      // half of the warps turn K, half V, so that neither operand waits behind
      // the other's stages
      // (warps 8-11; with one block also 4-7, with two streams 2, 3, 6 and 7)
      const int turn = M == kStreams ? (warp < kWarpDeq0 ? (warp & 1) + (warp >> 2) * 2 : warp - 4)
                                     : warp - (M == kSingle ? 4 : kWarpDeq0);
      const int row_w = (turn >> 1) * kTurnRows;  // the warp's first row
      const bool is_v = turn & 1;
      constexpr int kPieces = D / 16, kRowsIt = 32 / kPieces, kIts = kTurnRows / kRowsIt, kU = 2;
      static_assert(kIts % kU == 0, "rows of a warp");
      const int piece = lane % kPieces, row_l = lane / kPieces;
      // K-major (and for V MN-major) 128-byte swizzle: row * 128 + 16-byte
      // chunk ^ (row & 7) inside a box of 64 channels; a lane's two chunks.
      // The upper box's lanes store their odd chunk first, so the eight lanes
      // of a row cover the eight chunk positions (all banks) at once.
      const int box = piece / 4, c0 = (2 * piece) & 7;
      const uint32_t odd_first = box == 1 ? 1u : 0u;
      uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
      const int n_st = is_v ? NV : NK;
      const uint32_t codes_off = (is_v ? Y::kCodes : 0) + (row_w + row_l) * D + piece * 16 + 8 * odd_first;
      const uint32_t scale_off = 2 * Y::kCodes + (is_v ? Y::kScales : 0) + 4 * ((row_w + row_l) * NG + piece / 2);
      const uint32_t row_off = (is_v ? sV(0) : sK(0)) + (row_w + row_l) * 128 + box * (BN * 128);
      // a lane's rows are kRowsIt (4 or 8) apart: the swizzle of the second of
      // a pair differs from the first's in one bit at most
      const uint32_t first_c = ((c0 + odd_first) ^ (row_l & 7)) << 4;  // and the other chunk: ^ 16
      Ring<NR> raw;
      int so = 0;
      uint32_t so_phase = 1;
      for (int x = x0; x < x1 && !fail;) {
        const Seg s = seg_at(x);
#pragma unroll 1
        for (int j = 0; j < s.n; ++j, raw.next()) {
          // the scan waited for the tile's copies before it arrived
          if (!ring_wait(&scan_full[raw.i], raw.phase, p.err, abort_flag) ||
              !ring_wait(&empty[so], so_phase, p.err, abort_flag)) {
            fail = true;
            break;
          }
          const uint32_t raw_at = sR(raw.i) + codes_off, sc_at = sR(raw.i) + scale_off;
          const uint32_t dst = row_off + so * Y::kKV;
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
              const uint32_t at = dst + (i0 + i) * kRowsIt * 128 + (first_c ^ ((i * kRowsIt & 4) << 4));
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const uint32_t wa = w[i][q].x ^ 0x80808080u, wb = w[i][q].y ^ 0x80808080u;
                st_shared_v4(q ? at ^ 16u : at, hmul2(codes_to_half2(wa, kSelBytes01), s2[i]),
                             hmul2(codes_to_half2(wa, kSelBytes23), s2[i]),
                             hmul2(codes_to_half2(wb, kSelBytes01), s2[i]),
                             hmul2(codes_to_half2(wb, kSelBytes23), s2[i]));
              }
            }
          }
          // the MMA reads the tile through the async proxy
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&full[so]);
            mbar_arrive(&raw_empty[raw.i]);
          }
          if (++so == n_st) {
            so = 0;
            so_phase ^= 1u;
          }
        }
        x += s.n;
      }
    } else if (warp == kWarpScan) {
      // ------------------------------------------------ scales' exponents
      // ahead of the conversion: a tile's largest scales fix the powers of
      // two that its keys and values are taken with, and the scales become the
      // fp16 pairs that multiply the codes, in place
      Ring<NR> raw;
      int g = 0;
      for (int x = x0; x < x1 && !fail;) {
        const Seg s = seg_at(x);
        int e_v = INT_MAX;  // the exponent that V's operands have in O (unset)
        int left = pl.len - s.t0 * BN;
#pragma unroll 1
        for (int j = 0; j < s.n; ++j, ++g, raw.next(), left -= BN) {
          const int st = raw.i;
          if (!ring_wait(&raw_full[st], raw.phase, p.err, abort_flag)) {
            fail = true;
            break;
          }
          const uint32_t rks = sR(st) + 2 * Y::kCodes, rvs = rks + Y::kScales;
          constexpr int kPer = BN * NG / 32;
          float ksc[kPer], vsc[kPer], km = 0.f, vm = 0.f;
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int idx = lane + 32 * i;
            // a slot behind the prefix: whatever is staged counts 0
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
          float fix = 1.f;
          if (vm > 0.f) {
            const int want = clamp_exp(4 - ilog2(vm));
            if (e_v == INT_MAX) {
              e_v = want;  // every value so far was 0, and so is O
            } else if (want + 3 < e_v) {
              fix = pow2i(max(want - e_v, -126));
              e_v = want;
            }
          }
          const float up_k = pow2i(e_k), up_v = e_v == INT_MAX ? 1.f : pow2i(e_v);
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int idx = lane + 32 * i;
            const float a = ksc[i] * up_k, b = vsc[i] * up_v;
            sts32(rks + 4 * idx, pack_half2(a, a));
            sts32(rvs + 4 * idx, pack_half2(b, b));
          }
          __syncwarp();
          if (lane == 0) {
            // 2^-e of K; the factor that O needs before this tile's V; 2^-e of V
            s_info[g % kInfo] = make_float4(pow2i(-e_k), fix, e_v == INT_MAX ? 1.f : pow2i(-e_v), 0.f);
            mbar_arrive(&scan_full[st]);
            mbar_arrive(&raw_empty[st]);
          }
        }
        x += s.n;
      }
    } else if (warp == kWarpS) {
      // ------------------------------------------------ S(g) = Q K(g)^T of every block
      const uint32_t leader = elect_one();
      constexpr uint32_t kIdS = idesc_f16(BM, BN, 0);
      Ring<NK> kr;
      Ring<NS> sr[NB];  // a buffer is free once PV has read the P in it
      uint32_t q_phase[NB];
#pragma unroll
      for (int rb = 0; rb < NB; ++rb) sr[rb].phase = 1, q_phase[rb] = 0;
      // descriptors of the first stage's first 16 channels
      const uint64_t dq = sdesc_sw128(sQ(0), 16, 1024), dk = sdesc_sw128(sK(0), 16, 1024);
      for (int x = x0; x < x1 && !fail;) {
        const Seg s = seg_at(x);
        x += s.n;
#pragma unroll
        for (int rb = 0; rb < NB; ++rb)
          if (rb < s.nb && !fail) {
            fail = !ring_wait(&q_full[rb], q_phase[rb], p.err, abort_flag);
            q_phase[rb] ^= 1u;
          }
#pragma unroll 1
        for (int j = 0; j < s.n && !fail; ++j) {
          if (!ring_wait(&k_full[kr.i], kr.phase, p.err, abort_flag)) {
            fail = true;
            break;
          }
          const uint64_t kd = dk + uint64_t(kr.i * (Y::kKV >> 4));
#pragma unroll
          for (int rb = 0; rb < NB; ++rb) {
            if (M == kStreams ? (j & 1) != rb : rb >= s.nb) continue;
            const int u = sr[rb].i;
            if (!ring_wait(&pv_done[rb][u], sr[rb].phase, p.err, abort_flag)) {
              fail = true;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss(tS(rb, u), dq + rb * (Y::kQ >> 4) + (kk >> 2) * (Y::kQBox >> 4) + (kk & 3) * 2,
                     kd + (kk >> 2) * (BN * 128 >> 4) + (kk & 3) * 2, kIdS, kk > 0 ? 1u : 0u, leader);
            mma_commit(&s_full[rb][u], leader);
            sr[rb].next();
          }
          if (fail) break;
          mma_commit(&k_empty[kr.i], leader);
          kr.next();
        }
      }
    } else if (warp == kWarpPV) {
      // ------------------------------------------------ O += P(g) V(g) of every block
      // (a segment's first product overwrites O: its P exists only once the
      // block's softmax warps have read the segment before out of it)
      const uint32_t leader = elect_one();
      constexpr uint32_t kIdPV = idesc_f16(BM, D, 1);
      Ring<NV> vr;
      Ring<NS> pr[NB];
      const uint64_t dv = sdesc_sw128(sV(0), BN * 128, 1024);
      for (int x = x0; x < x1 && !fail;) {
        const Seg s = seg_at(x);
        x += s.n;
#pragma unroll 1
        for (int j = 0; j < s.n && !fail; ++j) {
          if (!ring_wait(&v_full[vr.i], vr.phase, p.err, abort_flag)) {
            fail = true;
            break;
          }
          const uint64_t vd = dv + uint64_t(vr.i * (Y::kKV >> 4));
#pragma unroll
          for (int rb = 0; rb < NB; ++rb) {
            if (M == kStreams ? (j & 1) != rb : rb >= s.nb) continue;
            const int u = pr[rb].i;
            if (!ring_wait(&p_full[rb][u], pr[rb].phase, p.err, abort_flag)) {
              fail = true;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)  // 16 keys = 8 TMEM columns of fp16 pairs
              mma_ts(tO(rb), tS(rb, u) + kk * 8, vd + kk * (16 * 128 >> 4), kIdPV,
                     (j >= (M == kStreams ? 2 : 1) || kk > 0) ? 1u : 0u, leader);
            mma_commit(&pv_done[rb][u], leader);
            pr[rb].next();
          }
          if (fail) break;
          mma_commit(&v_empty[vr.i], leader);
          vr.next();
        }
      }
    }
  } else {
    // ------------------------------------------------ softmax warps
    const int rb = warp >> 2, r = tid & (BM - 1);
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    int g = 0;
    Ring<NS> sr;
    for (int x = x0; x < x1 && !fail;) {
      const Seg s = seg_at(x);
      x += s.n;
      if (rb >= s.nb) {
        // a stream without a tile: its partials count nothing
        if (M == kStreams && r < p.R)
          p.out.ml[((size_t(blockIdx.x) + s.item) * 2 + rb) * BM + r] = make_float2(-INFINITY, 0.f);
        g += s.n;
        continue;
      }
      const int row0 = M == kPair ? s.r0 + rb * BM : 0, row = row0 + r;
      // a warp none of whose rows exists keeps the handshakes only; its part
      // of P is whatever TMEM holds, which reaches no other row
      const bool active = row0 + (warp & 3) * 32 < p.R;
      float c_row = 0.f;
      if (active) {
        // Q: the warp's 32 rows as fp16 times 2^eq of the row, D / 8 lanes to
        // a row (a thread per row would touch 32 lines an instruction: 7000
        // cycles for the two blocks, in the way of every copy).  The previous
        // segment's products, the last readers of the buffer, are done: the
        // warp waited for them before it read O.
        constexpr int kL = D / 8, kRows = 32 / kL, kIt = 32 / kRows;
        const int sub = lane / kL, ch = lane % kL;
        const int first = row0 + (warp & 3) * 32 + sub;  // and every kRows-th row after it
        // (a rolled loop, the next four rows' loads ahead of it: the code runs
        // once, and unrolled it would wait for its own instructions)
        auto load_rows = [&](int i0, uint4 (&w)[4]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rw = first + (i0 + i) * kRows;
            const int b = p.G == 1 ? rw : int(__umulhi(unsigned(rw), p.g_magic));
            const uint16_t *src = p.q + (size_t(b) * p.Hq + s.hk * p.G + (rw - b * p.G)) * D + 8 * ch;
            w[i] = rw < p.R ? *reinterpret_cast<const uint4 *>(src) : make_uint4(0u, 0u, 0u, 0u);
          }
        };
        uint4 ahead[4];
        load_rows(0, ahead);
        int eq_row = 0;
#pragma unroll 1
        for (int i0 = 0; i0 < kIt; i0 += 4) {
          uint4 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = ahead[i];
          if (i0 + 4 < kIt) load_rows(i0 + 4, ahead);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            float qm = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) qm = fmaxf(qm, fmaxf(fabsf(bf16_lo(u[e])), fabsf(bf16_hi(u[e]))));
#pragma unroll
            for (int off = kL / 2; off >= 1; off >>= 1) qm = fmaxf(qm, __shfl_xor_sync(0xffffffffu, qm, off));
            const int eq = clamp_exp(14 - ilog2(qm));
            const float up = pow2i(eq);
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = pack_half2(bf16_lo(u[e]) * up, bf16_hi(u[e]) * up);
            const int rw = (warp & 3) * 32 + sub + (i0 + i) * kRows;  // in the block
            st_shared_v4(sQ(rb) + (ch / 8) * Y::kQBox + rw * 128 + (((ch & 7) ^ (rw & 7)) << 4), h[0], h[1], h[2],
                         h[3]);
            // lane l is row l of the warp: its exponent sits in the lanes of sub l % kRows
            const int e_l = __shfl_sync(0xffffffffu, eq, (lane % kRows) * kL);
            if (lane / kRows == i0 + i) eq_row = e_l;
          }
        }
        c_row = pow2i(-eq_row) * (1.4426950408889634f * rsqrtf(float(D)));
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[rb]);

      float m_used = -INFINITY, l = 0.f, down = 1.f;
      constexpr int kEvery = M == kStreams ? 2 : 1;  // the set's tiles: every one, or every other
      const int j0 = M == kStreams ? rb : 0;
      int left = pl.len - (s.t0 + j0) * BN;
      uint64_t *pv_last = nullptr;  // PV of the tile before: its barrier and parity
      uint32_t pv_phase = 0;
#pragma unroll 1
      for (int j = j0; j < s.n; j += kEvery, sr.next(), left -= kEvery * BN) {
        const int u = sr.i;
        if (!fail) fail = !ring_wait(&s_full[rb][u], sr.phase, p.err, abort_flag);
        tc_fence_after();
        uint64_t *const pv_prev = pv_last;
        const uint32_t pv_prev_phase = pv_phase;
        pv_last = &pv_done[rb][u];
        pv_phase = sr.phase;
        if (!active) {
          if (lane == 0) mbar_arrive(&p_full[rb][u]);
          continue;
        }
        float4 info = s_info[(g + j) % kInfo];
        // the tile in between may have changed V's exponent too
        if (M == kStreams && j >= 2) info.y *= s_info[(g + j - 1) % kInfo].y;
        uint32_t v[BN];
        tmem_ld32(tS(rb, u) + lane_base, v);
        tmem_ld32(tS(rb, u) + lane_base + 32, v + 32);
        tmem_ld_wait();
        if (left < BN) {
#pragma unroll
          for (int i = 0; i < BN; ++i) v[i] = i < left ? v[i] : 0xff800000u;
        }
        // never 0, which would make NaN of the -inf of a slot behind the prefix:
        // |S| < 2^37, so at 2^-126 and below a score is 2^-89 at most and its
        // weight 1 to every bit, whatever the factor
        const float ct = fmaxf(c_row * info.x, 1.1754943508222875e-38f);
        down = info.z;
        float mxp[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          mxp[i] = max3(__uint_as_float(v[i]), __uint_as_float(v[8 + i]), __uint_as_float(v[16 + i]));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          mxp[i] = max3(mxp[i], __uint_as_float(v[24 + i]), __uint_as_float(v[32 + i]));
          mxp[i] = max3(mxp[i], __uint_as_float(v[40 + i]), __uint_as_float(v[48 + i]));
          mxp[i] = fmaxf(mxp[i], __uint_as_float(v[56 + i]));
        }
        const float mx =
            ct * max3(max3(mxp[0], mxp[1], mxp[2]), max3(mxp[3], mxp[4], mxp[5]), fmaxf(mxp[6], mxp[7]));
        const bool need = mx > m_used + kLazyLog2;  // the first tile included
        float alpha = info.y;  // what V's new exponent asks of O
        if (need) {
          const float a = ex2(m_used - mx);  // 0 at the first tile
          alpha *= a;
          l *= a;
          m_used = mx;
        }
        const uint64_t c2 = pack_f32x2(ct, ct), nmc2 = pack_f32x2(kPBias - m_used, kPBias - m_used);
        float rsp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < BN; i += 2) {
          float a, b;
          fma_f32x2(a, b, __uint_as_float(v[i]), __uint_as_float(v[i + 1]), c2, nmc2);
          a = ex2(a);
          b = ex2(b);
          add_f32x2(rsp[(i >> 1) & 1 ? 2 : 0], rsp[(i >> 1) & 1 ? 3 : 1], a, b);
          v[i / 2] = pack_half2(a, b);
        }
        l += (rsp[0] + rsp[1]) + (rsp[2] + rsp[3]);
        if (j >= kEvery && __any_sync(0xffffffffu, alpha != 1.f)) {
          // O once the set's PV before has landed
          if (!fail) fail = !ring_wait(pv_prev, pv_prev_phase, p.err, abort_flag);
          tc_fence_after();
#pragma unroll 1
          for (int ch = 0; ch < D; ch += 32) {
            uint32_t ov[32];
            tmem_ld32(tO(rb) + lane_base + ch, ov);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tmem_st32(tO(rb) + lane_base + ch, ov);
          }
        }
        tmem_st32(tS(rb, u) + lane_base, v);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[rb][u]);
      }
      g += s.n;
      // ---- the segment's partials
      if (!fail) fail = !ring_wait(pv_last, pv_phase, p.err, abort_flag);
      tc_fence_after();
      if (active && !fail) {
        const size_t slot = size_t(blockIdx.x) + s.item;
        float4 *o = reinterpret_cast<float4 *>(p.out.o) + (slot * 2 + rb) * (D / 4) * BM + r / 4 * D + r % 4;
#pragma unroll 1
        for (int ch = 0; ch < D; ch += 32) {
          uint32_t ov[32];
          tmem_ld32(tO(rb) + lane_base + ch, ov);
          tmem_ld_wait();
          if (row < p.R) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              o[ch + i] =
                  make_float4(__uint_as_float(ov[i]) * down, __uint_as_float(ov[i + 1]) * down,
                              __uint_as_float(ov[i + 2]) * down, __uint_as_float(ov[i + 3]) * down);
          }
        }
        if (row < p.R) p.out.ml[(slot * 2 + rb) * BM + r] = make_float2(m_used - kPBias, l);
        tc_fence_before();
      }
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

template <int D, Mode M>
cudaError_t launch_m(const PrefixParams &p, int grid, cudaStream_t stream) {
  auto kern = shared_prefix_kernel<D, M>;
  static std::atomic<unsigned long long> smem_set{0};  // the opt-in, once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
  if (!bit || !(smem_set.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D, M>::kBytes);
    if (e != cudaSuccess) return e;
    smem_set.fetch_or(bit, std::memory_order_release);
  }
  return launch_pdl(kern, dim3(grid), dim3(kThreads), size_t(Lay<D, M>::kBytes), stream, p);
}

template <int D>
cudaError_t launch_d(const PrefixParams &p, int grid, cudaStream_t stream) {
  if (prefix_streams(p.R) == 2) return launch_m<D, kStreams>(p, grid, stream);
  return p.R <= BM ? launch_m<D, kSingle>(p, grid, stream) : launch_m<D, kPair>(p, grid, stream);
}

}  // namespace

cudaError_t launch_shared_prefix(const void *q, const nd_kv_cache &prefix, int batch, int n_q_heads, int grid,
                                 const PrefixParts &out, int *err, cudaStream_t stream) {
  PrefixParams p;
  p.q = static_cast<const uint16_t *>(q);
  p.c = prefix;
  p.Hq = n_q_heads;
  p.G = n_q_heads / prefix.n_kv_heads;
  p.R = batch * p.G;
  p.g_magic = p.G > 1 ? unsigned((0x100000000ull + p.G - 1) / p.G) : 0u;
  p.out = out;
  p.err = err;
  if (prefix.head_dim == 128) return launch_d<128>(p, grid, stream);
  if (prefix.head_dim == 64) return launch_d<64>(p, grid, stream);
  return cudaErrorInvalidValue;
}

}  // namespace nd
