// Attention with modified scores (tanh cap, distance bias, key ranges, a shared
// prefix) on the tensor cores: one kernel body for prefill and for decode.
//
// Mathematics: O = softmax(x) V with x = scale <q, k>, capped and biased (see
// include/attn.h), in one pass over the keys with a running maximum m and sum
// l per row; everything in log2 units.  The pipeline is that of the prefill
// kernel in fwd_sm103a.cu: a TMA load warp, an MMA warp (S_t = Q_t K^T, O_t +=
// P_t V for two query tiles t, all accumulators in TMEM), sixteen softmax
// warps, a K/V ring.  What differs:
//
//   * A work item names the key tiles that its rows can see (each of the two
//     query tiles an interval of its own), found by a planning warp ahead of
//     the others and handed to them through shared memory.  Documents far from
//     a row cost it nothing, and an item that sees nothing is not loaded.
//   * The softmax warps clear the rows of V that lie outside of the item's
//     visible span in its first and last tile before they release their
//     weights: those are 0 there, but 0 * NaN in a cache's unused tail is not.
//   * Prefill (kSplit = false): an item is (batch, head, 256 query rows), handed
//     out by cluster launch control.
//   * Decode (kSplit = true): the rows of an item are the query heads that share
//     a KV head: those of 128 / G requests per tile for the shared prefix, of
//     one request for its own keys.  The prefix tiles of all items, laid end to
//     end, are cut into equal runs, one per CTA; so are the tiles of the
//     requests' own keys, whatever the lengths are, two runs per CTA: one for
//     each query tile, two chains of Q K^T, softmax and P V that do not wait
//     for one another.  Where there is enough of both, some CTAs have own keys
//     alone and the others the prefix (own_share in internal.h).  An item cut by
//     a run's end leaves fp32 partial states that a second kernel merges through
//     their log-sum-exp.  A prefix tile is read once for 256 rows, and at fewer
//     than ~300 rows its bytes cost more than its products.
//   * Own keys of at most 8 query heads per KV head are multiplied the other way
//     round, S^T = K Q^T and O^T += V^T P^T: the 128 keys of a tile are the rows
//     of the product, so 128 threads share a tile's scores, a key each, where
//     as rows of S the few heads would occupy a fraction of one warp.  P^T goes
//     through shared memory (it is the B operand).
//
// What bounds it and what it measures (us on a GB300, by CUDA events).
//   * Prefill, long rows: the chain of a query tile, product, softmax, product,
//     of which two run at a time.  B1 Hq32 Hkv8 N8192 D128 causal: 350 (1.57
//     PFLOP/s, as without modifications in fwd_sm103a.cu), capped 465, biased 460,
//     both 568; D64 271, 460, 380, 520.  The tensor pipe is 50% busy capped, the issue
//     slots 56%: a pass over a tile is longer than the products of the other.
//   * Prefill, short rows: what an item costs besides its tiles, about 5k cycles
//     for its first scores and its epilogue next to 2.9k a tile.  Packed documents
//     B4 H16 N4096 D128: 89, tensor pipe 37%.
//   * Decode of own keys: DRAM.  8 requests of up to 64k keys, Hkv8 D128: 84, 533
//     MB at 6.3 TB/s with the merge (94% of a measured copy).
//   * Decode behind a prefix: the prefix' chain of product, softmax, product on some
//     CTAs (1.5 us a tile of 256 rows, capped 2.1), on the others the latency of short
//     items of own keys (0.6 us a tile of them at 2.5 tiles an item).  64 requests
//     behind 16384 keys 38, 256 (capped) behind 8192 76.
// Code that is not in the instruction cache shows: 264 KB of a decode instead of
// 96 KB cost it 40% of its time, and a prefill's rarely taken ways 5 to 15%.
#pragma once

#include <cuda_bf16.h>
#include <limits.h>
#include <math_constants.h>

#include <atomic>

#include "fwd_tile.cuh"
#include "mod_plan.cuh"
#include "score_mod.cuh"

namespace attn {
namespace {

// mbar_wait of ptx.cuh in fewer instructions: the kernel has a wait at every turn,
// and its code has to stay in the instruction cache.
__device__ __forceinline__ bool mod_wait(uint64_t* bar, uint32_t parity, uint32_t abort_sa,
                                         unsigned int* err, uint32_t site, uint64_t limit_ns) {
  uint32_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0u) {
      uint32_t now;  // wraps after 4.3 s, the limit is 2
      asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(now));
      if (it == 64u) t0 = now;
      if (abort_set(abort_sa)) return false;
      if (now - t0 > static_cast<uint32_t>(limit_ns)) {
        abort_raise(abort_sa);
        atomicOr(err, site);
        return false;
      }
    }
  }
}

static_assert(kKeyTile == kBN, "key tiles");
constexpr int kModThreads = 640;  // 16 softmax warps, load, MMA, 2 planning warps
constexpr int kModWarpLoad = 16, kModWarpMma = 17, kModWarpPlan = 18;
// setmaxnreg split of the 61440 registers the launch gets (640 threads x 96).  A
// prefill's other roles fit 32 registers, which leaves its softmax the most (B1 Hq32
// Hkv8 N8192 D128 causal capped: 489 us, with 104 / 64 530); a decode's loaders and
// planners need more, its scores are few.
template <bool kSplit>
constexpr uint32_t kModRegSoftmax = kSplit ? 104 : 112;
template <bool kSplit>
constexpr uint32_t kModRegOther = kSplit ? 64 : 32;
static_assert(4 * 128 * kModRegSoftmax<true> + 128 * kModRegOther<true> <= 640 * 96, "registers");
static_assert(4 * 128 * kModRegSoftmax<false> + 128 * kModRegOther<false> <= 640 * 96, "registers");

// A decode's own keys use the ring's slots as four rings, K and V of either query
// tile, so that each is loaded as soon as its own slot is free.  Tile n of one is
// given the ring item number that stands for its slot (% kS) and the slot's use (/
// kS), after `before` items of the shared prefix.
template <uint32_t kS>
__device__ __forceinline__ uint32_t own_item(uint32_t before, bool is_v, int t, uint32_t n) {
  constexpr uint32_t kPer = kS / 4;
  const uint32_t slot = ((is_v ? 2u : 0u) + t) * kPer + n % kPer;
  return ((before + kS - 1 - slot) / kS + n / kPer) * kS + slot;
}

// What the softmax warps know about a row: it sees keys [lo, hi) of the item's
// K/V, and with a bias key j gets -slope * (|pos - j| - ref), pos and j counted
// alike.  Kept in shared memory: a pass needs its registers for the scores.
struct RowInfo {
  int lo, hi, pos, ref;
};

// Is S_t written in two halves, that of the keys [64, 128) while the softmax warps
// still have the tile before?  Not with a cap or a bias: D64 B1 Hq32 Hkv8 N8192
// causal 460 us capped (in halves 452, but packed documents 94, not 92), 380 biased
// (387); D128 468 (486), 461 (472).
template <int D, bool kCap, bool kBias>
constexpr bool kSplitScores = Cfg<D, false>::kSplitS && !kCap && !kBias;

// Items of a query tile in flight: a decode's are short, and planned well ahead;
// a prefill's are taken from the grid, and only one ahead, late in the item before
// (see the planner): B2 H16 N4001 D64 causal biased 106 us, where it was taken at
// that item's start 109; prefix documents capped and biased 102, 106.
template <bool kSplit>
constexpr int kWorkSlots = kSplit ? 4 : 2;

struct ModMisc {
  RowInfo rows[2 * kBM];
  float slopes[2 * kBM];  // times log2(e)
  uint64_t q_full[2], q_empty[2], unit_done;
  uint64_t s_full[2], s_read[2], p_full[2], o_done[2];
  uint64_t mma_done;
  uint64_t kv_full[8], kv_empty[8];
  uint64_t q2_full[2][2], q2_empty[2][2];  // own keys, keys as rows: Q_t in two buffers
  uint64_t s2_full[2][2], s2_read[2][2];   // S^T of a team: in TMEM; read (an arrival per warp)
  uint64_t pv2_done[2][2];                 // O^T += V^T P^T of a tile of a team retired
  uint64_t own_start[2];                   // the query tile's warps are done with prefix items
  uint64_t item_loaded;   // prefill: every load of an item has been issued
  uint64_t clc_full;      // the answer to the request for more work arrived
  uint64_t work_full[2][4], work_empty[2][4];
  uint4 clc_resp;
  Work work[2][4];        // query tile t's item k in slot k % kWorkSlots
  int2 ranges[2][2 * kBM];  // prefill: keys [x, y) that the rows of item k % 2 see
  float red[4][4][16];      // keys as rows: per team, warp and head, a maximum or a sum
  float own_slopes[4][16];  // times log2(e)
  bool slow[16];  // per softmax warp, biased: scores are modified before the exponential
  int4 seen[16];  // per softmax warp: keys [x, y) that all its rows see, [z, w) that any does
  int own_pv[2];  // O^T += V^T P^T issued so far in the query tile's run of own keys
  uint32_t tmem_base;
  int abort_flag;
};

// TMEM columns of query tile 0: S (P over its first half), O, at D = 64 Q; tile
// 1's lie kTileCols behind.
constexpr uint32_t kTileCols = 128, kColS = 0, kColO = 256;
template <int D>
constexpr uint32_t kColQ = kColO + D;  // D = 64: 320 and 448

// softcap * tanh(scale s / softcap) in log2 units, plus `add`, of two raw
// products: s T(s^2) with T of degree N - 1 and all factors in its coefficients.
// T's degree is what costs: N + 1 packed operations.  (FFMA2 does two fmas an
// issue slot, but takes the fp32 pipe twice as long as one.)
template <int N>
struct CapPoly {
  uint64_t c[N];
  __device__ __forceinline__ explicit CapPoly(const float* coef) {
    // volatile: else the coefficients of every polynomial stay in registers
    // across the tiles, and others spill
#pragma unroll
    for (int i = 0; i < N; ++i)
      asm volatile("mov.b64 %0, {%1, %1};" : "=l"(c[i]) : "f"(coef[i]));
  }
  __device__ __forceinline__ uint64_t operator()(uint64_t s, uint64_t add) const {
    const uint64_t y = mul_f32x2(s, s);
    uint64_t t = fma_f32x2(y, c[N - 1], c[N - 2]);
#pragma unroll
    for (int i = N - 3; i >= 0; --i) t = fma_f32x2(y, t, c[i]);
    return fma_f32x2(s, t, add);
  }
};

// Which of a thread's 64 columns its row sees: bit i of words[i / 32].
struct Seen {
  uint32_t words[2];
};
__device__ __forceinline__ Seen seen_columns(int from, int to) {  // columns [from, to)
  Seen m;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int f = min(max(from - 32 * h, 0), 32), e = min(max(to - 32 * h, 0), 32);
    // funnel shifts take 32: all ones from f on, none from e on
    m.words[h] = e > f ? (__funnelshift_lc(0u, 0xFFFFFFFFu, f)) &
                             ~(__funnelshift_lc(0u, 0xFFFFFFFFu, e))
                       : 0u;
  }
  return m;
}
__device__ __forceinline__ void mask_to(float (&s)[64], const Seen& m, float with) {
#pragma unroll
  for (int i = 0; i < 64; ++i) s[i] = (m.words[i / 32] >> (i % 32)) & 1u ? s[i] : with;
}

// The pass over one tile of 64 scores of a thread (half a row): from raw
// products s to weights 2^(x - m) of the scores x in log2 units.
//
// m need not be the row's largest score, only near enough that no weight
// overflows and none that matters underflows, and the same for all of a row's
// keys.  So where the modifications are cheap to apply together with the
// exponential (`fused`), they are not applied before it just to find the maximum.
//   * Capped: with A the largest raw magnitude of the warp's scores, capped, and
//     the bias of the key that it favours, m = A + bias: at most 2 A above the
//     score of that key.  (-inf for a row that sees no key of the tile.)
//   * Biased only: m is the largest of the sums of a group's largest raw product
//     and its most favoured key's bias, for groups of 16 keys: too large by the
//     bias' change over a group at most.
// kLoose limits both.  Weights then lie above 2^-kLoose where exact ones lie above
// 1/2, as precise.
//
// The bias relative to its reference is -|slope| |j - c0| with one key c0 per row
// (its own position if it sees that; else, and for a negative slope, the end of
// its keys that the bias favours), which no key of a tile passes (`linear`) but
// in the diagonal's tile of a row that sees keys on both sides.  A negative slope
// on both sides has no such c0.
constexpr float kLoose = 100.f;

template <int D, bool kCap, bool kBias>
struct Scores {
  // A capped tile's unseen keys: 0 for the maximum and cap_off for the weights in one
  // go, or one after the other.  The work is the same; which one the compiler makes the
  // better kernel of was measured, B1 Hq32 Hkv8 N8192 causal in us: D128 464 in one go
  // (one after the other 472), D64 469 (460), D64 biased 525 (547).
  static constexpr bool kOneGo = D == 128 || kBias;
  static constexpr int kModified = 4;
  int tier;          // capped: which polynomial; 3: the longest, not linear;
                     // kModified: the scores are modified already
  Seen seen;         // if masked
  bool linear;
  float slope, rel;  // biased: key kb + i has bias -slope * |rel + i|, slope >= 0
  float most[4];     // bias of the most favoured key that the row sees: capped: of the
                     // tile, in [0] (-inf: it sees none); else of every 16 keys

  // What does not depend on the scores, found while they are still multiplied.
  // kb: key of the thread's first score, kt: of the tile.  masked: some row of the
  // warp does not see all 128 keys of the tile.
  __device__ __forceinline__ void look(const RowInfo* info, const float* row_slope, int kt, int kb,
                                       bool masked) {
    RowInfo row;
    if (masked || kBias) row = *info;
    linear = true;
    if constexpr (kBias) {
      tier = 0;
      const bool left = row.hi - 1 <= row.pos || kt + kBN - 1 <= row.pos;
      slope = fabsf(*row_slope);
      const unsigned c0 = static_cast<unsigned>(row.pos) +
                          static_cast<unsigned>(left ? -row.ref : row.ref);
      const int to_c0 = static_cast<int>(c0 - static_cast<unsigned>(kt));
      linear = __all_sync(0xFFFFFFFFu, to_c0 <= 0 || to_c0 >= kBN - 1);
      rel = static_cast<float>(static_cast<int>(static_cast<unsigned>(kb) - c0));
      if constexpr (kCap) {
        const int from = max(row.lo, kt) - kt, to = min(row.hi - kt, kBN) - 1;
        const int off = max(max(from - to_c0, to_c0 - to), 0);  // c0 to the nearest
        // (a row that sees none of the tile's keys: neither is there a nearest)
        most[0] = from <= to ? -slope * static_cast<float>(off) : -CUDART_INF_F;
      } else if (linear) {
        const float step = rel < 0.f ? slope : -slope;
        most[0] = step * (rel < 0.f ? rel + 15.f : rel);
#pragma unroll
        for (int g = 1; g < 4; ++g) most[g] = fmaf(step, 16.f * g, most[0]);
      } else {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float at = rel + 16.f * g;  // c0 to the keys
          most[g] = -slope * fmaxf(fmaxf(at, -15.f - at), 0.f);
        }
      }
    }
    if (masked) seen = seen_columns(row.lo - kb, row.hi - kb);
    // Without a bias too: a row that sees none of the tile's keys takes nothing from the
    // others' scores, its own may lie any distance below them.
    if (kCap && !kBias)
      most[0] = masked && (row.lo >= kt + kBN || row.hi <= kt) ? -CUDART_INF_F : 0.f;
  }

  // From s to the row's m for the tile (both halves); false: it cannot be fused.
  __device__ __forceinline__ bool prepare(float (&s)[64], const ModKernelParams& p, bool masked,
                                          float& m) {
    if constexpr (kCap) {
      float a0 = 0.f, a1 = 0.f;
      // what lies at unseen keys has no say, and gets a weight of 0
      if (kOneGo && masked) {
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          const bool in0 = (seen.words[i / 32] >> (i % 32)) & 1u;
          const bool in1 = (seen.words[i / 32] >> (i % 32 + 1)) & 1u;
          const float x0 = in0 ? s[i] : 0.f, x1 = in1 ? s[i + 1] : 0.f;
          if (i % 4 == 0)
            a0 = max3f(a0, fabsf(x0), fabsf(x1));
          else
            a1 = max3f(a1, fabsf(x0), fabsf(x1));
          s[i] = in0 ? s[i] : p.mod.cap_off;
          s[i + 1] = in1 ? s[i + 1] : p.mod.cap_off;
        }
      } else if (masked) {
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          const uint32_t w = seen.words[i / 32];
          const float x0 = (w >> (i % 32)) & 1u ? s[i] : 0.f;
          const float x1 = (w >> (i % 32 + 1)) & 1u ? s[i + 1] : 0.f;
          const float x2 = (w >> (i % 32 + 2)) & 1u ? s[i + 2] : 0.f;
          const float x3 = (w >> (i % 32 + 3)) & 1u ? s[i + 3] : 0.f;
          a0 = max3f(a0, fabsf(x0), fabsf(x1));
          a1 = max3f(a1, fabsf(x2), fabsf(x3));
        }
        mask_to(s, seen, p.mod.cap_off);
      } else {
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          a0 = max3f(a0, fabsf(s[i]), fabsf(s[i + 1]));
          a1 = max3f(a1, fabsf(s[i + 2]), fabsf(s[i + 3]));
        }
      }
      a0 = fmaxf(a0, a1);
      // the shortest polynomial that holds for all of the warp's scores
      // (magnitudes are ordered like their bits)
      const float all = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(a0)));
      tier = !masked && all <= p.mod.cap_limit[0] ? 0 : (all <= p.mod.cap_limit[1] ? 1 : 2);
      if (!linear) tier = 3;
      const bool holds = tier < 2 || all <= p.mod.cap_limit[2];
      // no score of the warp's rows is larger: |tanh x| <= |x|, 1
      const float top = fminf(all * p.scale_log2, p.mod.cap_out);
      m = top + most[0];
      return holds && 2.f * top <= kLoose;
    } else {
      if (masked) mask_to(s, seen, -CUDART_INF_F);
      if constexpr (kBias) {
        if (tier == kModified) {
          m = row_max(s);
          return true;
        }
        m = -CUDART_INF_F;
#pragma unroll
        for (int g = 0; g < 64; g += 16) {
          float a0 = fmaxf(s[g], s[g + 1]), a1 = fmaxf(s[g + 2], s[g + 3]);
#pragma unroll
          for (int i = g + 4; i < g + 16; i += 4) {
            a0 = max3f(a0, s[i], s[i + 1]);
            a1 = max3f(a1, s[i + 2], s[i + 3]);
          }
          m = fmaxf(m, fmaf(fmaxf(a0, a1), p.scale_log2, most[g / 16]));
        }
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));  // the row's other half
      } else {
        const float mx = row_max(s);
        m = mx == -CUDART_INF_F ? mx : mx * p.scale_log2;
      }
      return true;
    }
  }

  // The thread's 64 products in TMEM, at s_addr, become scores, -inf for unseen
  // keys.  In a loop over TMEM and not in the registers: unrolled over those, this
  // rare way was a quarter of the kernel (117 KB, now 90), and the usual one slower
  // for it (prefix documents, capped and biased: 112 us, now 107).
  __device__ static __forceinline__ void modify(uint32_t s_addr, const ModKernelParams& p,
                                                const RowInfo* info, const float* row_slope,
                                                int kb) {
    const RowInfo row = *info;
    const float away = kBias ? -*row_slope : 0.f;
#pragma unroll 1
    for (int i0 = 0; i0 < 64; i0 += 16) {
      uint32_t v[16];
      tmem_ld_pair16<64>(s_addr + i0, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int key = kb + i0 + i;
        float x = __uint_as_float(v[i]);
        x = kCap ? tanh_any(x * p.mod.cap_in) * p.mod.cap_out : x * p.scale_log2;
        if constexpr (kBias) x = fmaf(away, static_cast<float>(abs(row.pos - key) - row.ref), x);
        v[i] = __float_as_uint(key >= row.lo && key < row.hi ? x : -CUDART_INF_F);
      }
      tmem_st_pair16<64>(s_addr + i0, v);
    }
    tmem_st_wait();
  }

  __device__ static __forceinline__ float row_max(const float (&s)[64]) {
    float a0 = fmaxf(s[0], s[1]), a1 = fmaxf(s[2], s[3]);
    float a2 = fmaxf(s[4], s[5]), a3 = fmaxf(s[6], s[7]);
#pragma unroll
    for (int i = 8; i < 64; i += 8) {
      a0 = max3f(a0, s[i], s[i + 1]);
      a1 = max3f(a1, s[i + 2], s[i + 3]);
      a2 = max3f(a2, s[i + 4], s[i + 5]);
      a3 = max3f(a3, s[i + 6], s[i + 7]);
    }
    const float mx = max3f(a0, a1, fmaxf(a2, a3));
    return fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));  // the row's other half
  }

  // pk = the weights as bf16 pairs, low key first; returns their sum in fp32
  // before the rounding to bf16 (2^-9 of a weight on average: its effect on O
  // is that of the rounding of O itself).  Unseen keys are -inf and give
  // exactly 0 (scale_log2 is never 0, see mod_launch.cu); capped they are cap_off,
  // for which the polynomials give less than -10^6.
  __device__ __forceinline__ float weights(const float (&s)[64], const ModKernelParams& p,
                                           float neg_m, uint32_t (&pk)[32]) const {
    uint64_t acc0 = f32x2(0.f, 0.f), acc1 = acc0;
    // pass(.., f): f(pair of s, what to add to its scores) -> exponents
    enum Bias { kNone, kLinear, kBent };
    auto pass = [&](Bias bias, auto f) {
      uint64_t add = f32x2(neg_m, neg_m), a = add;
      // linear: the bias minus m itself; else what |.| is taken of
      const float step = bias == kBent || rel < 0.f ? slope : -slope;
      const float from = bias == kBent ? 0.f : neg_m;
      const uint64_t next = f32x2(2.f * step, 2.f * step);
#pragma unroll
      for (int e = 0; e < 64; e += 4) {
        uint64_t add2[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // Pair by pair: exact at every 16th key, a sum of a few steps in
          // between (its roundings are below the score's).
          if (bias != kNone) {
            const float at = rel + static_cast<float>(e);
            if (h == 0 && e % 16 == 0)
              a = f32x2(fmaf(step, at, from), fmaf(step, at + 1.f, from));
            else
              a = add_f32x2(a, next);
            add = a;
            if (bias == kBent) {
              float b0, b1;
              unpack_f32x2(a, b0, b1);
              add = f32x2(neg_m - fabsf(b0), neg_m - fabsf(b1));
            }
          }
          add2[h] = add;
        }
        float x0, x1, x2, x3;
        unpack_f32x2(f(f32x2(s[e], s[e + 1]), add2[0]), x0, x1);
        unpack_f32x2(f(f32x2(s[e + 2], s[e + 3]), add2[1]), x2, x3);
        const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
        const float p2 = ex2_approx(x2), p3 = ex2_approx(x3);
        acc0 = add_f32x2(acc0, f32x2(p0, p1));
        acc1 = add_f32x2(acc1, f32x2(p2, p3));
        pk[e / 2] = pack_bf16x2(p0, p1);
        pk[e / 2 + 1] = pack_bf16x2(p2, p3);
      }
    };
    constexpr Bias kLin = kBias ? kLinear : kNone;
    if ((kCap || kBias) && tier == kModified) {
      pass(kNone, [](uint64_t x, uint64_t add) { return add_f32x2(x, add); });
    } else if constexpr (kCap) {
      if (tier == 0)
        pass(kLin, CapPoly<kCapN0>(p.mod.cap_coef[0]));
      else if (tier == 1)
        pass(kLin, CapPoly<kCapN1>(p.mod.cap_coef[1]));
      else if (!kBias || tier == 2)
        pass(kLin, CapPoly<kCapN2>(p.mod.cap_coef[2]));
      else
        pass(kBent, CapPoly<kCapN2>(p.mod.cap_coef[2]));
    } else {
      const uint64_t scale2 = f32x2(p.scale_log2, p.scale_log2);
      auto scaled = [&](uint64_t x, uint64_t add) { return fma_f32x2(x, scale2, add); };
      if (kBias && !linear)
        pass(kBent, scaled);
      else
        pass(kLin, scaled);
    }
    float u0, u1;
    unpack_f32x2(add_f32x2(acc0, acc1), u0, u1);
    return u0 + u1;
  }
};

// Query tile t's item k is in slot k % kSlots from work_full (phase k / kSlots)
// until every reader arrived on work_empty.
template <int kSlots>
__device__ __forceinline__ bool work_wait(ModMisc& ms, const ModKernelParams& p, int t, int k,
                                          uint32_t abort_flag, uint32_t site) {
  return warp_all(mod_wait(&ms.work_full[t][k % kSlots], (k / kSlots) & 1, abort_flag, p.err,
                            site, p.wait_limit_ns));
}
template <int kSlots>
__device__ __forceinline__ void work_done(ModMisc& ms, int t, int k, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(&ms.work_empty[t][k % kSlots]);
}
template <int kSlots>
__device__ __forceinline__ bool work_publish(ModMisc& ms, const ModKernelParams& p, int t, int k,
                                             const Work& w, uint32_t abort_flag, int lane) {
  if (k >= kSlots &&
      !warp_all(mod_wait(&ms.work_empty[t][k % kSlots], (k / kSlots + 1) & 1, abort_flag, p.err,
                          kErrWaitLoad, p.wait_limit_ns)))
    return false;
  __syncwarp();  // every lane's stores (the rows' ranges) come before the arrival
  if (lane == 0) {
    ms.work[t][k % kSlots] = w;
    mbar_arrive(&ms.work_full[t][k % kSlots]);
  }
  return true;
}

// Row r of query tile t of an item: whether it exists, its query head, and where
// its output (decode: its partial state) goes.
template <bool kSplit>
__device__ __forceinline__ bool item_row(const ModKernelParams& p, const Work& w, int t, int r,
                                         bool tile_used, int& head, size_t& out) {
  if constexpr (kSplit) {
    const int req = w.kind ? 0 : r / p.G, g = r - req * p.G;
    head = w.id * p.G + g;
    out = w.kind ? static_cast<size_t>(w.slot) * p.G + r
                 : static_cast<size_t>(w.slot) * p.pre_rows + t * kBM + r;
    return tile_used &&
           (w.kind ? r < p.G : req < p.per_tile && w.q0 + t * p.per_tile + req < p.B);
  } else {
    const int i = w.q0 + t * kBM + r;
    head = w.id % p.Hq;
    out = static_cast<size_t>(w.id) * p.Nq + i;
    return i < p.Nq;
  }
}

// Prefill item u (warp-wide): the query rows, and the key tiles they see; with
// ranges also every row's, in rows[].
__device__ __forceinline__ Work plan_unit(const ModKernelParams& p, int u, int2* rows, int lane) {
  const int nqb = (p.Nq + 2 * kBM - 1) / (2 * kBM);
  int qblk, bh;
  if (p.longest_first) {  // as decode_unit of fwd_sm103a.cu
    const int BH = p.B * p.Hq;
    const int per_group = p.group_heads * nqb;
    const int g = u / per_group;
    const int idx = u % per_group;
    const int heads = min(p.group_heads, BH - g * p.group_heads);
    qblk = nqb - 1 - idx / heads;
    bh = g * p.group_heads + idx % heads;
  } else {
    qblk = u % nqb;
    bh = u / nqb;
  }
  Work w;
  w.id = bh;
  w.q0 = qblk * 2 * kBM;
  w.kind = 1;
  w.slot = 0;
  int lo[2], hi[2];
  if (p.ranges) {
    // row lane + 32 i of the item; all loads before the first use
    constexpr int kRows = 2 * kBM / 32;
    const int2* rg =
        reinterpret_cast<const int2*>(p.ranges) + static_cast<size_t>(bh / p.Hq) * p.Nq;
    int2 r[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int row = w.q0 + i * 32 + lane;
      r[i] = row < p.Nq ? rg[row] : make_int2(0, 0);
    }
    lo[0] = lo[1] = INT_MAX;
    hi[0] = hi[1] = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      r[i].x = max(max(r[i].x, 0) - p.key0, 0);
      r[i].y = min(max(r[i].y, 0) - p.key0, p.Nk);
      if (p.causal) r[i].y = min(r[i].y, p.q_offset + w.q0 + i * 32 + lane + 1);
      if (r[i].x < r[i].y) {
        lo[i / (kRows / 2)] = min(lo[i / (kRows / 2)], r[i].x);
        hi[i / (kRows / 2)] = max(hi[i / (kRows / 2)], r[i].y);
      } else {
        r[i] = make_int2(0, 0);
      }
      rows[i * 32 + lane] = r[i];
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      lo[t] = __reduce_min_sync(0xFFFFFFFFu, lo[t]);
      hi[t] = __reduce_max_sync(0xFFFFFFFFu, hi[t]);
    }
  } else {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int first = w.q0 + t * kBM;
      lo[t] = INT_MAX;
      hi[t] = 0;
      if (first < p.Nq) {
        lo[t] = 0;
        hi[t] = p.causal ? min(p.Nk, p.q_offset + min(first + kBM, p.Nq)) : p.Nk;
      }
    }
  }
  w.lo = min(lo[0], lo[1]);
  w.hi = max(hi[0], hi[1]);
  w.n = 0;
  w.tile0 = 0;
  w.edges = 0;
  if (w.hi > 0) w.tile0 = w.lo / kBN;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const bool any = hi[t] > 0;
    w.a[t] = any ? lo[t] / kBN - w.tile0 : 0;
    w.b[t] = any ? (hi[t] + kBN - 1) / kBN - w.tile0 : 0;
    w.n = max(w.n, w.b[t]);
  }
  if (w.n > 0) {
    if (w.lo > w.tile0 * kBN) w.edges |= 1;
    if (w.hi < min((w.tile0 + w.n) * kBN, p.Nk)) w.edges |= 2;
  }
  return w;
}

// Decode of the requests' own keys with the keys as rows (G <= 8 query
// heads per KV head).  The items of a query tile's run alternate between two teams
// of four warps, each with its own S^T [128 keys, 16 heads] and O^T [D, 16 heads]
// (16 columns of the query tile's S and O), Q and P^T [16 heads, 128 keys] (in
// its Q tile of shared memory, 128-byte-swizzled as K-major operands), so one
// team's epilogue and the next item's products and softmax overlap (256 requests
// behind 8192 shared keys: 85 us with one team, 82 with two, 79 where the teams
// issue their own products with V).
constexpr int kSwapHeads = 16;  // the least a product has; columns from G on mean nothing
constexpr uint32_t kTeamCols = 16;
constexpr uint32_t kTeamQ = 4096, kSwapP = 8192, kTeamP = 4096;  // bytes
constexpr uint32_t kSwapPChunk = kSwapHeads * 128;               // 64 keys of P^T

template <int D>
struct SwapMma {
  static constexpr uint32_t kIdescS = idesc_bf16_f32(128, kSwapHeads, false);
  // A = V^T: V is [keys, D], so M runs along its rows (A MN-major, bit 15)
  static constexpr uint32_t kIdescO = idesc_bf16_f32(128, kSwapHeads, false) | (1u << 15);
  template <uint32_t kCol, int KK = 0>
  __device__ static __forceinline__ void s(uint32_t tmem, uint32_t k_desc, uint32_t q_desc) {
    if constexpr (KK < D / 16) {
      constexpr uint32_t off = ((KK >> 2) * (kBM * 128) + (KK & 3) * 32) >> 4;
      mma_ss<false, kCol, off, off, kIdescS>(tmem, k_desc, q_desc, KK > 0 ? 1u : 0u);
      s<kCol, KK + 1>(tmem, k_desc, q_desc);
    }
  }
  // the first 16 * steps keys of the tile
  template <uint32_t kCol, int KK = 0>
  __device__ static __forceinline__ void o(uint32_t tmem, uint32_t v_desc, uint32_t p_desc,
                                           uint32_t acc, int steps) {
    if constexpr (KK < kBN / 16) {
      if (KK >= steps) return;
      // the 64-element chunks of M are a tile's chunks apart; at D = 64 there
      // is one, taken twice (lanes 64.. of O^T are not used)
      constexpr uint32_t lbo = D == 128 ? static_cast<uint32_t>((kBM * 128) >> 4) << 16 : 0u;
      constexpr uint32_t off_v = ((KK * 16 * 128) >> 4) + lbo - (1u << 16);  // desc has lbo 16
      constexpr uint32_t off_p = ((KK >> 2) * kSwapPChunk + (KK & 3) * 32) >> 4;
      mma_ss<false, kCol, off_v, off_p, kIdescO>(tmem, v_desc, p_desc, KK > 0 ? 1u : acc);
      o<kCol, KK + 1>(tmem, v_desc, p_desc, acc, steps);
    }
  }
};

// Waits, as mod_wait does, until the products of the first n tiles of query tile
// t's run have been issued.
__device__ __forceinline__ bool own_turn(ModMisc& ms, const ModKernelParams& p, int t, uint32_t n,
                                         uint32_t abort_sa) {
  uint32_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    const int done = *const_cast<volatile int*>(&ms.own_pv[t]);
    if (warp_all(done >= static_cast<int>(n))) return true;
    if ((it & 255u) == 0u) {
      uint32_t now;
      asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(now));
      if (it == 256u) t0 = now;
      const bool late = now - t0 > static_cast<uint32_t>(p.wait_limit_ns);
      if (!warp_all(!abort_set(abort_sa))) return false;
      if (!warp_all(!late)) {
        abort_raise(abort_sa);
        if ((threadIdx.x & 31) == 0) atomicOr(p.err, kErrWaitSoftmax);
        return false;
      }
    }
  }
}

// Softmax, epilogue and V's edge: four warps, thread = key of the tile (S^T, P^T)
// or element of the head (O^T); NH >= G heads in registers.  The running maximum
// is common to all 128 threads.  It is kept while no score exceeds it by more than
// 2^8: one barrier that votes on that, and on every warp's waits having ended
// well, is all that the threads of a tile exchange.
// fine: the warp's waits so far ended well.  Every warp of a team comes here, also one
// that gave up: the others may be here already, at a barrier that counts it.
template <int D, int NH, bool kCap, bool kBias>
__device__ __forceinline__ void own_keys(const ModKernelParams& p, ModMisc& ms, uint8_t* smem,
                                         uint32_t tmem, int t, int k, bool fine) {
  using C = Cfg<D, false>;
  constexpr uint32_t kS = C::kStages;
  constexpr int kSlots = kWorkSlots<true>;
  const uint32_t abort_flag = smem_u32(&ms.abort_flag);
  const int q = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, me = q * 32 + lane;
  const int team = (threadIdx.x >> 7) & 1, id = t * 2 + team;
  const uint32_t bar = 1 + id;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16) + t * kTileCols +
                         team * kTeamCols;
  const uint32_t s_addr = lanes + kColS, o_addr = lanes + kColO;
  // P^T[n][me]: row n of chunk me / 64, 16-byte unit (me % 64) / 8 swizzled by n
  uint8_t* const pt = smem + C::kOffQ + t * C::kTileBytes + kSwapP + team * kTeamP +
                      (me >> 6) * kSwapPChunk + (me & 7) * 2;
  const int unit = (me & 63) >> 3;
  const int G = p.G;
  uint32_t step = 0;  // tiles of this team: phases
  // PV in flight land before this team's warps leave
  auto leave = [&]() {
    if (q == 0 && step > 0) drain_wait(&ms.pv2_done[t][team], (step - 1) & 1);
  };
  // the other warps may still be reading the last prefix item's O
  __syncwarp();
  if (lane == 0) mbar_arrive(&ms.own_start[t]);
  const bool started = fine && warp_all(mod_wait(&ms.own_start[t], 0, abort_flag, p.err,
                                                 kErrWaitSoftmax, p.wait_limit_ns));
  for (int turn = 0;; turn ^= 1, ++k) {
    bool ok = started && work_wait<kSlots>(ms, p, t, k, abort_flag, kErrWaitSoftmax);
    const Work& w = ms.work[t][k % kSlots];
    const bool mine = turn == team;
    if constexpr (kBias) {
      if (ok && mine && w.n > 0 && me < G)
        ms.own_slopes[id][me] = p.mod.slopes[w.id * G + me] * kLog2e;
    }
    if (bar_any(bar, 128, !ok)) break;
    const int n_tiles = w.n, tile0 = w.tile0, len = w.hi;
    if (n_tiles < 0) return;  // (every product of this team has retired)
    if (!mine) {
      work_done<kSlots>(ms, t, k, lane);
      continue;
    }
    float m[NH], l[NH];
#pragma unroll
    for (int n = 0; n < NH; ++n) {
      m[n] = -CUDART_INF_F;
      l[n] = 0.f;
    }
    for (int j = 0; j < n_tiles; ++j, ++step) {
      const int key = (tile0 + j) * kBN + me;
      ok = warp_all(mod_wait(&ms.s2_full[t][team], step & 1, abort_flag, p.err, kErrWaitSoftmax,
                              p.wait_limit_ns));
      tc_fence_after();
      float s[NH];
      {
        uint32_t sr[16];
        tmem_ld_lane16(s_addr, sr);
#pragma unroll
        for (int n = 0; n < NH; ++n) s[n] = __uint_as_float(sr[n]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.s2_read[t][team]);
      bool above = false;
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        if constexpr (kCap)
          s[n] = tanh_any(s[n] * p.mod.cap_in) * p.mod.cap_out;
        else
          s[n] *= p.scale_log2;
        if constexpr (kBias) {
          // the query is at the request's last key; a negative slope counts
          // from the first key of all
          const float slope = ms.own_slopes[id][n];
          const int dist = len - 1 - key - (slope < 0.f ? p.Np + len - 1 : 0);
          s[n] = fmaf(-slope, static_cast<float>(dist), s[n]);
        }
        if (key >= len || n >= G) s[n] = -CUDART_INF_F;
        above = above || s[n] > m[n] + C::kRescale;
      }
      // this team's last product is done with P^T and O^T
      if (step > 0)
        ok = ok && warp_all(mod_wait(&ms.pv2_done[t][team], (step - 1) & 1, abort_flag, p.err,
                                     kErrWaitCorr, p.wait_limit_ns));
      if (bar_any(bar, 128, above || !ok)) {
        if (bar_any(bar, 128, !ok)) return leave();
        // the tile's maximum of every head
#pragma unroll
        for (int n = 0; n < NH; ++n) {
          // as integers of the same order
          int x = __float_as_int(s[n]);
          x ^= (x >> 31) & 0x7FFFFFFF;
          x = __reduce_max_sync(0xFFFFFFFFu, x);
          if (lane == n) ms.red[id][q][n] = __int_as_float(x ^ ((x >> 31) & 0x7FFFFFFF));
        }
        bar_sync(bar, 128);
        bool scale_o = false;
        float alpha[NH];
#pragma unroll
        for (int n = 0; n < NH; ++n) {
          const float mx = fmaxf(fmaxf(ms.red[id][0][n], ms.red[id][1][n]),
                                 fmaxf(ms.red[id][2][n], ms.red[id][3][n]));
          alpha[n] = 1.f;
          if (mx > m[n] + C::kRescale) {
            if (m[n] != -CUDART_INF_F) alpha[n] = ex2_approx(m[n] - mx);
            m[n] = mx;
          }
          l[n] *= alpha[n];
          scale_o = scale_o || alpha[n] != 1.f;
        }
        if (j > 0 && scale_o) {  // alike in all threads
          uint32_t v[16];
          tc_fence_after();
          tmem_ld_lane16(o_addr, v);
#pragma unroll
          for (int n = 0; n < NH; ++n) v[n] = __float_as_uint(__uint_as_float(v[n]) * alpha[n]);
          tmem_st_lane16(o_addr, v);
          tmem_st_wait();
        }
      }
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        // -inf - -inf: nothing was seen yet, nor is this key
        const float x = s[n] == -CUDART_INF_F ? 0.f : ex2_approx(s[n] - m[n]);
        l[n] += x;
        if (n < G)
          *reinterpret_cast<__nv_bfloat16*>(pt + n * 128 + ((unit ^ (n & 7)) << 4)) =
              __float2bfloat16_rn(x);
      }
      // V, once the tile before it in the run has been multiplied (the slot's barrier is
      // then in this tile's phase)
      const uint32_t n_run = w.v_last + j;
      const uint32_t iv = own_item<kS>(w.v_first, true, t, n_run);
      const bool edge = (w.edges & 2) && j == n_tiles - 1;
      const int keep = len - (tile0 + j) * kBN;  // keys of the tile, if it is an edge
      if (edge || q == 0) {
        ok = own_turn(ms, p, t, n_run, abort_flag) &&
             warp_all(mod_wait(&ms.kv_full[iv % kS], (iv / kS) & 1u, abort_flag, p.err,
                               kErrWaitSoftmax, p.wait_limit_ns));
        if (edge && ok) {
          // Behind the request's keys the weights are 0, but 0 * NaN is not.  The product
          // takes 16 keys at a time, up to the last that holds one.
          uint8_t* v = smem + C::kOffKV + (iv % kS) * C::kTileBytes;
          const int row0 = keep & ~15;
          for (int i = me; i < 16 * C::kChunks * 8; i += 128) {
            const int row = row0 + ((i >> 3) & 15);
            if (row >= keep && row < kBN)
              *reinterpret_cast<uint4*>(v + (i >> 7) * (kBM * 128) + row * 128 + (i & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      if (bar_any(bar, 128, !ok)) return leave();
      if (q == 0) {
        // O^T (+)= V^T P^T, issued by this team itself: its P^T is complete here, and the
        // MMA warp need not wait for it
        tc_fence_after();
        const uint32_t desc_k = sdesc_sw128_lo(smem_u32(smem + C::kOffKV), 16);
        const uint32_t p_desc = sdesc_sw128_lo(
            smem_u32(smem + C::kOffQ + t * C::kTileBytes + kSwapP + team * kTeamP), 16);
        SwapMma<D>::template o<kColO>(tmem + t * kTileCols + team * kTeamCols,
                                      desc_k + (iv % kS) * (C::kTileBytes >> 4), p_desc,
                                      j > 0 ? 1u : 0u, edge ? (keep + 15) / 16 : kBN / 16);
        mma_commit(&ms.kv_empty[iv % kS]);
        mma_commit(&ms.pv2_done[t][team]);
        if (lane == 0) *const_cast<volatile int*>(&ms.own_pv[t]) = static_cast<int>(n_run) + 1;
      }
    }
    ok = warp_all(mod_wait(&ms.pv2_done[t][team], (step - 1) & 1, abort_flag, p.err, kErrWaitCorr,
                           p.wait_limit_ns));
#pragma unroll
    for (int n = 0; n < NH; ++n) {
#pragma unroll
      for (int d = 16; d >= 1; d /= 2) l[n] += __shfl_xor_sync(0xFFFFFFFFu, l[n], d);
      if (lane == n) ms.red[id][q][n] = l[n];
    }
    if (bar_any(bar, 128, !ok)) return leave();
    tc_fence_after();
    const size_t row0 = static_cast<size_t>(w.slot) * G;
    uint32_t o[16];
    tmem_ld_lane16(o_addr, o);
#pragma unroll
    for (int n = 0; n < NH; ++n) {
      const float sum =
          (ms.red[id][0][n] + ms.red[id][1][n]) + (ms.red[id][2][n] + ms.red[id][3][n]);
      const bool none = sum == 0.f;
      const float inv = none ? 0.f : 1.f / sum;
      if (n < G) {
        if (me < D) p.part_o[(row0 + n) * D + me] = none ? 0.f : __uint_as_float(o[n]) * inv;
        if (me == 0) p.part_lse[row0 + n] = none ? -CUDART_INF_F : m[n] + __log2f(sum);
      }
    }
    tc_fence_before();
    work_done<kSlots>(ms, t, k, lane);
  }
  leave();
}

template <int D, bool kSplit, bool kCap, bool kBias, int kHeads>
__global__ void __launch_bounds__(kModThreads, 1)
    mod_attn_kernel(const __grid_constant__ ModKernelParams p) {
  using C = Cfg<D, false>;
  constexpr uint32_t kS = C::kStages;
  constexpr int kSlots = kWorkSlots<kSplit>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ ModMisc ms;
  const uint32_t abort_flag = smem_u32(&ms.abort_flag);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- set-up: barriers (load warp), TMEM (MMA warp)
  if (warp == kModWarpLoad && lane == 0) {
    mbar_init(&ms.unit_done, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&ms.q_full[t], 1);
      mbar_init(&ms.q_empty[t], 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(&ms.q2_full[t][i], 1);
        mbar_init(&ms.q2_empty[t][i], 1);
        mbar_init(&ms.s2_full[t][i], 1);
        mbar_init(&ms.s2_read[t][i], 4);
        mbar_init(&ms.pv2_done[t][i], 1);
      }
      mbar_init(&ms.own_start[t], 8);
      ms.own_pv[t] = 0;
      mbar_init(&ms.s_full[t], 1);
      mbar_init(&ms.s_read[t], 8);
      mbar_init(&ms.p_full[t], 8);
      mbar_init(&ms.o_done[t], 1);
      // readers: 8 softmax warps, load and MMA warp (a prefill's last two read
      // the first query tile's copy only)
      for (int i = 0; i < kSlots; ++i) {
        mbar_init(&ms.work_full[t][i], 1);
        mbar_init(&ms.work_empty[t][i], kSplit || t == 0 ? 10 : 8);
      }
    }
    mbar_init(&ms.mma_done, 1);
    mbar_init(&ms.clc_full, 1);
    mbar_init(&ms.item_loaded, 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&ms.kv_full[s], 1);
      mbar_init(&ms.kv_empty[s], 1);
    }
    ms.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tmap_q);
    tma_prefetch_desc(&p.tmap_k);
    tma_prefetch_desc(&p.tmap_v);
  }
  if (warp == kModWarpMma) {
    tmem_alloc(&ms.tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  if constexpr (kSplit) {
    // Q rows that no request fills hold zeros, not what was left here: their
    // scores then never send a warp down a slow path
    for (int i = threadIdx.x; i < C::kOffKV / 16; i += kModThreads)
      reinterpret_cast<uint4*>(smem + C::kOffQ)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem_base;
  // the merge kernel may be scheduled as this one's CTAs leave; it waits for all
  if constexpr (kSplit) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp < 16) {
    // =====================================================================
    // softmax + epilogue: warps 8t .. 8t + 7 serve query tile t; a warp has 16
    // rows, threads i and i + 16 the two 64-key halves of row i (the layout of
    // fwd_sm103a.cu).
    // =====================================================================
    reg_alloc<kModRegSoftmax<kSplit>>();
    const int t = warp >> 3;
    const int lbase = (warp & 3) * 32 + ((warp >> 2) & 1) * 16;  // first TMEM lane of the warp
    const int r = lbase + (lane & 15);                           // row within the tile
    const int c = lane >> 4;                                     // column half of the row
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(lbase) << 16);
    const uint32_t s_addr = lane_addr + kColS + t * kTileCols;
    const uint32_t o_addr = lane_addr + kColO + t * kTileCols;
    uint32_t step = 0;   // tiles done by this query tile: phase of s_full
    uint32_t units = 0;  // items that this query tile took part in: phase of o_done
    constexpr bool swap = kHeads > 0;  // own keys as rows
    int k = 0;
    bool fine = true;
    for (; !swap || p.prefix_tiles > 0; ++k) {
      fine = work_wait<kSlots>(ms, p, t, k, abort_flag, kErrWaitSoftmax);
      if (!fine) break;
      const Work& w = ms.work[t][k % kSlots];  // read where needed: registers are scarce
      if (w.n < 0) break;
      if (swap && w.kind == 2) {
        work_done<kSlots>(ms, t, k++, lane);
        break;
      }
      const int ja = w.a[t], jb = w.b[t];
      // the row: which query, which keys
      bool live;  // does a row of the warp exist and see a key?
      {
        RowInfo row;
        float slope = 0.f;
        int head;
        size_t out;
        const bool valid = item_row<kSplit>(p, w, t, r, jb > 0, head, out);
        // rows that are not there take the item's span and see what the others do
        row.lo = w.lo;
        row.hi = w.hi;
        row.pos = row.ref = 0;
        if constexpr (kSplit) {
          if constexpr (kBias) {
            if (valid) {
              // positions count from the item's first key
              const int b = w.q0 + (w.kind ? 0 : t * p.per_tile + r / p.G);
              row.pos = (w.kind ? w.hi : p.Np + request_len(p, b)) - 1;
              slope = p.mod.slopes[head] * kLog2e;
              // nearest: the query's own position; farthest: the first key of all
              if (slope < 0.f) row.ref = (w.kind ? p.Np : 0) + row.pos;
            }
          }
        } else {
          const int i = w.q0 + t * kBM + r;
          row.pos = p.q_offset + i;
          if (valid) {
            row.lo = 0;
            row.hi = p.Nk;
            if (p.ranges) {
              const int2 rg = ms.ranges[k & 1][t * kBM + r];
              row.lo = rg.x;
              row.hi = rg.y;
            } else if (p.causal) {
              row.hi = min(row.hi, row.pos + 1);
            }
            if constexpr (kBias) {
              slope = p.mod.slopes[head] * kLog2e;
              if (row.lo < row.hi) row.ref = bias_ref(slope, row.pos, row.lo, row.hi);
            }
          }
        }
        live = __any_sync(0xFFFFFFFFu, valid && row.lo < row.hi);
        // keys that all rows of the warp see, and that any does
        int4 seen;
        seen.x = __reduce_max_sync(0xFFFFFFFFu, row.lo);
        seen.y = __reduce_min_sync(0xFFFFFFFFu, row.hi);
        seen.z = __reduce_min_sync(0xFFFFFFFFu, row.lo < row.hi ? row.lo : INT_MAX);
        seen.w = live ? __reduce_max_sync(0xFFFFFFFFu, row.hi) : 0;
        if (lane == 0) ms.seen[warp] = seen;
        if constexpr (kBias) {
          // Rows whose bias does not go with the exponential: those that look both ways with
          // a negative slope, and steep slopes, for which the biases of 16 keys, summed up in
          // steps, lose digits of the nearest one's (and, without a cap, say too little
          // about the largest score).
          const bool slow =
              __any_sync(0xFFFFFFFFu, (slope < 0.f && row.lo < row.pos && row.hi - 1 > row.pos) ||
                                          fabsf(slope) * 15.f > kLoose);
          if (lane == 0) ms.slow[warp] = slow;
        }
        if (c == 0) {
          ms.rows[t * kBM + r] = row;
          if constexpr (kBias) ms.slopes[t * kBM + r] = slope;
        }
        __syncwarp();
      }
      float m = -CUDART_INF_F, l = 0.f;  // l: sum over this thread's half of the row
      bool ok = true;
      for (int j = ja; j < jb; ++j, ++step) {
        const int kt = (w.tile0 + j) * kBN;  // first key of the tile
        bool masked, dead;
        {
          const int4 seen = ms.seen[warp];
          masked = kt < seen.x || kt + kBN > seen.y;
          dead = kt >= seen.w || kt + kBN <= seen.z;  // no row sees a key of the tile
        }
        Scores<D, kCap, kBias> scores;
        bool slow = false;
        if (!dead) {
          scores.look(&ms.rows[t * kBM + r], &ms.slopes[t * kBM + r], kt, kt + c * 64, masked);
          if constexpr (kBias) slow = ms.slow[warp];
        }
        const int edges = w.edges;
        const bool edge = ((edges & 1) && j == 0) || ((edges & 2) && j == w.n - 1);
        if (!warp_all(mod_wait(&ms.s_full[t], step & 1, abort_flag, p.err, kErrWaitSoftmax,
                                p.wait_limit_ns))) {
          ok = false;
          break;
        }
        if (edge) {
          // clear V's unseen rows, all warps of the query tile together (where
          // both query tiles use the tile, each does).  The tile of V that was
          // in its ring slot before has been multiplied already (before this
          // S), so the slot's barrier is in this tile's phase.
          uint32_t iv = j == w.n - 1 ? w.v_last : w.v_first;
          if (kSplit && w.kind == 1) iv = own_item<kS>(w.v_first, true, t, w.v_last + j);
          if (!warp_all(mod_wait(&ms.kv_full[iv % kS], (iv / kS) & 1u, abort_flag, p.err,
                                  kErrWaitSoftmax, p.wait_limit_ns))) {
            ok = false;
            break;
          }
          uint4* v = reinterpret_cast<uint4*>(smem + C::kOffKV + (iv % kS) * C::kTileBytes);
          for (int i = (warp & 7) * 32 + lane; i < kBN * C::kChunks * 8; i += 256) {
            const int key = kt + ((i >> 3) & (kBN - 1));
            if (key < w.lo || key >= w.hi) v[i] = make_uint4(0, 0, 0, 0);
          }
        }
        if (dead) {
          if (live) {
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) pk[i] = 0;
            tc_fence_after();
            tmem_st_pair32<32>(s_addr, pk);
            tmem_st_wait();
          }
          if (edge) fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (kSplitScores<D, kCap, kBias>) mbar_arrive(&ms.s_read[t]);
            mbar_arrive(&ms.p_full[t]);
          }
          continue;
        }
        tc_fence_after();
        float s[64], m_tile;
        auto load = [&] {
          uint32_t sr[64];
          tmem_ld_pair64<64>(s_addr, sr);
#pragma unroll
          for (int i = 0; i < 64; ++i) s[i] = __uint_as_float(sr[i]);
        };
        auto modify = [&] {
          scores.modify(s_addr, p, &ms.rows[t * kBM + r], &ms.slopes[t * kBM + r], kt + c * 64);
          scores.tier = scores.kModified;
        };
        if constexpr (kCap) {
          load();
          if (slow || !scores.prepare(s, p, masked, m_tile)) {
            modify();
            load();
            m_tile = scores.row_max(s);
          }
        } else {
          if constexpr (kBias) {
            if (slow) modify();
          }
          load();
          scores.prepare(s, p, masked, m_tile);
        }
        if constexpr (kSplitScores<D, kCap, kBias>) {
          // S_t has been read: the MMA warp may write the next tile's keys
          // [64, 128) over columns 64..127, which P does not use
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms.s_read[t]);
        }
        float alpha = 1.f;
        if (m_tile > m + C::kRescale || m == -CUDART_INF_F) {
          // nothing is accumulated yet while m = -inf: no rescale
          if (m != -CUDART_INF_F) alpha = ex2_approx(m - m_tile);
          m = m_tile;
        }
        const float neg_m = m == -CUDART_INF_F ? 0.f : -m;
        uint32_t pk[32];
        const float rsum = scores.weights(s, p, neg_m, pk);
        l = fmaf(l, alpha, rsum);
        // rescale O_t when a row's maximum rose past the threshold: every P V
        // of earlier tiles has retired (it was issued before this S_t)
        if (j > ja && __any_sync(0xFFFFFFFFu, alpha != 1.f)) {
#pragma unroll 1
          for (int kk = 0; kk < D / 32; ++kk) {
            uint32_t v[16];
            tmem_ld_pair16<D / 2>(o_addr + kk * 16, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
            tmem_st_pair16<D / 2>(o_addr + kk * 16, v);
          }
          tmem_st_wait();
        }
        tmem_st_pair32<32>(s_addr, pk);
        if (edge) fence_proxy_async_smem();
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.p_full[t]);
      }
      fine = ok;
      if (!ok) break;
      if (jb > ja) {
        ok = warp_all(mod_wait(&ms.o_done[t], units & 1, abort_flag, p.err, kErrWaitCorr,
                                p.wait_limit_ns));
        ++units;
        fine = ok;
        if (!ok) break;
      }
      if (!kSplit || live) {
        tc_fence_after();
        // ---- epilogue: O / l and the LSE; a row that saw nothing gives 0 and -inf
        int head;
        size_t out;
        const bool valid = item_row<kSplit>(p, w, t, r, jb > 0, head, out);
        const float l_row = l + __shfl_xor_sync(0xFFFFFFFFu, l, 16);
        const bool none = l_row == 0.f;  // or no tiles: O in TMEM is not the item's
        const float inv = none ? 0.f : 1.f / l_row;
        const float lse2 = none ? -CUDART_INF_F : m + __log2f(l_row);
        // rolled: code that runs once an item comes from far at every line
#pragma unroll 1
        for (int kk = 0; kk < D / 32; ++kk) {
          uint32_t v[16];  // columns c * D / 2 + [16 kk, 16 kk + 16) of the row
          tmem_ld_pair16<D / 2>(o_addr + kk * 16, v);
          const size_t at = out * D + c * (D / 2) + kk * 16;
          if constexpr (kSplit) {
            float* dst = (w.kind ? p.part_o : p.pre_o) + at;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              v[i] = none ? 0u : __float_as_uint(__uint_as_float(v[i]) * inv);
            if (valid) {
              st_global_v8(dst, v);  // a whole 32-byte sector
              st_global_v8(dst + 8, v + 8);
            }
          } else {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + at;
            uint32_t o2[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              o2[i] = none ? 0u
                           : pack_bf16x2(__uint_as_float(v[2 * i]) * inv,
                                         __uint_as_float(v[2 * i + 1]) * inv);
            if (valid) {
              if (p.o_sectors) {
                st_global_v8(dst, o2);
              } else {
#pragma unroll
                for (int g = 0; g < 2; ++g)
                  reinterpret_cast<uint4*>(dst)[g] =
                      make_uint4(o2[4 * g], o2[4 * g + 1], o2[4 * g + 2], o2[4 * g + 3]);
              }
            }
          }
        }
        if (valid && c == 0) {
          if constexpr (kSplit)
            (w.kind ? p.part_lse : p.pre_lse)[out] = lse2;
          else
            p.lse[out] = (kBias ? lse2 - ms.slopes[t * kBM + r] *
                                             static_cast<float>(ms.rows[t * kBM + r].ref)
                                : lse2) * kLn2;
        }
      }
      work_done<kSlots>(ms, t, k, lane);
    }
    if constexpr (swap) own_keys<D, kHeads, kCap, kBias>(p, ms, smem, tmem, t, k, fine);
  } else if (warp == kModWarpLoad) {
    // =====================================================================
    // TMA loader and planner.  Ring items run on across work items: the item's
    // tile j is ring items 2 (j + tiles before), + 1 (K, then V).
    // =====================================================================
    reg_dealloc<kModRegOther<kSplit>>();
    uint32_t g = 0;              // next ring item
    uint32_t q0_loads = 0, q1_loads = 0;  // loads of Q_0, Q_1 issued
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t phase) {
      return warp_all(mod_wait(bar, phase & 1u, abort_flag, p.err, kErrWaitLoad, p.wait_limit_ns));
    };
    // a K or V tile into the ring
    auto load_tile = [&](const CUtensorMap* map, int key, int bh, uint64_t policy) {
      const uint32_t s = g % kS;
      if (!wait(&ms.kv_empty[s], (g / kS) + 1)) return false;
      mbar_arrive_expect_tx_elect(&ms.kv_full[s], C::kTileBytes);
      uint8_t* dst = smem + C::kOffKV + s * C::kTileBytes;
#pragma unroll
      for (int ch = 0; ch < C::kChunks; ++ch)
        tma_load_3d_elect(dst + ch * (kBM * 128), map, &ms.kv_full[s], ch * C::kAtomElems, key, bh,
                          policy);
      ++g;
      return true;
    };
    // Q_t of an item of two query tiles, once its last Q K^T (or copy to TMEM) read it
    auto load_q = [&](int t, int id, int q0) {
      const uint32_t before = t ? q1_loads : q0_loads;
      if (before > 0 && !wait(&ms.q_empty[t], before - 1)) return false;
      if (t)
        ++q1_loads;
      else
        ++q0_loads;
      uint8_t* dst = smem + C::kOffQ + t * C::kTileBytes;
      if constexpr (kSplit) {
        mbar_arrive_expect_tx_elect(&ms.q_full[t], C::kChunks * p.per_tile * p.G * 128);
        for (int ch = 0; ch < C::kChunks; ++ch)
          tma_load_4d_elect(dst + ch * (kBM * 128), &p.tmap_q, &ms.q_full[t], ch * C::kAtomElems, 0,
                            id, q0 + t * p.per_tile, l2_policy_evict_last());
      } else {
        mbar_arrive_expect_tx_elect(&ms.q_full[t], C::kTileBytes);
        for (int ch = 0; ch < C::kChunks; ++ch)
          tma_load_3d_elect(dst + ch * (kBM * 128), &p.tmap_q, &ms.q_full[t], ch * C::kAtomElems,
                            q0 + t * kBM, id, l2_policy_evict_first());
      }
      return true;
    };
    // ---- items of two query tiles that share their K and V tiles
    int k = 0;
    for (; ok && (!kSplit || p.prefix_tiles > 0); ++k) {
      ok = work_wait<kSlots>(ms, p, 0, k, abort_flag, kErrWaitLoad);
      if (!ok) break;
      const Work& w = ms.work[0][k % kSlots];
      const int n = w.n, tile0 = w.tile0, id = w.id, q0 = w.q0;
      const bool use0 = w.b[0] > w.a[0], use1 = w.b[1] > w.a[1];
      const bool last_item = kSplit ? w.kind == 2 : n < 0;
      work_done<kSlots>(ms, 0, k, lane);
      if constexpr (kSplit) {
        ok = work_wait<kSlots>(ms, p, 1, k, abort_flag, kErrWaitLoad);
        if (!ok) break;
        work_done<kSlots>(ms, 1, k, lane);
      }
      if (last_item) {
        ++k;
        break;
      }
      int bh = id;
      uint64_t policy = l2_policy_evict_last();
      if constexpr (kSplit) {
        if (p.row_blocks == 1) policy = l2_policy_evict_first();  // read once
      } else {
        bh = (id / p.Hq) * p.Hkv + (id % p.Hq) / p.G;
      }
#pragma unroll 1
      for (int i = 0; i < 2 * n && ok; ++i) {  // K, V, K, V, ..
        ok = load_tile((i & 1) ? (kSplit ? &p.tmap_vp : &p.tmap_v)
                               : (kSplit ? &p.tmap_kp : &p.tmap_k),
                       (tile0 + (i >> 1)) * kBN, bh, policy);
        if (i == 0) {
          ok = ok && (!use0 || load_q(0, id, q0));
          ok = ok && (!use1 || load_q(1, id, q0));
        }
      }
      if (!kSplit && lane == 0) mbar_arrive(&ms.item_loaded);
    }
    // ---- decode: the two runs of own keys, a tile of either in turn
    if constexpr (kSplit) {
      // K of query tile 0, of 1, V of 0, of 1: four sequences of tiles, one a lane,
      // each issued when its ring slot is free.
      const uint32_t before = g;  // ring items of the prefix
      const int t = lane & 1;
      const bool is_v = (lane & 2) != 0;
      int item = 0, left = 0;         // next item's number; tiles left of this one
      int key = 0, hi = 0, bh = 0;    // next key, the item's end, row of the cache
      uint32_t n = 0;                 // tiles issued
      bool over = lane >= 4;
      // (an item's Q comes with its first K; the buffer has to be free of the item
      // two, without buffers by team one, before, and of the prefix items' Q)
      const uint32_t loads = t ? q1_loads : q0_loads;
      const uint64_t policy = l2_policy_evict_first();  // every byte is read once
      uint32_t idle = 0, t0 = 0;
#pragma unroll 1
      for (;;) {
        const int k_item = __shfl_sync(0xFFFFFFFFu, item, t);  // V follows K's items
        const uint32_t it = own_item<kS>(before, is_v, t, n);
        bool did = false;
        if (!over && mbar_test(&ms.kv_empty[it % kS], ((it / kS) + 1) & 1u)) {
          const bool fresh = left == 0;
          const int at = k + item, slot = at % kSlots;
          bool go = true;
          if (fresh) {
            go = is_v ? item < k_item
                      : mbar_test(&ms.work_full[t][slot], (at / kSlots) & 1u);
            if (go) {
              const Work& w = ms.work[t][slot];
              if (w.n < 0) {
                over = did = true;
                go = false;
                ++item;
                if (is_v) mbar_arrive(&ms.work_empty[t][slot]);
              } else if (!is_v) {
                if (kHeads > 0 && item >= 2)
                  go = mbar_test(&ms.q2_empty[t][item & 1], ((item >> 1) + 1) & 1u);
                else if (kHeads > 0)
                  go = loads == 0 || mbar_test(&ms.q_empty[t], (loads - 1) & 1u);
                else
                  go = loads + item == 0 || mbar_test(&ms.q_empty[t], (loads + item - 1) & 1u);
              }
            }
          }
          if (go) {
            const Work& w = ms.work[t][slot];
            if (fresh) {
              left = w.n;
              key = w.tile0 * kBN;
              hi = w.hi;
              bh = w.q0 * p.Hkv + w.id;
            }
            // as many boxes of 32 keys as hold keys: little of a cache's unused tail is read
            const int boxes = (min(hi - key, kBN) + 31) / 32;
            const CUtensorMap* map = is_v ? &p.tmap_v : &p.tmap_k;
            uint64_t* full = &ms.kv_full[it % kS];
            uint8_t* dst = smem + C::kOffKV + (it % kS) * C::kTileBytes;
            mbar_arrive_expect_tx(full, boxes * 32 * (C::kChunks * 128));
#pragma unroll 1
            for (int x = 0; x < boxes; ++x) {
#pragma unroll
              for (int ch = 0; ch < C::kChunks; ++ch)
                tma_load_3d(dst + ch * (kBM * 128) + x * (32 * 128), map, full,
                            ch * C::kAtomElems, key + 32 * x, bh, policy);
            }
            if (fresh && !is_v) {
              const int buf = kHeads > 0 ? item & 1 : 0;
              uint64_t* q_full = kHeads > 0 ? &ms.q2_full[t][buf] : &ms.q_full[t];
              uint8_t* q = smem + C::kOffQ + t * C::kTileBytes + buf * kTeamQ;
              mbar_arrive_expect_tx(q_full, C::kChunks * p.G * 128);
#pragma unroll
              for (int ch = 0; ch < C::kChunks; ++ch)
                tma_load_4d(q + ch * (kBM * 128), &p.tmap_q1, q_full, ch * C::kAtomElems, 0, w.id,
                            w.q0, l2_policy_evict_last());
            }
            if (fresh) {
              if (is_v) mbar_arrive(&ms.work_empty[t][slot]);
              ++item;
            }
            key += kBN;
            --left;
            ++n;
            did = true;
          }
        }
        __syncwarp();
        if (warp_all(over)) break;
        // as mod_wait: give up on an abort or after the time limit
        idle = warp_all(!did) ? idle + 1 : 0;
        if (idle && (idle & 255u) == 0u) {
          uint32_t now;
          asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(now));
          if (idle == 256u) t0 = now;
          const bool late = now - t0 > static_cast<uint32_t>(p.wait_limit_ns);
          if (!warp_all(!abort_set(abort_flag))) break;
          if (!warp_all(!late)) {
            abort_raise(abort_flag);
            if (lane == 0) atomicOr(p.err, kErrWaitLoad);
            break;
          }
        }
      }
      if (lane < 4 && abort_set(abort_flag)) {
        // let the copies still in flight land: the last use of every slot and Q buffer
        for (uint32_t i = n > kS / 4 ? n - kS / 4 : 0; i < n; ++i) {
          const uint32_t it = own_item<kS>(before, is_v, t, i);
          drain_wait(&ms.kv_full[it % kS], (it / kS) & 1);
        }
        if (!is_v) {
          const int items = item - (over ? 1 : 0);
          if (kHeads > 0) {
            for (int i = max(items - 2, 0); i < items; ++i)
              drain_wait(&ms.q2_full[t][i & 1], (i >> 1) & 1);
          } else if (items > 0) {
            drain_wait(&ms.q_full[t], (loads + items - 1) & 1);
          }
        }
      }
      __syncwarp();
    }
    if (abort_set(abort_flag)) {
      // let the copies still in flight land before the CTA exits
      if (q0_loads > 0) drain_wait(&ms.q_full[0], (q0_loads - 1) & 1);
      if (q1_loads > 0) drain_wait(&ms.q_full[1], (q1_loads - 1) & 1);
      for (uint32_t it = g > kS ? g - kS : 0u; it < g; ++it)
        drain_wait(&ms.kv_full[it % kS], (it / kS) & 1u);
    }
  } else if (warp == kModWarpMma) {
    // =====================================================================
    // MMA issuer (warp-wide, one elected thread per instruction).  Step j of an
    // item issues, per query tile, O_t += P_t V_{j-1} and S_t = Q_t K_j^T.
    // =====================================================================
    reg_dealloc<kModRegOther<kSplit>>();
    constexpr uint32_t kTileDesc = C::kTileBytes >> 4;
    const uint32_t desc_k = sdesc_sw128_lo(smem_u32(smem + C::kOffKV), 16);
    constexpr uint32_t kQFromK = static_cast<uint32_t>((C::kOffKV - C::kOffQ) >> 4);
    constexpr uint32_t kVFromK = static_cast<uint32_t>(((kBM * 128) >> 4) - 1) << 16;
    static_assert((kS & (kS - 1)) == 0, "ring depth must be a power of two");
    constexpr uint32_t kQ0 = 0u - kQFromK;
    // Query tile 1's TMEM columns all lie kTileCols behind tile 0's and its Q in
    // shared memory a tile behind, so one copy of the issuing code serves both.
    constexpr uint32_t kTQ = C::kQInTmem ? kColQ<D> : 0;
    // S_t = Q_t K^T: all keys, or (half) the lower / upper 64
    auto issue_s = [&](int t, uint32_t b0, int half) {
      const uint32_t base = tmem + t * kTileCols, a0 = desc_k + t * kTileDesc;
      if (half == 0)
        issue_s_steps<D, false, kColS, kQ0, 0, kTQ>(base, a0, b0);
      else if (half == 1)
        issue_s_steps<D, false, kColS, kQ0, 1, kTQ>(base, a0, b0);
      else
        issue_s_steps<D, false, kColS, kQ0, 2, kTQ>(base, a0, b0);
    };
    auto issue_pv = [&](int t, uint32_t b0, uint32_t acc) {
      issue_pv_steps<D, false, kColO, kColS, kVFromK>(tmem + t * kTileCols, b0, acc);
    };
    auto wait = [&](uint64_t* bar, uint32_t phase) {
      return warp_all(mod_wait(bar, phase & 1u, abort_flag, p.err, kErrWaitMma, p.wait_limit_ns));
    };
    uint32_t tiles = 0;          // key tiles so far: ring items 2 tiles ..
    uint32_t steps0 = 0, steps1 = 0;  // S_0, S_1 issued so far
    uint32_t qs0 = 0, qs1 = 0;        // Q_0, Q_1 taken so far
    int k = 0;
    bool ok = true;
    // ---- items of two query tiles on the same K and V tiles
    for (uint32_t items = 0; ok && (!kSplit || p.prefix_tiles > 0); ++k) {
      ok = work_wait<kSlots>(ms, p, 0, k, abort_flag, kErrWaitMma);
      if (!ok) break;
      const Work& w = ms.work[0][k % kSlots];
      const int n = w.n;
      const int a0 = w.a[0], a1 = w.a[1], b0 = w.b[0], b1 = w.b[1];
      const bool last_item = kSplit ? w.kind == 2 : n < 0;
      work_done<kSlots>(ms, 0, k, lane);
      if constexpr (kSplit) {
        ok = work_wait<kSlots>(ms, p, 1, k, abort_flag, kErrWaitMma);
        if (!ok) break;
        work_done<kSlots>(ms, 1, k, lane);
      }
      if (last_item) {
        ++k;
        break;
      }
      if (n == 0) continue;
      if (b0 > a0) ok = wait(&ms.q_full[0], qs0++);
      if (ok && b1 > a1) ok = wait(&ms.q_full[1], qs1++);
      if constexpr (C::kQInTmem) {
        // Q_0, Q_1 into TMEM once every MMA of the previous item retired (see
        // fwd_sm103a.cu)
        if (ok && items > 0) ok = wait(&ms.unit_done, items - 1);
        if (ok) {
          tc_fence_after();
#pragma unroll 1
          for (int t = 0; t < 2; ++t) {
            if (t ? b1 <= a1 : b0 <= a0) continue;
            const uint32_t base = tmem + t * kTileCols, q = desc_k + kQ0 + t * kTileDesc;
            tmem_cp_128x256b<kTQ + 0, 0>(base, q);
            tmem_cp_128x256b<kTQ + 8, 2>(base, q);
            tmem_cp_128x256b<kTQ + 16, 4>(base, q);
            tmem_cp_128x256b<kTQ + 24, 6>(base, q);
            mma_commit(&ms.q_empty[t]);
          }
        }
      }
      for (int j = 0; ok && j <= n; ++j) {
        const uint32_t ik = 2u * (tiles + j), iv = ik - 1u;
        const uint32_t bk = desc_k + (ik % kS) * kTileDesc, bv = desc_k + (iv % kS) * kTileDesc;
        if (j < n) ok = wait(&ms.kv_full[ik % kS], ik / kS);
        if (ok && j > 0) ok = wait(&ms.kv_full[iv % kS], iv / kS);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
          if (!ok) break;
          const int a = t ? a1 : a0, b = t ? b1 : b0;
          const bool pv = j > a && j <= b, qk = j >= a && j < b;
          const uint32_t last = (t ? steps1 : steps0) - 1u;  // the step whose P V is due
          if (pv) {
            if constexpr (kSplitScores<D, kCap, kBias>) {
              ok = wait(&ms.s_read[t], last);
              if (!ok) break;
              tc_fence_after();
              if (qk) issue_s(t, bk, 2);
            }
            ok = wait(&ms.p_full[t], last);
            if (!ok) break;
            tc_fence_after();
            issue_pv(t, bv, j - 1 > a ? 1u : 0u);
            if (j == b) mma_commit(&ms.o_done[t]);
            if (kSplitScores<D, kCap, kBias> && qk) issue_s(t, bk, 1);
          }
          if (qk) {
            if (!(kSplitScores<D, kCap, kBias> && pv)) issue_s(t, bk, 0);
            mma_commit(&ms.s_full[t]);
            if (t)
              ++steps1;
            else
              ++steps0;
            if (!C::kQInTmem && j == b - 1) mma_commit(&ms.q_empty[t]);
          }
        }
        if (!ok) break;
        if (j < n) mma_commit(&ms.kv_empty[ik % kS]);
        if (j > 0) mma_commit(&ms.kv_empty[iv % kS]);
      }
      if (!ok) break;
      if (C::kQInTmem) mma_commit(&ms.unit_done);
      ++items;
      tiles += n;
    }
    // ---- decode: the requests' own keys, a chain of its own per query tile.
    // The chains take turns, a tile each, so that one's softmax runs beside
    // the other's MMAs.  S reads Q from shared memory at D = 64 too: the bytes
    // of K and V set the pace here.
    if constexpr (kSplit) {
      const uint32_t ring = 2u * tiles;
      if constexpr (kHeads > 0) {
        // S^T = K Q^T of either run, whenever its K and Q are there and the team's S is
        // free; the teams multiply with V themselves.
        struct Chain {
          int k, left;     // next item; tiles left of this one
          uint32_t items;  // items taken: the next one's team = items % 2
          uint32_t n;      // S issued
          uint32_t s0, s1; // of them for either team
          bool over;
        };
        Chain cur = {k, 0, 0, 0, 0, 0, false}, other = cur;
        uint32_t idle = 0, t0 = 0;
        auto ready = [&](uint64_t* bar, uint32_t phase) {
          return warp_all(mbar_test(bar, phase & 1u));
        };
#pragma unroll 1
        for (int t = 0; !(cur.over && other.over); t ^= 1) {
          bool did = false;
          if (!cur.over) {
            const bool first = cur.left == 0;
            const int slot = cur.k % kSlots;
            const uint32_t team = (first ? cur.items : cur.items - 1u) & 1;
            const uint32_t used = team ? cur.s1 : cur.s0;
            const uint32_t ik = own_item<kS>(ring, false, t, cur.n);
            bool go = !first || ready(&ms.work_full[t][slot], cur.k / kSlots);
            int n = cur.left;
            if (go && first) {
              n = ms.work[t][slot].n;
              if (n < 0) {
                work_done<kSlots>(ms, t, cur.k, lane);
                cur.over = did = true;
                go = false;
              } else {
                go = ready(&ms.q2_full[t][team], cur.items >> 1);
              }
            }
            if (go && (used == 0 || ready(&ms.s2_read[t][team], used - 1)) &&
                ready(&ms.kv_full[ik % kS], ik / kS)) {
              tc_fence_after();
              SwapMma<D>::template s<kColS>(
                  tmem + t * kTileCols + team * kTeamCols, desc_k + (ik % kS) * kTileDesc,
                  desc_k + kQ0 + t * kTileDesc + team * (kTeamQ >> 4));
              mma_commit(&ms.s2_full[t][team]);
              mma_commit(&ms.kv_empty[ik % kS]);
              if (n == 1) mma_commit(&ms.q2_empty[t][team]);
              if (first) {
                work_done<kSlots>(ms, t, cur.k++, lane);
                ++cur.items;
              }
              if (team)
                ++cur.s1;
              else
                ++cur.s0;
              ++cur.n;
              cur.left = n - 1;
              did = true;
            }
          }
          const Chain next = other;
          other = cur;
          cur = next;
          // as mod_wait: give up on an abort or after the time limit
          idle = did ? 0 : idle + 1;
          if (idle && (idle & 255u) == 0u) {
            uint32_t now;
            asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(now));
            if (idle == 256u) t0 = now;
            const bool late = now - t0 > static_cast<uint32_t>(p.wait_limit_ns);
            if (!warp_all(!abort_set(abort_flag))) break;
            if (!warp_all(!late)) {
              abort_raise(abort_flag);
              if (lane == 0) atomicOr(p.err, kErrWaitMma);
              break;
            }
          }
        }
      } else {
        struct Chain {
          int k, left;      // next item; tiles left of this one
          int due;          // P V: 0 none; bit 0: due; 1: accumulate; 2: the item's last
          uint32_t v_item;  // ring item of its V
          uint32_t q, pv;   // Q taken, P V issued
          uint32_t n;       // S issued
          bool over;
        };
        Chain cur = {k, 0, 0, 0, qs0, steps0, 0, false};
        Chain other = {k, 0, 0, 0, qs1, steps1, 0, false};
#pragma unroll 1
        for (int t = 0; ok && !(cur.over && other.over && !cur.due && !other.due); t ^= 1) {
          if (cur.due) {
            const uint32_t iv = cur.v_item;
            ok = wait(&ms.kv_full[iv % kS], iv / kS) && wait(&ms.p_full[t], cur.pv);
            if (!ok) break;
            ++cur.pv;
            tc_fence_after();
            issue_pv(t, desc_k + (iv % kS) * kTileDesc, (cur.due >> 1) & 1u);
            mma_commit(&ms.kv_empty[iv % kS]);
            if (cur.due & 4) mma_commit(&ms.o_done[t]);
            cur.due = 0;
          }
          if (!cur.over) {
            const bool first = cur.left == 0;
            if (first) {
              ok = work_wait<kSlots>(ms, p, t, cur.k, abort_flag, kErrWaitMma);
              if (!ok) break;
              cur.left = ms.work[t][cur.k % kSlots].n;
              work_done<kSlots>(ms, t, cur.k++, lane);
              cur.over = cur.left < 0;
              if (!cur.over) ok = wait(&ms.q_full[t], cur.q++);
            }
            if (!cur.over) {
              const uint32_t ik = own_item<kS>(ring, false, t, cur.n);
              ok = ok && wait(&ms.kv_full[ik % kS], ik / kS);
              if (!ok) break;
              tc_fence_after();
              issue_s_steps<D, false, kColS, kQ0, 0, 0>(tmem + t * kTileCols,
                                                        desc_k + t * kTileDesc,
                                                        desc_k + (ik % kS) * kTileDesc);
              mma_commit(&ms.s_full[t]);
              mma_commit(&ms.kv_empty[ik % kS]);
              const bool last = cur.left == 1;
              if (last) mma_commit(&ms.q_empty[t]);
              cur.v_item = own_item<kS>(ring, true, t, cur.n);
              ++cur.n;
              cur.due = 1 | (first ? 0 : 2) | (last ? 4 : 0);
              --cur.left;
            }
          }
          const Chain next = other;
          other = cur;
          cur = next;
        }
      }
    }
    // all issued MMAs retire before the CTA releases TMEM
    mma_commit(&ms.mma_done);
    drain_wait(&ms.mma_done, 0);
  } else {
    // =====================================================================
    // planning warps
    // =====================================================================
    reg_dealloc<kModRegOther<kSplit>>();
    Work w;
    bool ok = true;
    uint32_t ring = 0;  // ring items so far
    int k = 0;
    if constexpr (kSplit) {
      const int t = warp - kModWarpPlan;  // plans for this query tile
      plan_decode(p, t, lane, w, [&] {
        return work_publish<kSlots>(ms, p, t, k++, w, abort_flag, lane);
      });
    } else if (warp == kModWarpPlan) {
      w = plan_unit(p, static_cast<int>(blockIdx.x), ms.ranges[0], lane);
      for (;; ++k) {
        w.v_first = ring + 1u;
        w.v_last = ring + 2u * w.n - 1u;
        ok = work_publish<kSlots>(ms, p, 0, k, w, abort_flag, lane) &&
             work_publish<kSlots>(ms, p, 1, k, w, abort_flag, lane);
        if (!ok || w.n < 0) break;
        ring += 2u * w.n;
        // Ask for another item when the last loads of this one are issued, a few tiles
        // before its end: early enough to be planned in time, and so late that the
        // items, longest first, go to the CTAs that are done first.  (And once the one
        // before this is done, whose ranges[] the next takes.)
        ok = warp_all(mod_wait(&ms.item_loaded, k & 1, abort_flag, p.err, kErrWaitLoad,
                               p.wait_limit_ns));
        if (k >= 1)
          for (int t = 0; t < 2; ++t)
            ok = ok && warp_all(mod_wait(&ms.work_empty[t][(k - 1) % kSlots],
                                         ((k - 1) / kSlots) & 1, abort_flag, p.err, kErrWaitLoad,
                                         p.wait_limit_ns));
        if (!ok) break;
        mbar_arrive_expect_tx_elect(&ms.clc_full, 16);
        clc_try_cancel_elect(smem_u32(&ms.clc_resp), &ms.clc_full);
        if (!warp_all(mod_wait(&ms.clc_full, k & 1, abort_flag, p.err, kErrWaitLoad,
                                p.wait_limit_ns))) {
          drain_wait(&ms.clc_full, k & 1);
          break;
        }
        const int nu = clc_response_ctaid_x(smem_u32(&ms.clc_resp));
        fence_proxy_async_smem();
        __syncwarp();
        if (nu < 0)
          w.n = -1;
        else
          w = plan_unit(p, nu, ms.ranges[(k + 1) & 1], lane);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kModWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D, bool kSplit, bool kCap, bool kBias, int kHeads>
cudaError_t launch_one(const ModKernelParams& p, unsigned grid, int dev, cudaStream_t stream) {
  using C = Cfg<D, false>;
  auto kernel = mod_attn_kernel<D, kSplit, kCap, kBias, kHeads>;
  // the shared-memory opt-in is a per-device property of the function
  static std::atomic<bool> attr_done[64];  // zero-initialised: false
  cudaError_t e;
  if (!attr_done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    attr_done[dev].store(true, std::memory_order_release);
  }
  kernel<<<grid, kModThreads, C::kSmemBytes, stream>>>(p);
  return cudaGetLastError();
}

// The variant is the caller's request alone: what is not asked for is not computed.
// kHeads: query heads per KV head that a decode's threads hold, or 0: the heads are
// the rows.
template <int D, bool kSplit, int kHeads>
cudaError_t launch_variant(const ModKernelParams& p, unsigned grid, int dev,
                           cudaStream_t stream) {
  const bool cap = p.mod.cap_out > 0.f, bias = p.mod.slopes != nullptr;
  if (cap && bias) return launch_one<D, kSplit, true, true, kHeads>(p, grid, dev, stream);
  if (cap) return launch_one<D, kSplit, true, false, kHeads>(p, grid, dev, stream);
  if (bias) return launch_one<D, kSplit, false, true, kHeads>(p, grid, dev, stream);
  return launch_one<D, kSplit, false, false, kHeads>(p, grid, dev, stream);
}

}  // namespace
}  // namespace attn
