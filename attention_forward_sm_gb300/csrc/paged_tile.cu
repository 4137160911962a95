// Attention of many new tokens of each request over its paged cache: chunks of
// prompts, alone or beside single tokens.
//
// The rows of a (request, KV head) are its new tokens times the G query heads that
// share the head, token by token, so that K and V are read once for all of them; a
// tile is the 128 / G tokens that fit 128 rows.  A CTA works on two tiles (an item:
// 2 * (128 / G) tokens of one KV head) as in fwd_sm103a.cu, whose roles and barriers
// these are: S_t = Q_t K^T and O_t in tensor memory, sixteen softmax warps that write
// P_t over S_t, a warp that issues every tcgen05.mma, one that loads.
//
// Pages.  A key tile is 128 keys, one tensor copy per page (and 128 bytes of a row).
// What lies behind the last token may hold anything, and an unseen key's weight of 0
// times a NaN of V is none.  So the copy of the last page begins above the page, at a
// negative row, which fills with zeros: the page's tokens come to stand at the end of
// its rows (the mask knows), and pages behind it are copied from behind the last page
// there is, as zeros.
//
// Quantised pages come in as they are, and four warps turn them into f16 tiles next to
// the softmax (convert, below).
//
// Work is dealt out by keys: every item has a cost, its keys and a constant, the items
// of all requests make one line, and each CTA takes an equal stretch of it.  An item
// that is cut has a partial state in each CTA, which tile_merge_kernel joins.
// Bound by the tensor cores, 4 D flops per row and key, and the chain of a query tile
// (scores, softmax pass, products), two of which alternate.  32 heads on 8, D = 128: bf16,
// 2048 tokens behind 16001 350 to 380 us (with the power cap), of which 338 this kernel (1.7
// PFLOP/s, tensor pipe 74%) and 15 the joining; e4m3, 1024 behind 30000 407 us, 400 and
// 14, tensor pipe 55%, issue slots 55%: the conversion's instructions and 96 registers for
// the softmax warps.  Short chunks are bound by 6 us until the first product and 5 from one
// item to the next.
#include <math_constants.h>

#include <atomic>

#include "../../include/attn.h"
#include "fwd_tile.cuh"
#include "paged_plan.cuh"

namespace attn {
namespace {

constexpr int kWarpLoad = 16, kWarpMma = 17, kWarpLoadV = 18, kWarpConvert = 20;

template <int D, bool kQuant>
struct TileCfg {
  static constexpr int kConvert = 4;  // warps that convert
  static constexpr int kThreads = kQuant ? 768 : 640;
  // setmaxnreg: 4 softmax warpgroups and 1 or 2 others, out of what the launch gets
  static constexpr uint32_t kRegSoftmax = kQuant ? 96 : 104, kRegOther = kQuant ? 48 : 64;
  static constexpr int kReaders = kQuant ? 21 : 17;  // of an item, besides the loader
  static constexpr int kTileBytes = kBM * D * 2, kChunks = D / 64;
  static constexpr int kStages = D == 128 ? 4 : 8;
  // Quantised tiles in a ring of their own, their scales (K: and those of V) behind.
  // D = 128: two, one of K and one of V; with four there would be room for three converted
  // ones, and K_j+1 would wait for K_j's place (6% slower).  D = 64 has room for six (16
  // requests of 30000 tokens with 8 of 32 heads on 8 each 307 -> 279 us, long chunks the same).
  static constexpr int kRaw = D == 128 ? 2 : 6, kRawBytes = kBN * D, kScaleBytes = 2 * kBN;
  static constexpr int kOffKV = 2 * kTileBytes;
  static constexpr int kOffRaw = kOffKV + kStages * kTileBytes;
  static constexpr int kOffScale = kOffRaw + (kQuant ? kRaw * kRawBytes : 0);
  static constexpr int kSmem = kOffScale + (kQuant ? kRaw * kScaleBytes : 0) + 1024;
  // bf16 operands, or f16 ones
  static constexpr uint32_t kTypes = kQuant ? (1u << 7 | 1u << 10) : 0;
  static constexpr uint32_t kIdescS = idesc_bf16_f32(128, kBN, false) & ~kTypes;
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, true) & ~kTypes;
  static constexpr uint32_t kColS0 = 0, kColS1 = 128, kColO0 = 256, kColO1 = 256 + D;
  static_assert(4 * 128 * kRegSoftmax + (kThreads - 512) * kRegOther <=
                    kThreads * (65536 / kThreads / 8 * 8),
                "register split");
};

struct Item {
  int row0, left;    // first dense row; tokens of the request from there on
  int before, len;   // keys in front of that token; tokens of the request
  int h, tiles;      // KV head; query tiles with rows, 0: no item
  int tile0, tile1;  // key tiles
  int slot, b;       // partial state, -1: none; request
};

// The items of a CTA's stretch of the line, one after the other.
struct CostWalk {
  const CostPlan& plan;
  const CostPlace& at;
  CostItem item;
  int b, blocks;
  bool fresh = true;
  __device__ CostWalk(const CostPlan& plan, const CostPlace& at) : plan(plan), at(at), b(at.b) {
    if (b < plan.c.B && at.first < at.end) {
      item = plan.item(at);
      blocks = plan.items(request_rows(plan.c, b).n);
    } else {
      b = plan.c.B;
    }
  }
  // The next part with key tiles; slot: of its partial state, 0 or 1, or -1.
  __device__ bool next(Item* it, int* slot) {
    while (b < plan.c.B) {
      if (!fresh) {
        const long long x0 = item.x0 + item.cost;
        if (x0 >= at.end) break;
        int h = item.h, j = item.j + 1;
        if (j == blocks) {
          j = 0;
          ++h;
        }
        if (h == plan.c.Hkv) {
          h = 0;
          do ++b;
          while (b < plan.c.B && request_rows(plan.c, b).n == 0);
          if (b == plan.c.B) break;
          blocks = plan.items(request_rows(plan.c, b).n);
        }
        item = plan.make(b, h, j, x0);
      }
      fresh = false;
      const int t0 = plan.cut(item, at.first - item.x0), t1 = plan.cut(item, at.end - item.x0);
      if (t0 >= t1) continue;
      *it = Item{item.row0, item.left, item.before, item.len, item.h,
                 item.left > plan.tokens / 2 ? 2 : 1, t0, t1, -1, b};
      *slot = t0 == 0 && t1 == item.n_kv ? -1 : t0 == 0;
      return true;
    }
    return false;
  }
};

// What the softmax needs to have a key tile's scales one by one.
struct FarKeys {
  uint2 by;             // as scale bytes, or kScaleEach
  uint4 silent;         // rows of V that are zeros, NaN or not there (row 4 l + i: bit l of word i)
  int b, h, len, key0;  // request, KV head, its tokens, the tile's first key
};

template <bool kQuant>
struct TileShared {
  uint64_t q_full[2], q_ready[2];    // per item of query tile t (ready: converted to f16)
  uint64_t q_empty;                  // per item
  uint64_t s_full[2], p_full[2];     // per key tile of query tile t
  uint64_t o_done[2];                // per item of query tile t
  uint64_t mma_done;
  uint64_t kv_full[8], kv_empty[8];
  uint64_t raw_full[6], raw_empty[6];
  uint64_t item_full[2], item_empty[2];
  Item item[2];
  uint32_t raw_bad[6];  // copies of the tile whose page is out of range, a bit each
  // Quantised: what the converted K and V of a key tile are to be multiplied by, 2^a and 2^e, as
  // 2^a, E = e + kWeightLift, 2^-E and whether it is in `far` how (then 1, and where V's scales
  // are each key's own kWeightLift and 0): of the tiles i, i + 8, ...; the converting warps
  // are three ahead at most.
  float4 kv_scale[8];
  FarKeys far[8];
  CostShared plan;
  uint32_t tmem_base;
  int abort_flag;
};

// In place of the scale byte of a tile: its codes were converted as they are, and each key has
// its own.
constexpr uint32_t kScaleEach = 0;
// Scales so far apart at most are brought under the largest one.  K: a code is a multiple of
// 2^-9, and f16 holds multiples of 2^-24.  V: the tile's weights are over that of a
// row with the largest scale, which need not have any, and end at 2^-24 too.
constexpr uint32_t kScaleSpanK = 14, kScaleSpanV = 8;
// The sum of a tile's 2^x is taken from its weights, of 2^(x + e), while e is this near 0: then
// none is lost under another tile's reference.
constexpr uint32_t kScaleReachV = 48;

// The factor 2^(scale - most) of a row among those of a tile, as f16; 1 where each key has its
// own scale, NaN for a row that stands for it.  (Further below there are only zeros.)
__device__ __forceinline__ uint32_t f16_factor(uint32_t scale, uint32_t most) {
  const uint32_t d = most == kScaleEach ? 0 : most - scale;
  return scale == kScaleNan ? 0x7FFFu : d <= kScaleSpanK ? (15 - d) << 10 : 0u;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}

// The warps that make f16 operands K_0, V_0, K_1 ... of codes.  f16 holds every code, and
// turning codes into it is one instruction for two, where bf16 takes five: with bf16
// the schedulers had no room for them next to the softmax (1024 tokens behind 30000, 32
// heads on 8, D 128: 460 us; f16 402).  A tile's values are over the largest of its scales,
// which the softmax puts back, or, where these lie far apart, over each key's own (see
// far_scores).  Q is converted by the softmax warps at an item's start.
template <int D, class C, class Shared, class Next>
__device__ __forceinline__ void convert(const PagedParams& p, Shared& ms, uint8_t* smem,
                                        uint32_t abort_flag, Next next_item) {
  constexpr int kThreads = 32 * C::kConvert;
  const int tid = threadIdx.x - kWarpConvert * 32, lane = threadIdx.x & 31;
  // A thread has the same 16 elements of every kStep-th row.  The lanes of a row's two
  // halves store their 16-byte pieces in opposite order, so that no two of eight
  // lanes meet in a bank.
  constexpr int kPieces = D / 16, kStep = kThreads / kPieces, kRounds = kBN / kStep;
  const int row0 = tid / kPieces, piece = tid % kPieces;
  const bool hi = piece >= kPieces / 2;
  uint8_t* const dst = smem + C::kOffKV + (piece >> 2) * (kBN * 128) + row0 * 128;
  const uint32_t at0 = ((((piece * 2) & 7) ^ (row0 & 7)) << 4) ^ (hi ? 16u : 0u);
  auto one = [&](uint8_t* to, const uint4& x, uint32_t f) {
    const uint32_t w[4] = {hi ? x.z : x.x, hi ? x.w : x.y, hi ? x.x : x.z, hi ? x.y : x.w};
    uint32_t y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = mul_f16x2(e4m3_lo(w[i]), f);
      y[2 * i + 1] = mul_f16x2(e4m3_hi(w[i]), f);
    }
    *reinterpret_cast<uint4*>(to + at0) = make_uint4(y[0], y[1], y[2], y[3]);
    *reinterpret_cast<uint4*>(to + (at0 ^ 16u)) = make_uint4(y[4], y[5], y[6], y[7]);
  };
  // The largest of a tile's scales, and whether all are within `span` of it and there is
  // nothing odd: then every factor is a normal f16 number.  Else only rows count that are
  // there and not NaN, nor zeros, whose scale says 2^0 and could leave nothing of the
  // others (of V also those of other tiles); landed() says that the codes are in place
  // (false: they never will be).  kScaleEach where those that count are more than `span`
  // apart, or `reach` from 2^0; silent: the others.
  auto largest = [&](const uint8_t* scales, const uint8_t* codes, bool whole, int rows, uint32_t bad,
                     bool of_v, bool* plain, uint32_t* most, uint4* silent, auto landed) {
    const uint32_t span = of_v ? kScaleSpanV : kScaleSpanK, reach = of_v ? kScaleReachV : 255u;
    const uint32_t w = reinterpret_cast<const uint32_t*>(scales)[lane];
    uint32_t s[4] = {w & 255u, w >> 8 & 255u, w >> 16 & 255u, w >> 24};
    *most = __reduce_max_sync(0xFFFFFFFFu, max(max(s[0], s[1]), max(s[2], s[3])));
    const uint32_t least = __reduce_min_sync(0xFFFFFFFFu, min(min(s[0], s[1]), min(s[2], s[3])));
    auto within = [&](uint32_t lo) {
      return *most - lo <= span && *most + reach >= 127u && *most <= 127u + reach;
    };
    *plain = whole && *most != kScaleNan && within(least) &&
             !(of_v && least <= kScaleOfZeros && kScaleOfZeros <= *most);
    if (*plain) return true;
    bool zeros = false;
    uint32_t counts = 15;  // a bit for each of the lane's rows
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 4 * lane + i;
      if (s[i] == kScaleNan || row >= rows || (bad >> (row >> p.c.page_bits) & 1u))
        counts &= ~(1u << i);
      zeros = zeros || ((counts >> i & 1u) && s[i] == kScaleOfZeros);
    }
    if (__any_sync(0xFFFFFFFFu, zeros)) {
      if (!landed()) return false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t bits = s[i] == kScaleOfZeros ? 0u : ~0u;
#pragma unroll 1
        for (int at = 0; at < D; at += 16)  // (each lane begins elsewhere: other banks)
          bits |= or_of(*reinterpret_cast<const uint4*>(codes + (4 * lane + i) * D +
                                                        (at + 16 * lane) % D));
        if (!(bits & 0x7F7F7F7Fu)) counts &= ~(1u << i);
      }
    }
    uint32_t hi_scale = kScaleLeast, lo_scale = kScaleNan;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!(counts >> i & 1u)) continue;
      hi_scale = max(hi_scale, s[i]);
      lo_scale = min(lo_scale, s[i]);
    }
    *most = __reduce_max_sync(0xFFFFFFFFu, hi_scale);
    if (!within(min(__reduce_min_sync(0xFFFFFFFFu, lo_scale), *most))) {
      *most = kScaleEach;
      *silent = make_uint4(__ballot_sync(0xFFFFFFFFu, !(counts & 1u)),
                           __ballot_sync(0xFFFFFFFFu, !(counts & 2u)),
                           __ballot_sync(0xFFFFFFFFu, !(counts & 4u)),
                           __ballot_sync(0xFFFFFFFFu, !(counts & 8u)));
    }
    return true;
  };

  uint32_t raw = 0, raw_round = 0, slot = 0, round = 0, step = 0;
  Item it;
  for (uint32_t k = 0; next_item(k, &it, kErrWaitLoad); ++k) {
    const uint32_t n = 2u * static_cast<uint32_t>(it.tile1 - it.tile0);
    uint32_t most = 0, next_most = 0;  // the largest scale of the tile; of V of the same keys
    bool plain = false, next_plain = false;
    for (uint32_t i = 0; i < n; ++i) {
      if (!warp_all(mbar_wait(&ms.raw_full[raw], raw_round & 1, abort_flag, p.err, kErrWaitLoad,
                              p.wait_limit_ns)) ||
          !warp_all(mbar_wait(&ms.kv_empty[slot], (round & 1) ^ 1, abort_flag, p.err, kErrWaitLoad,
                              p.wait_limit_ns)))
        return;
      const bool of_v = i & 1;
      const int there = it.len - (it.tile0 + static_cast<int>(i >> 1)) * kBN;  // rows
      const uint32_t bad = ms.raw_bad[raw];
      const uint8_t* tile = smem + C::kOffRaw + raw * C::kRawBytes;
      const uint8_t* codes = tile + tid * 16;
      const uint8_t* scales = smem + C::kOffScale + raw * C::kScaleBytes;
      const bool whole = there >= kBN && !bad;
      if (!of_v) {
        // (V's raw tile is the next one, and comes in while this one is held)
        uint4 silent = make_uint4(0, 0, 0, 0);
        if (!largest(scales, tile, whole, there, bad, false, &plain, &most, &silent,
                     [] { return true; }) ||
            !largest(scales + kBN, tile + C::kRawBytes, whole, there, bad, true, &next_plain,
                     &next_most, &silent, [&] {
              return warp_all(mbar_wait(&ms.raw_full[raw + 1], raw_round & 1, abort_flag, p.err,
                                        kErrWaitLoad, p.wait_limit_ns));
            }))
          return;
        if (tid == 0) {
          const bool far_k = most == kScaleEach, far_v = next_most == kScaleEach;
          ms.kv_scale[step % 8] =
              make_float4(far_k || far_v ? 1.f : scale_value(most),
                          kWeightLift + (far_v ? 0.f : scale_exponent(next_most)),
                          far_v ? 0.f
                                : __uint_as_float((254u - static_cast<uint32_t>(kWeightLift) -
                                                   next_most) << 23),
                          far_k || far_v ? 1.f : 0.f);
          if (far_k || far_v)
            ms.far[step % 8] = FarKeys{make_uint2(most, next_most), silent, it.b, it.h, it.len,
                                       (it.tile0 + static_cast<int>(i >> 1)) * kBN};
        }
      } else {
        most = next_most;
        plain = next_plain;
        scales += kBN;
      }
      uint8_t* to = dst + slot * C::kTileBytes;
      if (!plain) {  // rows that are not there: zeros
#pragma unroll 1
        for (int q = 0; q < kRounds; ++q) {
          const int row = row0 + q * kStep;
          const bool none = row >= there || (bad >> (row >> p.c.page_bits) & 1u);
          const uint4 x = none ? make_uint4(0, 0, 0, 0)
                               : *reinterpret_cast<const uint4*>(codes + q * (kStep * D));
          one(to + q * (kStep * 128), x, none ? 0u : f16_factor(scales[row], most) * 0x10001u);
        }
      } else {
        // (their loads ahead of their stores, which might alias them)
        constexpr int kAhead = 2;
#pragma unroll
        for (int q = 0; q < kRounds; q += kAhead) {
          uint4 x[kAhead];
          uint32_t f[kAhead];
#pragma unroll
          for (int e = 0; e < kAhead; ++e) {
            x[e] = *reinterpret_cast<const uint4*>(codes + (q + e) * (kStep * D));
            f[e] = scales[row0 + (q + e) * kStep];
          }
#pragma unroll
          for (int e = 0; e < kAhead; ++e)
            one(to + (q + e) * (kStep * 128), x[e], (f[e] + 15u - most) * 0x04000400u);
        }
      }
      if (of_v) ++step;
      // (also of the reads: without it, or ahead of what uses their values, the next copy
      // may land before them)
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ms.kv_full[slot]);
        mbar_arrive(&ms.raw_empty[raw]);
      }
      if (++raw == C::kRaw) {
        raw = 0;
        ++raw_round;
      }
      if (++slot == C::kStages) {
        slot = 0;
        ++round;
      }
    }
  }
}

// A key tile whose scales lie far apart: a thread's 64 scores in tensor memory, from s_addr on,
// get K's scales, or, where V's are each key's own, x + e takes their place, and what is
// returned is the sum of 2^x over the reference that the tile gets.  Such tiles are few, and
// none of the softmax' registers are spent on them: a function of its own, which reads the
// scales where they are.  (1024 tokens behind 30000, 32 heads on 8, D 128, no such tile:
// without all this 401 us, so 407, as branches within the loop 415; 1106 if every tile's
// K has one, 2450 if V has, 2060 if V is zeros.)
__device__ __noinline__ float far_scores(const PagedArrays& c, const FarKeys& far, uint32_t s_addr,
                                         float row_scale, float m, int vis, int half) {
  const uint2 by = far.by;
  const float by_k = fmaxf(by.x == kScaleEach ? row_scale : row_scale * scale_value(by.x), 1e-37f);
  const uint32_t none[4] = {far.silent.x, far.silent.y, far.silent.z, far.silent.w};
  // 16 scale bytes from key on; 2^0 where there are none
  auto bytes = [&](const uint8_t* scales, int key) {
    const int* entry = c.table + static_cast<size_t>(far.b) * c.M + (key >> c.page_bits);
    const int id = key < far.len ? __ldcg(entry) : -1;
    if (static_cast<unsigned>(id) >= static_cast<unsigned>(c.P))
      return make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
    return __ldcg(reinterpret_cast<const uint4*>(
        scales + (static_cast<size_t>(id) * c.Hkv + far.h) * c.page + (key & (c.page - 1))));
  };
  const bool zeros = (none[0] & none[1] & none[2] & none[3]) == ~0u;  // all of V
  auto exponents = [&](int col, float (&e)[16]) {
    const uint4 x = zeros ? make_uint4(0, 0, 0, 0) : bytes(c.vscale, far.key0 + col);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const bool silent = none[i % 4] >> ((col + i) / 4) & 1u;
      e[i] = scale_exponent(silent ? kScaleLeast : w[i / 4] >> (8 * (i % 4)) & 255u);
    }
  };
  float top = -CUDART_INF_F;
#pragma unroll 1
  for (int i = 0; i < 64; i += 16) {
    const int col = half * 64 + i;
    uint32_t v[16];
    tmem_ld_pair16<64>(s_addr + i, v);
    if (by.x == kScaleEach) {
      const uint4 x = bytes(c.kscale, far.key0 + col);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int n = 0; n < 16; ++n)
        v[n] = __float_as_uint(__uint_as_float(v[n]) *
                               scale_value(w[n / 4] >> (8 * (n % 4)) & 255u));
    }
    if (by.y == kScaleEach) {
      float e[16];
      exponents(col, e);
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        const float x = fmaf(__uint_as_float(v[n]), by_k, e[n]);
        if (far.key0 + col + n < vis) top = fmaxf(top, x);
        v[n] = __float_as_uint(x);
      }
    }
    __syncwarp();
    tmem_st_pair16<64>(s_addr + i, v);
  }
  tmem_st_wait();
  float sum = 0.f;
  if (by.y == kScaleEach) {
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
    top += kWeightLift;  // (from here as the softmax will)
    if (top > m + (kWeightTop + kWeightRoom)) m = top - kWeightTop;
    const float from_m = m == -CUDART_INF_F ? 0.f : -m;
#pragma unroll 1
    for (int i = 0; i < 64; i += 16) {
      const int col = half * 64 + i;
      uint32_t v[16];
      float e[16];
      tmem_ld_pair16<64>(s_addr + i, v);
      exponents(col, e);
#pragma unroll
      for (int n = 0; n < 16; ++n)
        if (far.key0 + col + n < vis) sum += ex2_approx(__uint_as_float(v[n]) + (from_m - e[n]));
      __syncwarp();
    }
  }
  return sum;
}

template <int D, bool kQuant>
__global__ void __launch_bounds__(TileCfg<D, kQuant>::kThreads, 1)
    paged_tile_kernel(const __grid_constant__ PagedParams p) {
  using C = TileCfg<D, kQuant>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  __shared__ TileShared<kQuant> ms;
  static_assert(C::kSmem + sizeof(ms) <= 227 * 1024, "shared memory");
  const uint32_t abort_flag = smem_u32(&ms.abort_flag);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // A copy costs a loading warp some 80 cycles, and a key tile of small pages is 2 * 8 or
  // 2 * 16 of them: there V has a loading warp of its own (2048 tokens behind 16001, 32 heads
  // on 8, D = 128, pages of 16: 428 -> 345 us, of 32 381 -> 365; of 64 362 either way, and
  // quantised what two gave short chunks lost).
  const bool split = !kQuant && p.c.page <= 32;

  if (warp == kWarpLoad && lane == 0) {
    mbar_init(&ms.q_empty, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&ms.q_full[t], 1);
      mbar_init(&ms.q_ready[t], 8);
      mbar_init(&ms.s_full[t], 1);
      mbar_init(&ms.p_full[t], 8);
      mbar_init(&ms.o_done[t], 1);
      mbar_init(&ms.item_full[t], 1);
      mbar_init(&ms.item_empty[t], C::kReaders + split);
    }
    mbar_init(&ms.mma_done, 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&ms.kv_full[s], kQuant ? C::kConvert : 1);
      mbar_init(&ms.kv_empty[s], 1);
    }
    for (int s = 0; s < C::kRaw; ++s) {
      mbar_init(&ms.raw_full[s], 1);
      mbar_init(&ms.raw_empty[s], C::kConvert);
    }
    ms.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tmap_q);
    if (!kQuant) {
      tma_prefetch_desc(&p.tmap_k);
      tma_prefetch_desc(&p.tmap_v);
    }
  }
  if (warp == kWarpMma) {
    tmem_alloc(&ms.tmem_base, 512);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for what the stream did before
  const CostPlan plan(p.c, p.G, p.causal);
  const CostPlace at = plan.place<C::kThreads>(ms.plan, blockIdx.x, p.ctas);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = ms.tmem_base;

  // waits for item k; false when there is none
  auto next_item = [&](uint32_t k, Item* it, uint32_t site) -> bool {
    if (!warp_all(mbar_wait(&ms.item_full[k & 1], (k >> 1) & 1, abort_flag, p.err, site,
                            p.wait_limit_ns)))
      return false;
    *it = ms.item[k & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&ms.item_empty[k & 1]);
    return it->tiles > 0;
  };

  if (warp < 16) {
    // ---- softmax and epilogue: warps 8t .. 8t + 7 serve query tile t, two warps a
    // 32-lane quarter of tensor memory, two threads a row (64 keys of a tile each)
    reg_alloc<C::kRegSoftmax>();
    const int t = warp >> 3;
    const int lbase = (warp & 3) * 32 + ((warp >> 2) & 1) * 16;
    const int r = lbase + (lane & 15);  // row within the tile
    const int c = lane >> 4;            // half of the row's keys
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(lbase) << 16);
    const uint32_t s_addr = lane_addr + (t ? C::kColS1 : C::kColS0);
    const uint32_t o_addr = lane_addr + (t ? C::kColO1 : C::kColO0);
    const int per_tile = kBM / p.G;                // tokens of a tile
    const int token = t * per_tile + r / p.G;      // of the item
    const bool in_tile = r < per_tile * p.G;
    uint32_t step = 0, done = 0;  // key tiles and items of query tile t so far
    [[maybe_unused]] uint32_t all_steps = 0;  // key tiles of the CTA
    Item it;
    for (uint32_t k = 0; next_item(k, &it, kErrWaitSoftmax); ++k) {
      const uint32_t steps = all_steps;
      if constexpr (kQuant) all_steps += static_cast<uint32_t>(it.tile1 - it.tile0);
      if (t >= it.tiles) continue;
      const bool real = in_tile && token < it.left;
      // keys that the row sees, and that every row of the tile does
      const int vis = !real ? 0 : p.causal ? min(it.len, it.before + token + 1) : it.len;
      const int all_see = p.causal ? min(it.len, it.before + t * per_tile + 1) : it.len;
      // the last page's tokens stand `shift` rows further down from key `cut` on
      const int cut = kQuant ? 0 : max(it.len - 1, 0) & -p.c.page;
      const int shift = kQuant ? 0 : cut + p.c.page - it.len;
      float m = -CUDART_INF_F, l = 0.f;
      bool ok = true;
      [[maybe_unused]] float row_scale = p.scale_log2;
      if constexpr (kQuant) {
        // Q to f16, a thread's half of its row: over a power of two that makes the row's
        // largest element 1 to 2, exact but below 2^-14, where a step is 2^-24
        if (!warp_all(mbar_wait(&ms.q_full[t], done & 1, abort_flag, p.err, kErrWaitSoftmax,
                                p.wait_limit_ns)))
          break;
        uint8_t* q = smem + t * C::kTileBytes + (D == 128 ? c * (kBM * 128) : 0) + r * 128;
        constexpr int kPieces = D / 16;  // of 16 bytes in half a row
        auto at = [&](int i) {
          return reinterpret_cast<uint4*>(q + (((D == 128 ? i : kPieces * c + i) ^ (r & 7)) << 4));
        };
        uint4 x[kPieces];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          x[i] = *at(i);
          top = max(top, max(max(bf16x2_top(x[i].x), bf16x2_top(x[i].y)),
                             max(bf16x2_top(x[i].z), bf16x2_top(x[i].w))));
        }
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
        const uint32_t e = min(max(top >> 23, 1u), 253u);
        row_scale *= __uint_as_float(e << 23);
        const float inv = __uint_as_float((254u - e) << 23);
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          *at(i) = make_uint4(bf16x2_to_f16x2(x[i].x, inv), bf16x2_to_f16x2(x[i].y, inv),
                              bf16x2_to_f16x2(x[i].z, inv), bf16x2_to_f16x2(x[i].w, inv));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.q_ready[t]);
      }
      for (int j = it.tile0; j < it.tile1; ++j, ++step) {
        if (!warp_all(mbar_wait(&ms.s_full[t], step & 1, abort_flag, p.err, kErrWaitSoftmax,
                                p.wait_limit_ns))) {
          ok = false;
          break;
        }
        tc_fence_after();
        float s[64];
        [[maybe_unused]] float4 by;
        [[maybe_unused]] float by_row = row_scale;
        [[maybe_unused]] float each_sum = 0.f;
        if constexpr (kQuant) {
          // (there since S is: its operands were converted before)
          const uint32_t tile = (steps + static_cast<uint32_t>(j - it.tile0)) % 8;
          // (in two: the launch's 80 registers do not hold 64 results of one instruction)
          uint32_t sr[2][32];
          tmem_ld_pair32_start<64>(s_addr, sr[0]);
          tmem_ld_pair32_start<64>(s_addr + 32, sr[1]);
          by = ms.kv_scale[tile];
          if (__builtin_expect(by.w != 0.f, 0)) {
            tmem_ld_finish(sr[0]);  // (what has come is not used)
            tmem_ld_finish(sr[1]);
            each_sum = far_scores(p.c, ms.far[tile], s_addr, row_scale, m, vis, c);
            if (by.z == 0.f) by_row = 1.f;
            tmem_ld_pair32_start<64>(s_addr, sr[0]);
            tmem_ld_pair32_start<64>(s_addr + 32, sr[1]);
          }
          tmem_ld_finish(sr[0]);
          tmem_ld_finish(sr[1]);
#pragma unroll
          for (int i = 0; i < 64; ++i) s[i] = __uint_as_float(sr[i / 32][i % 32]);
        } else {
          uint32_t sr[64];
          tmem_ld_pair64<64>(s_addr, sr);
#pragma unroll
          for (int i = 0; i < 64; ++i) s[i] = __uint_as_float(sr[i]);
        }
        if ((j + 1) * kBN > all_see) {
          // columns [0, end) and [from, to) of this thread's are visible
          const int col0 = j * kBN + c * 64;
          const bool moved = shift > 0 && (j + 1) * kBN > cut;
          const int end = (moved ? min(cut, vis) : vis) - col0;
          const int from = moved ? cut + shift - col0 : 64;
          const int to = vis + shift - col0;
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i >= end && (i < from || i >= to)) s[i] = -CUDART_INF_F;
        }
        float mx;
        {
          float a0 = fmaxf(s[0], s[1]), a1 = fmaxf(s[2], s[3]);
          float a2 = fmaxf(s[4], s[5]), a3 = fmaxf(s[6], s[7]);
#pragma unroll
          for (int i = 8; i < 64; i += 8) {
            a0 = max3f(a0, s[i], s[i + 1]);
            a1 = max3f(a1, s[i + 2], s[i + 3]);
            a2 = max3f(a2, s[i + 4], s[i + 5]);
            a3 = max3f(a3, s[i + 6], s[i + 7]);
          }
          mx = max3f(a0, a1, fmaxf(a2, a3));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
        }
        // Quantised, the tile's K and V are to be multiplied by 2^a and 2^e: scores by 2^a,
        // and the weights stand for 2^(x + e), with the maximum of x + e; the sum is of 2^x
        // (with the references of kWeightTop).
        float scale = p.scale_log2;
        [[maybe_unused]] float e = 0.f, sum_scale = 1.f;
        if constexpr (kQuant) {
          // (never 0, as scale_log2: the product of a row of zeros and the smallest of scales)
          scale = fmaxf(by_row * by.x, 1e-37f);
          e = by.y;
          sum_scale = by.z;
        }
        float m_tile = mx * scale;  // (scale > 0)
        if constexpr (kQuant) m_tile += e;
        float alpha = 1.f;
        constexpr float kTop = kQuant ? kWeightTop : 0.f;
        if (m_tile > m + (kQuant ? kTop + kWeightRoom : 8.f)) {  // a stale maximum is as good
          const float2 f = ex2_factors<kQuant>(m - (m_tile - kTop));  // up to there
          alpha = f.x * f.y;                                          // 0 the first time
          m = m_tile - kTop;
          if constexpr (kQuant) l = l * f.x * f.y;
        }
        // p = 2^(s * scale - m); a row that has seen nothing keeps m = -inf: its
        // scores are -inf and stay it next to a reference of 0
        const float neg_m = (m == -CUDART_INF_F ? 0.f : -m) + (kQuant ? e : 0.f);
        const uint64_t scale2 = f32x2(scale, scale);
        const uint64_t negm2 = f32x2(neg_m, neg_m);
        uint64_t acc0 = f32x2(0.f, 0.f), acc1 = acc0;
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          float x0, x1, x2, x3;
          unpack_f32x2(fma_f32x2(f32x2(s[i], s[i + 1]), scale2, negm2), x0, x1);
          unpack_f32x2(fma_f32x2(f32x2(s[i + 2], s[i + 3]), scale2, negm2), x2, x3);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          const float p2 = ex2_approx(x2), p3 = ex2_approx(x3);
          acc0 = add_f32x2(acc0, f32x2(p0, p1));
          acc1 = add_f32x2(acc1, f32x2(p2, p3));
          pk[i / 2] = kQuant ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
          pk[i / 2 + 1] = kQuant ? pack_f16x2(p2, p3) : pack_bf16x2(p2, p3);
        }
        float u0, u1;
        unpack_f32x2(add_f32x2(acc0, acc1), u0, u1);
        l = kQuant ? l + fmaf(u0 + u1, sum_scale, each_sum) : fmaf(l, alpha, u0 + u1);
        // Rescale O_t where a maximum moved: every product of earlier key tiles has
        // retired (issued before the S_t that woke this warp), that of this one waits.
        if (j > it.tile0 && __any_sync(0xFFFFFFFFu, alpha != 1.f)) {
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
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.p_full[t]);
      }
      // ---- epilogue: O / l and LSE, or the partial state
      ok = ok && warp_all(mbar_wait(&ms.o_done[t], done & 1, abort_flag, p.err, kErrWaitCorr,
                                    p.wait_limit_ns));
      if (!ok) break;
      ++done;
      tc_fence_after();
      const float l_row = l + __shfl_xor_sync(0xFFFFFFFFu, l, 16);
      const bool whole = it.slot < 0;
      const float inv = !whole ? 1.f : l_row == 0.f ? 0.f : (kQuant ? kWeightUnit : 1.f) / l_row;
      const size_t out_row = static_cast<size_t>(it.row0 + token) * p.Hq + it.h * p.G + r % p.G;
      const size_t part_row = static_cast<size_t>(max(it.slot, 0)) * (2 * kBM) + t * kBM + r;
#pragma unroll
      for (int kk = 0; kk < D / 64; ++kk) {
        uint32_t v[32];
        tmem_ld_pair32<D / 2>(o_addr + kk * 32, v);
        const int col = c * (D / 2) + kk * 32;
        if (!real) continue;
        if (whole) {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + out_row * D + col;
#pragma unroll
          for (int g = 0; g < 2; ++g, dst += 16) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              w[i] = pack_bf16x2(__uint_as_float(v[16 * g + 2 * i]) * inv,
                                 __uint_as_float(v[16 * g + 2 * i + 1]) * inv);
            if ((reinterpret_cast<uintptr_t>(p.o) & 31) == 0) {
              st_global_v8(dst, w);
            } else {
              st_global_v4_evict_first(dst, w[0], w[1], w[2], w[3]);
              st_global_v4_evict_first(dst + 8, w[4], w[5], w[6], w[7]);
            }
          }
        } else {
          // (whole sectors)
#pragma unroll
          for (int g = 0; g < 4; ++g) st_global_v8(p.part_o + part_row * D + col + 8 * g, v + 8 * g);
        }
      }
      if (c == 0 && real) {
        if (whole)
          p.lse[out_row] =
              l_row == 0.f ? -CUDART_INF_F : (m + log2f(l_row)) * 0.69314718055994530942f;
        else
          p.part_ml[part_row] = make_float2(m, l_row);
      }
    }
  } else if (warp == kWarpLoad || (!kQuant && warp == kWarpLoadV)) {
    // ---- the plan's items, their Q tiles, and K_j, V_j through the ring
    reg_dealloc<C::kRegOther>();
    constexpr uint32_t kRing = kQuant ? C::kRaw : C::kStages;
    static_assert(kRing % 2 == 0, "K and V have places of their own");
    uint64_t* const full = kQuant ? ms.raw_full : ms.kv_full;
    uint64_t* const empty = kQuant ? ms.raw_empty : ms.kv_empty;
    const int page = p.c.page, page_bits = p.c.page_bits;
    const int boxes = kBN >> page_bits;
    const int per_tile = kBM / p.G;
    const uint64_t policy = l2_policy_evict_last();
    uint32_t k = 0;                      // items
    uint32_t q_loads = 0, q_loads1 = 0;  // of query tiles 0 and 1
    const uint32_t first = !kQuant && warp == kWarpLoadV, every = split ? 2 : 1;  // tiles that it loads
    uint32_t slot = first, round = 0;  // next place in the ring
    // Q of item k, once the item before has used its own
    auto load_q = [&](const Item& it) -> bool {
      if (k > 0 && !warp_all(mbar_wait(&ms.q_empty, (k - 1) & 1, abort_flag, p.err, kErrWaitLoad,
                                       p.wait_limit_ns)))
        return false;
      for (int t = 0; t < it.tiles; ++t) {
        mbar_arrive_expect_tx_elect(&ms.q_full[t], static_cast<uint32_t>(per_tile * p.G * D * 2));
        for (int ch = 0; ch < C::kChunks; ++ch)
          tma_load_4d_elect(smem + t * C::kTileBytes + ch * (kBM * 128), &p.tmap_q, &ms.q_full[t],
                            ch * 64, 0, it.h, it.row0 + t * per_tile, l2_policy_evict_first());
      }
      ++q_loads;
      q_loads1 += it.tiles > 1;
      return true;
    };
    auto load_tiles = [&](const Item& it) -> bool {
      int pbase = -256, ids = 0;
      const uint32_t n = 2u * static_cast<uint32_t>(it.tile1 - it.tile0);
      for (uint32_t i = first; i < n; i += every) {
        const bool of_v = i & 1;
        const int key0 = (it.tile0 + static_cast<int>(i >> 1)) * kBN;
        // copy `box` of the tile: page and rows (lane l holds entry pbase + l of the table)
        if ((key0 >> page_bits) < pbase || (key0 >> page_bits) + boxes > pbase + 32) {
          pbase = key0 >> page_bits;
          ids = pbase + lane < p.c.M
                    ? p.c.table[static_cast<size_t>(it.b) * p.c.M + pbase + lane]
                    : -1;
        }
        const int box = kQuant ? lane : lane / C::kChunks;
        const int key = key0 + (box << page_bits);
        const int id = __shfl_sync(0xFFFFFFFFu, ids, ((key >> page_bits) - pbase) & 31);
        const bool mine = box < boxes;
        const bool there = key < it.len;
        const bool good = static_cast<unsigned>(id) < static_cast<unsigned>(p.c.P);
        const uint32_t bad = __ballot_sync(0xFFFFFFFFu, mine && there && !good);
        if (bad && lane == 0) atomicOr(p.err, kErrPage);
        if (!warp_all(mbar_wait(&empty[slot], (round & 1) ^ 1, abort_flag, p.err, kErrWaitLoad,
                                p.wait_limit_ns)))
          return false;
        if constexpr (kQuant) {
          const bool copy = mine && there && good;
          const int rows = min(page, it.len - key);
          const int scales = of_v ? 1 : 2;  // with K, V's too
          uint32_t bytes = copy ? static_cast<uint32_t>(rows * D + scales * page) : 0;
          bytes = __reduce_add_sync(0xFFFFFFFFu, bytes);
          if (lane == 0) {
            ms.raw_bad[slot] = bad;
            mbar_arrive_expect_tx(&full[slot], bytes);
          }
          __syncwarp();
          if (copy) {
            const size_t from = (static_cast<size_t>(id) * p.c.Hkv + it.h) * page;
            const uint8_t* src = static_cast<const uint8_t*>(of_v ? p.c.vpages : p.c.kpages);
            bulk_copy(smem + C::kOffRaw + slot * C::kRawBytes + box * page * D, src + from * D,
                      static_cast<uint32_t>(rows * D), &full[slot], policy);
            uint8_t* to = smem + C::kOffScale + slot * C::kScaleBytes + (box << page_bits);
            if (!of_v)
              bulk_copy(to, p.c.kscale + from, static_cast<uint32_t>(page), &full[slot], policy);
            bulk_copy(to + kBN, p.c.vscale + from, static_cast<uint32_t>(page), &full[slot],
                      policy);
          }
        } else {
          mbar_arrive_expect_tx_elect(&full[slot], C::kTileBytes);
          if (mine) {
            const int z = there && good ? id * p.c.Hkv + it.h : p.c.P * p.c.Hkv;
            const int y = min(it.len - key, page) - page;  // the tokens at the end of the rows
            const int ch = lane % C::kChunks;
            tma_load_4d(smem + C::kOffKV + slot * C::kTileBytes + ch * (kBN * 128) +
                            box * page * 128,
                        of_v ? &p.tmap_v : &p.tmap_k, &full[slot], 0, there ? y : 0, ch, z, policy);
          }
          __syncwarp();
        }
        slot += every;
        if (slot >= kRing) {
          slot -= kRing;
          ++round;
        }
        if (i == 0 && !load_q(it)) return false;
      }
      return true;
    };
    if (!kQuant && warp == kWarpLoadV) {
      Item it;
      while (split && next_item(k, &it, kErrWaitLoad) && load_tiles(it)) ++k;
    } else {
      CostWalk walk(plan, at);
      PagedCut cut = {};
      for (;; ++k) {
        Item it;
        int part = 0;
        const bool more = walk.next(&it, &part);
        if (!warp_all(mbar_wait(&ms.item_empty[k & 1], ((k >> 1) & 1) ^ 1, abort_flag, p.err,
                                kErrWaitLoad, p.wait_limit_ns)))
          break;
        if (!more) it.tiles = 0;
        if (more && part == 1) {  // the CTA's last item, which goes on in the next ones
          const long long end = walk.item.x0 + min(walk.item.cost,
                                                   kItemCost + walk.item.n_kv * 1ll * kTileKeys);
          unsigned last = blockIdx.x + 1;
          while (at.deal.start(last + 1) < end) ++last;
          cut = PagedCut{static_cast<int>(last - blockIdx.x) + 1, it.row0, it.left, it.h};
        }
        if (lane == 0) {
          it.slot = part < 0 ? -1 : 2 * static_cast<int>(blockIdx.x) + part;
          ms.item[k & 1] = it;
          mbar_arrive(&ms.item_full[k & 1]);
        }
        if (!more || !load_tiles(it)) break;
      }
      if (lane == 0) p.cuts[blockIdx.x] = cut;
    }
    if (abort_set(abort_flag)) {
      // copies in flight land before the CTA leaves: the last Q tiles, and the last round
      // of the ring
      if (q_loads > 0) drain_wait(&ms.q_full[0], (q_loads - 1) & 1);
      if (q_loads1 > 0) drain_wait(&ms.q_full[1], (q_loads1 - 1) & 1);
      for (uint32_t i = first; i < kRing; i += every) {
        if (i < slot)
          drain_wait(&full[i], round & 1);
        else if (round > 0)
          drain_wait(&full[i], (round - 1) & 1);
      }
    }
  } else if (warp == kWarpMma) {
    // ---- S_t = Q_t K_j^T, O_t += P_t V_j
    reg_dealloc<C::kRegOther>();
    constexpr uint32_t kTileDesc = C::kTileBytes >> 4;
    const uint32_t desc_k = sdesc_sw128_lo(smem_u32(smem + C::kOffKV), 16);
    constexpr uint32_t kQ0 = 0u - static_cast<uint32_t>(C::kOffKV >> 4), kQ1 = kQ0 + kTileDesc;
    constexpr uint32_t kVFromK = static_cast<uint32_t>(((kBM * 128) >> 4) - 1) << 16;
    auto issue_s = [&](int t, uint32_t slot) {
      const uint32_t b0 = desc_k + slot * kTileDesc;
      if (t)
        issue_s_rec<false, C::kColS1, kQ1, 0, 0, C::kIdescS, 0, D / 16>(tmem, desc_k, b0);
      else
        issue_s_rec<false, C::kColS0, kQ0, 0, 0, C::kIdescS, 0, D / 16>(tmem, desc_k, b0);
      mma_commit(&ms.s_full[t]);
    };
    auto issue_pv = [&](int t, uint32_t slot, uint32_t acc) {
      const uint32_t b0 = desc_k + slot * kTileDesc;
      if (t)
        issue_pv_rec<false, C::kColO1, C::kColS1, kVFromK, C::kIdescPV, 0>(tmem, b0, acc);
      else
        issue_pv_rec<false, C::kColO0, C::kColS0, kVFromK, C::kIdescPV, 0>(tmem, b0, acc);
    };
    uint32_t p_step[2] = {0, 0}, q_step1 = 0;  // P tiles waited for, items with query tile 1
    uint32_t slot = 0, round = 0;
    auto wait_kv = [&]() -> bool {
      return warp_all(mbar_wait(&ms.kv_full[slot], round & 1, abort_flag, p.err, kErrWaitMma,
                                p.wait_limit_ns));
    };
    auto advance = [&]() {
      if (++slot == C::kStages) {
        slot = 0;
        ++round;
      }
    };
    auto wait_p = [&](int t) -> bool {
      const uint32_t step = t ? p_step[1]++ : p_step[0]++;
      if (!warp_all(mbar_wait(&ms.p_full[t], step & 1, abort_flag, p.err, kErrWaitMma,
                              p.wait_limit_ns)))
        return false;
      tc_fence_after();
      return true;
    };
    Item it;
    bool ok = true;
    for (uint32_t k = 0; ok && next_item(k, &it, kErrWaitMma); ++k) {
      const int tiles = it.tiles, n = it.tile1 - it.tile0;
      // ring order K_0 V_0 K_1 V_1 ...; S of key tile i + 1 goes out with P V of tile i
      uint32_t v_slot = 0;
      for (int i = 0; i < n && ok; ++i) {
        ok = wait_kv();  // K_i
        if (!ok) break;
        tc_fence_after();
        const uint32_t k_slot = slot;
        for (int t = 0; t < tiles && ok; ++t) {
          if (i > 0) {
            ok = wait_p(t);
            if (!ok) break;
            issue_pv(t, v_slot, i > 1 ? 1u : 0u);
          } else {
            const uint32_t q_phase = (t ? q_step1++ : k) & 1;  // (tile 0 is in every item)
            ok = warp_all(mbar_wait(kQuant ? &ms.q_ready[t] : &ms.q_full[t], q_phase, abort_flag,
                                    p.err, kErrWaitMma, p.wait_limit_ns));
            if (!ok) break;
            tc_fence_after();
          }
          issue_s(t, k_slot);
        }
        if (!ok) break;
        mma_commit(&ms.kv_empty[k_slot]);
        if (i > 0) mma_commit(&ms.kv_empty[v_slot]);
        advance();
        ok = wait_kv();  // V_i
        v_slot = slot;
        advance();
      }
      if (!ok) break;
      mma_commit(&ms.q_empty);
      tc_fence_after();
      for (int t = 0; t < tiles && ok; ++t) {
        ok = wait_p(t);
        if (ok) {
          issue_pv(t, v_slot, n > 1 ? 1u : 0u);
          mma_commit(&ms.o_done[t]);
        }
      }
      if (ok) mma_commit(&ms.kv_empty[v_slot]);
    }
    // all MMAs retire before the CTA gives tensor memory back
    mma_commit(&ms.mma_done);
    drain_wait(&ms.mma_done, 0);
  } else {
    reg_dealloc<C::kRegOther>();
    if constexpr (kQuant) {
      if (warp >= kWarpConvert) convert<D, C>(p, ms, smem, abort_flag, next_item);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partial states of the items that were cut: block (c, y) some rows of the one
// whose first part CTA c has, a warp each.  (Requests of 1 to 500 tokens behind 64 to 6000:
// with 8 blocks an item 37.9 us in all, with 16 34.8, 32 34.5; long chunks all the same.)
constexpr int kMergeSplit = 16;

template <int D, bool kQuant>
__global__ void __launch_bounds__(256) tile_merge_kernel(const __grid_constant__ PagedParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PagedCut cut = p.cuts[blockIdx.x];
  if (cut.parts == 0) return;
  const int per_tile = kBM / p.G, in_tile = per_tile * p.G;
  const int rows = min(2 * per_tile, cut.left) * p.G;
  for (int i = static_cast<int>(blockIdx.y) * 8 + warp; i < rows; i += 8 * kMergeSplit) {
    const int t = i / in_tile, r = t * kBM + i % in_tile;
    auto state = [&](int k) {
      return (static_cast<size_t>(blockIdx.x + k) * 2 + (k == 0)) * (2 * kBM) + r;
    };
    State<D, kQuant> sum;
    const float top = sum.join(p, cut.parts, lane, state);
    sum.finish(p, cut.row0 + i / p.G, cut.h * p.G + i % p.G, top, lane);
  }
}

template <int D, bool kQuant>
cudaError_t launch_tile(const PagedParams& p, int dev, cudaStream_t stream) {
  using C = TileCfg<D, kQuant>;
  static std::atomic<bool> ready[64];
  if (!ready[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(paged_tile_kernel<D, kQuant>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    ready[dev].store(true, std::memory_order_release);
  }
  if (cudaError_t e = launch_overlapped(paged_tile_kernel<D, kQuant>, dim3(p.ctas), C::kThreads,
                                        C::kSmem, stream, p))
    return e;
  if (p.ctas < 2) return cudaSuccess;
  // (the last CTA's items end there)
  return launch_overlapped(tile_merge_kernel<D, kQuant>, dim3(p.ctas - 1, kMergeSplit), 256, 0,
                           stream, p);
}

}  // namespace

size_t paged_tile_state(const PagedParams& p) { return static_cast<size_t>(p.ctas) * 2 * 2 * kBM; }

cudaError_t launch_paged_tile(const PagedParams& p, int dev, cudaStream_t stream) {
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (p.c.D == 128)
    return p.c.quant ? launch_tile<128, true>(p, dev, stream)
                     : launch_tile<128, false>(p, dev, stream);
  return p.c.quant ? launch_tile<64, true>(p, dev, stream) : launch_tile<64, false>(p, dev, stream);
}

}  // namespace attn
