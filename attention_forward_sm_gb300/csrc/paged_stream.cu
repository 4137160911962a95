// Attention of a few new tokens of each request over its paged cache: single tokens
// (decode) and a handful of drafted ones.
//
// The rows of a (request, KV head) are its new tokens times the G query heads that
// share the head, at most 8 NT per block of rows; all of them use every key that is
// read, so a call is bound by reading the cache once.  The keys of all blocks,
// 64 to a unit, make one long sequence of units, which is dealt out evenly among the
// CTAs (one or two per SM): a request of any length among any others costs its bytes.  A
// block that ends up in several CTAs has a partial state (maximum, sum, O) in each; the
// warp that is the last to store its part of a row joins them, in the CTAs' order.
//
// A CTA is one to three loading warps and two or three teams of four computing ones around a
// ring of stages, one unit each: K and V of 64 keys by tensor copies, a box per page or
// 16 whole rows of 256 bytes.  The teams take units in turn, a warp 16 keys of each.
// Rows are few, so the keys are the rows of the products (mma.sync m16n8k16):
//   S^T [16 keys, 8 rows] = K [16, D] Q^T,   O^T [D, 8 rows] += V^T [D, 16] P^T.
// A tcgen05.mma has at least 64 rows of one operand in shared memory or TMEM and
// would take the keys through either; here they go from shared memory straight into
// registers, where e4m3 codes become f16 on the way.  Which key and which
// dimension a thread's piece of an operand stands for is free as long as both
// operands agree, and chosen so that every load is 16 bytes of a swizzled row
// without bank conflicts: row i of a 16-key block is key block_key(i), and a thread
// has whole 16-byte pieces of the keys' rows.  P^T is S^T transposed within a warp
// (movmatrix).
//
// Measured, D = 128: 8 requests of 500 to 65536 tokens, 32 heads on 8, bf16 79 us, 6.7 TB/s;
// 64 of 16 to 12000, 64 heads on 8, e4m3 51 us, 4.9 TB/s (issue slots 50%; of a short call like
// this one 3.5 us go by until the first keys are there and some 5 at the end on the
// last parts); 16 of 100 to 16384 with 4 tokens each, bf16 45 us, 5.2 TB/s.
#include <math_constants.h>

#include <algorithm>
#include <atomic>

#include "../../include/attn.h"
#include "fwd_tile.cuh"
#include "paged_plan.cuh"

namespace attn {
namespace {

// One unit in the ring, as a loading warp describes it.
struct Unit {
  int flags, b, h, block;  // of kUnit..; request, KV head, block of rows
  int key0, len, slot;     // first key; tokens in the cache; partial state, -1: none
  int cta0, parts;         // where the block's first part is; how many there are
  int row0, rows;          // first row of the dense tensors; new tokens
};
constexpr int kUnitFirst = 1, kUnitLast = 2, kUnitEnd = 4;  // a team's first and last of an
                                                            // item; there are no more

template <int D, bool kQuant, int NT>
struct StreamCfg {
  // Quantised, 9 to 16 rows: latencies are the bound, and three teams hide more of them.  Their
  // 128 registers a thread hold no queries, which are in shared memory (16 requests of 30000
  // tokens 229 -> 198 us, 64 of 7000 225 -> 197; 200 both with the weights' present range).
  static constexpr bool kSharedQ = kQuant && NT == 2;
  static constexpr int kTeams = kSharedQ ? 3 : 2;
  static constexpr int kWarps = 4 * kTeams;  // computing
  // A copy costs a loading warp some 80 cycles, a unit more than 700, which is what brings a
  // quantised one in: there each team has a loader of its own (64 requests of 16 to 12000
  // tokens 57 -> 51 us).  bf16 units are on their way for 1400 (the same requests 77 us,
  // with two 82).
  static constexpr int kLoaders = kQuant ? kTeams : 1;
  static constexpr int kThreads = (kWarps + kLoaders) * 32;
  static constexpr int kRows = 8 * NT;
  static constexpr int kRowBytes = kQuant ? D : 2 * D;
  static constexpr int kTile = kUnitKeys * kRowBytes;  // K or V of a unit
  static constexpr int kScales = kQuant ? 2 * kUnitKeys : 0;
  static constexpr int kMerge = (kWarps - 4) * kRows * D * 4;
  static constexpr int kQueries = kSharedQ ? kRows * D * 2 : 0;
  // Two CTAs on an SM where the registers allow it: one joins its warps' states and
  // stores while the other goes on.
  static constexpr int kCtas = kQuant && NT == 1 ? 2 : 1;
  // As many stages as fit beside the buffer for merging, at most 16, and a multiple of the
  // teams: a stage belongs to one of them, which so sees every phase of its barrier.
  static constexpr int kRoom = (kCtas == 1 ? 224 : 110) * 1024 - kMerge - kQueries;
  static constexpr int kFit = kRoom / (2 * kTile + kScales);
  static constexpr int kStages = (kFit < 16 ? kFit : 16) / kTeams * kTeams;
  static constexpr int kOffMerge = kStages * 2 * kTile;
  static constexpr int kOffQueries = kOffMerge + kMerge;
  static constexpr int kOffScales = kOffQueries + kQueries;
  static constexpr int kSmem = kOffScales + kStages * kScales + 1024;  // + alignment
  static_assert(kStages >= kTeams, "shared memory");
};

template <int kStages, int kRows, int kWarps>
struct StreamShared {
  uint64_t full[kStages], empty[kStages];
  uint64_t team_full, merge_full, merge_empty;
  Unit unit[kStages];
  float2 ml[kWarps][kRows];
  PlanShared plan;
  int abort_flag;
};

// bf16 or f16 operands.
template <bool kHalf>
__device__ __forceinline__ void mma_16n8k16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
#define ATTN_MMA_16N8K16(TYPE)                                                                  \
  asm("mma.sync.aligned.m16n8k16.row.col.f32." TYPE "." TYPE                                    \
      ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"                    \
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                          \
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
  if constexpr (kHalf)
    ATTN_MMA_16N8K16("f16");
  else
    ATTN_MMA_16N8K16("bf16");
#undef ATTN_MMA_16N8K16
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <int kBytes>
__device__ __forceinline__ void load_piece(uint32_t (&x)[4], const uint8_t* from) {
  if constexpr (kBytes == 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(from);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(from);
    x[0] = v.x, x[1] = v.y, x[2] = x[3] = 0;
  }
}

// Key that row i of a 16-key block stands for.  For i = 2a + b < 8: the keys of
// b = 0 and 1 differ in bit 2 (the 16-byte pieces 4c .. 4c + 3 of both, exchanged by
// their key's low bits, are in different banks: loads of K), and those of one b over
// all a differ in bits 1 and 2 (so are pieces 2c and 2c + 1 of these four: V).
__device__ __forceinline__ int block_key(int i) {
  const int a = (i >> 1) & 3;
  return ((2 * a + (a >> 1)) ^ ((i & 1) << 2)) + (i & 8);
}

// Where byte `at` of row `row` of a copied tile is: 128-byte rows swizzled by 128
// bytes, 64-byte rows by 64; of wider rows, copied 16 at a time, the first halves and
// then the second ones.
template <int kRowBytes>
__device__ __forceinline__ uint32_t swizzled(int row, int at) {
  if constexpr (kRowBytes == 64)
    return static_cast<uint32_t>(row * 64 + (at ^ ((row >> 1 & 3) << 4)));
  else
    return static_cast<uint32_t>((kRowBytes == 256 ? (row & ~15) * 128 : 0) + (at >> 7) * 2048 +
                                 row * 128 + ((at & 127) ^ ((row & 7) << 4)));
}

// Where piece i (of 4 elements) of a row of O stands in the buffer for merging: eight lanes
// that store pieces of a row, 2 or 4 apart, do so in different banks.
__device__ __forceinline__ int merge_slot(int i) { return i ^ (i >> 3 & 3); }

template <int D, bool kQuant, int NT>
__global__ void __launch_bounds__(StreamCfg<D, kQuant, NT>::kThreads, (StreamCfg<D, kQuant, NT>::kCtas))
    paged_stream_kernel(const __grid_constant__ PagedParams p) {
  using C = StreamCfg<D, kQuant, NT>;
  constexpr int kStages = C::kStages, kRows = C::kRows, kRowBytes = C::kRowBytes;
  constexpr int kLoaders = C::kLoaders, kThreads = C::kThreads;
  constexpr int kTeams = C::kTeams, kWarps = C::kWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  __shared__ StreamShared<kStages, kRows, kWarps> ms;
  static_assert((C::kSmem + sizeof(ms) + 1024) * C::kCtas <= 228 * 1024, "shared memory");
  const uint32_t abort_flag = smem_u32(&ms.abort_flag);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ms.full[s], 1);
      mbar_init(&ms.empty[s], 4);
    }
    mbar_init(&ms.team_full, kWarps - 4);
    mbar_init(&ms.merge_full, 4);
    mbar_init(&ms.merge_empty, kWarps);
    ms.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tmap_k);
    tma_prefetch_desc(&p.tmap_v);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for what the stream did before
  const StreamPlan plan(p.c, p.G, kRows);
  // (its barriers also publish the mbarriers)
  const PlanPlace at = plan.place<kThreads>(ms.plan, blockIdx.x, p.ctas);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  clear_counts(p);

  if (warp >= kWarps) {
    // ---- a loading warp: of every kLoaders-th unit
    const uint32_t loader = static_cast<uint32_t>(warp - kWarps);
    const int box_bits = kRowBytes == 256 ? 4 : min(p.c.page_bits, 6), box = 1 << box_bits;
    static_assert(kUnitKeys == 64, "box_bits");
    const uint64_t policy = l2_policy_evict_first();
    uint32_t s = loader;
    bool ok = true;
    int b = at.b;
    uint32_t in_request = at.in_request;  // unit within the request
    const Deal deal(at.total, p.ctas);
    constexpr uint32_t kBlockCost = block_cost(kQuant, kRows);
    for (uint32_t u = at.first; u < at.end && b < p.c.B && ok;) {
      const Rows rows = b == at.b ? at.rows : request_rows(p.c, b);
      const int len = b == at.b ? at.len : clamp_len(p.c, b);
      const uint32_t tiles = plan.tiles(len), units = plan.units(rows.n, len);
      const int blocks = plan.blocks(rows.n);
      int pbase = -64, ids = 0;
      while (in_request < units && u < at.end && ok) {
        // an item's part that lies in this CTA, what it costs and its key tiles
        const uint32_t item = in_request / (tiles + kBlockCost);
        const uint32_t from = in_request % (tiles + kBlockCost);
        const uint32_t cost = min(tiles + kBlockCost - from, at.end - u);
        const uint32_t tile0 = max(from, kBlockCost) - kBlockCost;
        const uint32_t n = max(from + cost, kBlockCost) - kBlockCost - tile0;
        u += cost;
        in_request += cost;
        const int h = static_cast<int>(item) / blocks, block = static_cast<int>(item) % blocks;
        const int slot = n == tiles ? -1 : 2 * static_cast<int>(blockIdx.x) + (tile0 == 0);
        int cta0 = 0, parts = 0;
        if (n > 0 && n < tiles) {
          const uint32_t key_units = u - cost - from + kBlockCost;  // where its key tiles begin
          cta0 = static_cast<int>(deal.run_of(key_units));
          parts = static_cast<int>(deal.run_of(key_units + tiles - 1)) - cta0 + 1;
        }
        // the teams take turns, so that all have as many units: some may be without keys
        const uint32_t all = (n + kTeams - 1) / kTeams * kTeams;
        for (uint32_t i = loader; i < all; i += kLoaders, s += kLoaders) {
          const int key0 = static_cast<int>(tile0 + i) * kUnitKeys;
          const uint32_t st = s % kStages;
          // pages of this unit: lane l holds entry pbase + l of the table's row
          const int page0 = key0 >> p.c.page_bits;
          const int keys = i < n ? min(kUnitKeys, len - key0) : 0;
          const int n_box = (max(0, keys) + box - 1) >> box_bits;
          const int page1 = (key0 + (max(n_box - 1, 0) << box_bits)) >> p.c.page_bits;
          if (page0 < pbase || page1 >= pbase + 32) {
            pbase = page0;
            ids = pbase + lane < p.c.M ? p.c.table[static_cast<size_t>(b) * p.c.M + pbase + lane]
                                       : -1;
          }
          const int key = key0 + lane * box;
          const int id = __shfl_sync(0xFFFFFFFFu, ids, ((key >> p.c.page_bits) - pbase) & 31);
          if (!warp_all(mbar_wait(&ms.empty[st], ((s / kStages) & 1u) ^ 1u, abort_flag, p.err,
                                  kErrWaitLoad, p.wait_limit_ns))) {
            ok = false;
            break;
          }
          const bool good = static_cast<unsigned>(id) < static_cast<unsigned>(p.c.P);
          const uint32_t bad = __ballot_sync(0xFFFFFFFFu, lane < n_box && !good);
          uint8_t* scales = smem + C::kOffScales + st * C::kScales + lane * box;
          if (bad) {
            // a page of zeros: the copies fill with them; its scales, the least, are written here
            if (lane == 0) atomicOr(p.err, kErrPage);
            if (kQuant && (bad >> lane & 1u))
              for (int i = 0; i < 2 * box; ++i)
                scales[(i < box ? 0 : kUnitKeys) + i % box] = kScaleLeast;
            __syncwarp();
          }
          if (lane == 0) {
            ms.unit[st] = Unit{(i < kTeams ? kUnitFirst : 0) | (i + kTeams >= all ? kUnitLast : 0),
                               b, h, block, i < n ? key0 : len, len, slot, cta0, parts, rows.first,
                               rows.n};
            mbar_arrive_expect_tx(
                &ms.full[st],
                static_cast<uint32_t>(2 * box * (n_box * kRowBytes +
                                                 (kQuant ? n_box - __popc(bad) : 0))));
          }
          __syncwarp();
          if (lane < n_box) {
            const int z = good ? id * p.c.Hkv + h : p.c.P * p.c.Hkv;
            const int y = key & (p.c.page - 1);
            uint8_t* dst = smem + st * (2 * C::kTile) + lane * box * kRowBytes;
            tma_load_4d(dst, &p.tmap_k, &ms.full[st], 0, y, 0, z, policy);
            tma_load_4d(dst + C::kTile, &p.tmap_v, &ms.full[st], 0, y, 0, z, policy);
            if (kQuant && good) {
              const size_t from = static_cast<size_t>(z) * p.c.page + y;
              bulk_copy(scales, p.c.kscale + from, box, &ms.full[st], policy);
              bulk_copy(scales + kUnitKeys, p.c.vscale + from, box, &ms.full[st], policy);
            }
          }
        }
      }
      ++b;
      in_request = 0;
    }
    for (int i = 0; i < kTeams / kLoaders && ok; ++i, s += kLoaders) {
      const uint32_t st = s % kStages;
      if (warp_all(mbar_wait(&ms.empty[st], ((s / kStages) & 1u) ^ 1u, abort_flag, p.err,
                             kErrWaitLoad, p.wait_limit_ns)) &&
          lane == 0) {
        ms.unit[st].flags = kUnitEnd;
        mbar_arrive(&ms.full[st]);
      }
      __syncwarp();
    }
    if (abort_set(abort_flag))  // copies in flight land before the CTA leaves
      for (uint32_t i = s >= kStages ? s - kStages : loader; i < s; i += kLoaders)
        drain_wait(&ms.full[i % kStages], (i / kStages) & 1u);
    return;
  }

  // ---- computing warps
  const int g = lane >> 2, t = lane & 3;
  const int my_key = (warp & 3) * 16;  // first of the warp's keys in a unit
  const int row_lo = my_key + block_key(g), row_hi = row_lo + 8;  // K: keys of S^T's rows g, g + 8
  const int vkey = my_key + block_key(2 * t);  // V: keys vkey, ^4, + 8 of each
  const int vkey1 = my_key + block_key(2 * t + 1);
  constexpr int kSteps = D / 16;  // products per S^T, and 16-row tiles of O^T
  uint32_t qf[C::kSharedQ ? 1 : NT][2 * kSteps];
  uint4* const shared_q = reinterpret_cast<uint4*>(smem + C::kOffQueries) + lane;
  float o[NT][kSteps][4], m[NT][2], l[NT][2], by_row[NT][2];
  int vis[NT][2], first_vis = 0;
  uint32_t merges = 0;
  for (uint32_t s = static_cast<uint32_t>(warp) / 4;; s += kTeams) {  // the team's units
    const uint32_t st = s % kStages;
    if (!warp_all(mbar_wait(&ms.full[st], (s / kStages) & 1u, abort_flag, p.err, kErrWaitMma,
                            p.wait_limit_ns)))
      return;
    const Unit un = ms.unit[st];
    if (un.flags & kUnitEnd) return;
    const int n_rows = un.rows * p.G - un.block * kRows;  // of this block and those behind it
    if (un.flags & kUnitFirst) {
      const int before = un.len - un.rows;  // keys in front of the first new token
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = nt * 8 + g;
        const int row = un.block * kRows + r;
        const uint8_t* q =
            static_cast<const uint8_t*>(p.q) +
            2 * (static_cast<size_t>(un.row0 + row / p.G) * p.q_stride +
                 static_cast<size_t>(un.h * p.G + row % p.G) * D);
        // the elements that go with those of K that the thread loads: piece 4c + t of a
        // row, its pairs in order
        constexpr int kWords = kQuant ? 8 : 4;  // of the query for one piece
        uint32_t(&qn)[2 * kSteps] = qf[C::kSharedQ ? 0 : nt];
#pragma unroll
        for (int c = 0; c < kRowBytes / 64; ++c)
#pragma unroll
          for (int i = 0; i < kWords / 4; ++i) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (r < n_rows) x = *reinterpret_cast<const uint4*>(q + ((4 * c + t) * kWords + 4 * i) * 4);
            qn[c * kWords + 4 * i] = x.x;
            qn[c * kWords + 4 * i + 1] = x.y;
            qn[c * kWords + 4 * i + 2] = x.z;
            qn[c * kWords + 4 * i + 3] = x.w;
          }
        float scale = 1.f;
        if constexpr (kQuant) {
          // to f16, over a power of two that makes the row's largest element 1 to 2: exact
          // but below 2^-14, where a step is 2^-24
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 2 * kSteps; ++i)
            top = max(top, bf16x2_top(qn[i]));
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          const uint32_t e = min(max(top >> 23, 1u), 253u);
          scale = __uint_as_float(e << 23);
          const float inv = __uint_as_float((254u - e) << 23);
#pragma unroll
          for (int i = 0; i < 2 * kSteps; ++i)
            qn[i] = bf16x2_to_f16x2(qn[i], inv);
        }
        if constexpr (C::kSharedQ) {
          // (every warp stores the same; those of the item before are not read any more, since
          // all warps' states of it are joined)
#pragma unroll
          for (int i = 0; i < kSteps / 2; ++i)
            shared_q[(nt * (kSteps / 2) + i) * 32] =
                make_uint4(qn[4 * i], qn[4 * i + 1], qn[4 * i + 2], qn[4 * i + 3]);
          __syncwarp();
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int row_of = (un.block * kRows + nt * 8 + 2 * t + k) / p.G;
          vis[nt][k] = p.causal ? min(un.len, before + row_of + 1) : un.len;
          m[nt][k] = -CUDART_INF_F;
          l[nt][k] = 0.f;
          by_row[nt][k] =
              kQuant ? p.scale_log2 * __shfl_sync(0xFFFFFFFFu, scale, 8 * t + 4 * k) : p.scale_log2;
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[nt][i][k] = 0.f;
      }
      first_vis = p.causal ? min(un.len, before + un.block * kRows / p.G + 1) : un.len;
    }

    const int k0 = un.key0 + my_key;
    if (k0 < un.len) {
      const uint8_t *ktile = smem + st * (2 * C::kTile), *vtile = ktile + C::kTile;
      [[maybe_unused]] const uint8_t* scales = smem + C::kOffScales + st * C::kScales;
      float x[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) x[nt][k] = 0.f;
#pragma unroll
      for (int c = 0; c < kRowBytes / 64; ++c) {
        uint32_t a[4], e[4];
        load_piece<16>(a, ktile + swizzled<kRowBytes>(row_lo, (4 * c + t) * 16));
        load_piece<16>(e, ktile + swizzled<kRowBytes>(row_hi, (4 * c + t) * 16));
        if constexpr (kQuant) {
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const uint32_t a0 = e4m3_lo(a[i]), a2 = e4m3_hi(a[i]);
            const uint32_t a1 = e4m3_lo(e[i]), a3 = e4m3_hi(e[i]);
            const uint32_t b0 = e4m3_lo(a[i + 1]), b2 = e4m3_hi(a[i + 1]);
            const uint32_t b1 = e4m3_lo(e[i + 1]), b3 = e4m3_hi(e[i + 1]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint4 y;
              if constexpr (C::kSharedQ) {
                y = shared_q[(nt * (kSteps / 2) + 2 * c + i / 2) * 32];
              } else {
                const uint32_t* from = &qf[nt][8 * c + 2 * i];
                y = make_uint4(from[0], from[1], from[2], from[3]);
              }
              mma_16n8k16<true>(x[nt], a0, a1, a2, a3, y.x, y.y);
              mma_16n8k16<true>(x[nt], b0, b1, b2, b3, y.z, y.w);
            }
          }
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_16n8k16<false>(x[nt], a[0], e[0], a[1], e[1], qf[nt][4 * c], qf[nt][4 * c + 1]);
            mma_16n8k16<false>(x[nt], a[2], e[2], a[3], e[3], qf[nt][4 * c + 2], qf[nt][4 * c + 3]);
          }
        }
      }
      // scores in log2 units, unseen ones -inf
      const float by_lo = kQuant ? scale_value(scales[row_lo]) : 1.f;
      const float by_hi = kQuant ? scale_value(scales[row_hi]) : 1.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[nt][k] *= by_row[nt][k & 1];
          if constexpr (kQuant) x[nt][k] *= k < 2 ? by_lo : by_hi;
        }
      if (k0 + 16 > first_vis) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (un.key0 + (k < 2 ? row_lo : row_hi) >= vis[nt][k & 1]) x[nt][k] = -CUDART_INF_F;
      }
      // Quantised, a weight of V's codes is 2^(x + e), e the exponent of V's scale, and the
      // maximum is of x + e (see kWeightTop): what f16 loses is next to the largest
      // product, since every row of codes reaches beyond 224 but one of zeros, which says
      // 2^0 and counts as the least.  (ev: e + kWeightLift; m: the sum's reference.)
      constexpr float kTop = kQuant ? kWeightTop : 0.f, kLift = kQuant ? kWeightLift : 0.f;
      float ev[2] = {kLift, kLift};
      [[maybe_unused]] uint32_t vscale[2] = {127, 127};
      if constexpr (kQuant) {
        vscale[0] = scales[kUnitKeys + row_lo];
        vscale[1] = scales[kUnitKeys + row_hi];
        if (__any_sync(0xFFFFFFFFu, vscale[0] == kScaleOfZeros || vscale[1] == kScaleOfZeros)) {
          const int rows[2] = {row_lo, row_hi};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t bits = vscale[k] == kScaleOfZeros ? 0u : ~0u;
#pragma unroll 1
            for (int at = 0; at < D; at += 16)
              bits |= or_of(*reinterpret_cast<const uint4*>(vtile + swizzled<kRowBytes>(rows[k], at)));
            if (!(bits & 0x7F7F7F7Fu)) vscale[k] = kScaleLeast;
          }
        }
        if (vscale[0] != kScaleNan) ev[0] = scale_exponent(vscale[0]) + kLift;
        if (vscale[1] != kScaleNan) ev[1] = scale_exponent(vscale[1]) + kLift;
      }
      // The maximum moves only when a score is above it by more than 2^8 (quantised
      // 2^kWeightRoom): a stale one is as good (the sum has the same), and the vote is cheaper
      // than the maximum.
      constexpr float kStale = kQuant ? kWeightTop + kWeightRoom : 8.f;
      bool above = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) above = above || x[nt][k] + ev[k >> 1] > m[nt][k & 1] + kStale;
      if (__any_sync(0xFFFFFFFFu, above)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float top = fmaxf(x[nt][k] + ev[0], x[nt][k + 2] + ev[1]);
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
            if (top > m[nt][k] + kStale) {
              top -= kTop;
              const float2 f = ex2_factors<kQuant>(m[nt][k] - top);  // 0 the first time
              const float alpha = f.x * f.y;
              m[nt][k] = top;
              l[nt][k] = l[nt][k] * f.x * f.y;
#pragma unroll
              for (int i = 0; i < kSteps; ++i) {
                o[nt][i][k] *= alpha;
                o[nt][i][k + 2] *= alpha;
              }
            }
          }
      }
      uint32_t pf[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool none = x[nt][k] == -CUDART_INF_F;
          const float d = x[nt][k] - m[nt][k & 1];
          w[k] = none ? 0.f : ex2_approx(d);
          l[nt][k & 1] += w[k];
          if constexpr (kQuant) w[k] = none ? 0.f : ex2_approx(d + ev[k >> 1]);
        }
        // rounded for the product: to bf16, as V is, or f16
        pf[nt][0] = transpose_8x8(kQuant ? pack_f16x2(w[0], w[1]) : pack_bf16x2(w[0], w[1]));
        pf[nt][1] = transpose_8x8(kQuant ? pack_f16x2(w[2], w[3]) : pack_bf16x2(w[2], w[3]));
      }
      // V: rows behind the last token may hold anything, and 0 * NaN is none; rows that
      // stand for NaN
      const bool tail = k0 + 16 > un.len;
      const int keys[4] = {vkey, vkey1, vkey + 8, vkey1 + 8};
      constexpr int kVBytes = kQuant ? D / 8 : 16;  // a thread's piece of a row
      [[maybe_unused]] const bool odd =
          kQuant && (tail || __any_sync(0xFFFFFFFFu, max(vscale[0], vscale[1]) == kScaleNan));
#pragma unroll
      for (int part = 0; part < (kQuant ? 1 : D / 64); ++part) {
        uint32_t v[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          load_piece<kVBytes>(v[i], vtile + swizzled<kRowBytes>(keys[i], part * 128 + g * kVBytes));
          if (kQuant ? odd : tail) {
            const bool none = un.key0 + keys[i] >= un.len;
            const bool nan = kQuant && scales[kUnitKeys + keys[i]] == kScaleNan;
            if (none || nan)
#pragma unroll
              for (int k = 0; k < kVBytes / 4; ++k) v[i][k] = none ? 0u : 0x7F7F7F7Fu;
          }
        }
#pragma unroll
        for (int i = 0; i < kVBytes / 4; ++i) {
          if constexpr (kQuant) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {  // bytes 2k, 2k + 1 of the word
              // byte 2k of both keys, then byte 2k + 1
              const uint32_t both = k ? 0x7362 : 0x5140;
              const uint32_t lo = __byte_perm(v[0][i], v[1][i], both);
              const uint32_t hi = __byte_perm(v[2][i], v[3][i], both);
              const uint32_t a0 = e4m3_lo(lo), a1 = e4m3_hi(lo);
              const uint32_t a2 = e4m3_lo(hi), a3 = e4m3_hi(hi);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_16n8k16<true>(o[nt][2 * i + k], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
            }
          } else {
            const uint32_t a0 = __byte_perm(v[0][i], v[1][i], 0x5410);
            const uint32_t a1 = __byte_perm(v[0][i], v[1][i], 0x7632);
            const uint32_t a2 = __byte_perm(v[2][i], v[3][i], 0x5410);
            const uint32_t a3 = __byte_perm(v[2][i], v[3][i], 0x7632);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_16n8k16<false>(o[nt][part * 4 + i], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
          }
        }
      }
    }
    // (nothing orders a read whose value is still on its way before the next copy's writes)
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&ms.empty[st]);
    if (!(un.flags & kUnitLast)) continue;

    // ---- the warps' states of the block, joined through shared memory: the other teams'
    // with the first team's, register by register, then those four by rows
    float* const merge = reinterpret_cast<float*>(smem + C::kOffMerge) +
                         (warp < 4 ? warp : warp - 4) * kRows * D;
    if (!warp_all(mbar_wait(&ms.merge_empty, (merges & 1u) ^ 1u, abort_flag, p.err, kErrWaitCorr,
                            p.wait_limit_ns)))
      return;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int d = 4; d < 32; d *= 2) l[nt][k] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][k], d);
    auto say = [&](int as) {  // maximum and sum of every row
      if (g == 0)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) ms.ml[as][nt * 8 + 2 * t + k] = make_float2(m[nt][k], l[nt][k]);
    };
    float4* const mine = reinterpret_cast<float4*>(merge) + lane;
    if (warp >= 4) {
      say(warp);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
          mine[(nt * kSteps + i) * 32] = make_float4(o[nt][i][0], o[nt][i][1], o[nt][i][2], o[nt][i][3]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.team_full);
    } else {
      if (!warp_all(mbar_wait(&ms.team_full, merges & 1u, abort_flag, p.err, kErrWaitCorr,
                              p.wait_limit_ns)))
        return;
#pragma unroll
      for (int team = 1; team < kTeams; ++team)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float a[2], e[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 ml = ms.ml[warp + 4 * team][nt * 8 + 2 * t + k];
            const float top = fmaxf(m[nt][k], ml.x);
            const float2 f = ex2_factors<kQuant>(m[nt][k] == -CUDART_INF_F ? 0.f : m[nt][k] - top);
            const float2 h = ex2_factors<kQuant>(ml.x == -CUDART_INF_F ? 0.f : ml.x - top);
            a[k] = f.x * f.y;
            e[k] = h.x * h.y;
            m[nt][k] = top;
            l[nt][k] = l[nt][k] * f.x * f.y + ml.y * h.x * h.y;
          }
          const float4* theirs = mine + (team - 1) * (kRows * D);  // (4 warps' parts further)
#pragma unroll
          for (int i = 0; i < kSteps; ++i) {
            const float4 x = theirs[(nt * kSteps + i) * 32];
            o[nt][i][0] = o[nt][i][0] * a[0] + x.x * e[0];
            o[nt][i][1] = o[nt][i][1] * a[1] + x.y * e[1];
            o[nt][i][2] = o[nt][i][2] * a[0] + x.z * e[0];
            o[nt][i][3] = o[nt][i][3] * a[1] + x.w * e[1];
          }
        }
      __syncwarp();  // (the warp's part of the buffer is read)
      say(warp);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float* row = merge + (nt * 8 + 2 * t + k) * D;
#pragma unroll
          for (int i = 0; i < kSteps; i += 2) {
            // four elements of the row: the thread's tiles i and i + 1
            const int d = kQuant ? g * (D / 8) + 2 * i : (i / 4) * 64 + g * 8 + 2 * (i % 4);
            reinterpret_cast<float4*>(row)[merge_slot(d / 4)] =
                make_float4(o[nt][i][k], o[nt][i][k + 2], o[nt][i + 1][k], o[nt][i + 1][k + 2]);
          }
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.merge_full);
    }
    if (!warp_all(mbar_wait(&ms.merge_full, merges & 1u, abort_flag, p.err, kErrWaitCorr,
                            p.wait_limit_ns)))
      return;
    for (int r = warp; r < min(kRows, n_rows); r += kWarps) {
      State<D, kQuant> sum;
      float top = -CUDART_INF_F;
      const int from = D == 128 ? merge_slot(lane) : 2 * merge_slot(lane / 2) + lane % 2;
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, ms.ml[i][r].x);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sum.add(ms.ml[i][r], top,
                reinterpret_cast<const typename State<D, kQuant>::Vec*>(
                    reinterpret_cast<float*>(smem + C::kOffMerge) + (i * kRows + r) * D)[from]);
      const int row = un.block * kRows + r;
      if (un.slot < 0) {
        sum.finish(p, un.row0 + row / p.G, un.h * p.G + row % p.G, top, lane);
      } else {
        const size_t to = static_cast<size_t>(un.slot) * kRows + r;
        sum.store(p.part_o + to * D, lane);
        if (lane == 0) p.part_ml[to] = make_float2(top, sum.l);
      }
    }
    if (un.slot >= 0) {
      // the rows whose last part this was (lane i: the warp's i-th)
      const int r0 = warp + lane * kWarps;
      uint32_t last = last_to_arrive(&p.arrived[un.cta0 * 16 + min(r0, kRows - 1)], un.parts,
                                     r0 < min(kRows, n_rows));
      for (; last; last &= last - 1) {
        const int r = warp + (__ffs(last) - 1) * kWarps, row = un.block * kRows + r;
        State<D, kQuant> all;
        const float most = all.join(p, un.parts, lane, [&](int k) {
          return (static_cast<size_t>(un.cta0 + k) * 2 + (k == 0)) * kRows + r;
        });
        all.finish(p, un.row0 + row / p.G, un.h * p.G + row % p.G, most, lane);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&ms.merge_empty);
    ++merges;
  }
}

template <int D, bool kQuant, int NT>
cudaError_t launch_stream(const PagedParams& p, int dev, cudaStream_t stream) {
  using C = StreamCfg<D, kQuant, NT>;
  static std::atomic<bool> ready[64];
  if (!ready[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(paged_stream_kernel<D, kQuant, NT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    ready[dev].store(true, std::memory_order_release);
  }
  return launch_overlapped(paged_stream_kernel<D, kQuant, NT>, dim3(p.ctas), C::kThreads, C::kSmem,
                           stream, p);
}

}  // namespace

// Rows of 256 bytes, twice what a swizzled box holds, take a box with both halves of 16 rows,
// so that a warp's keys are in one of them: half the copies of boxes of single halves with
// pages of 16 (8 requests of 500 to 65536 tokens 101 -> 81 us, 16 of 65536 with 16 rows
// 774 -> 605), and with longer pages no more time than larger boxes.
int paged_stream_box(const PagedArrays& c) {
  return !c.quant && c.D == 128 ? 16 : std::min(c.page, kUnitKeys);
}

unsigned paged_stream_ctas(const PagedParams& p, int rows) {
  return p.c.quant && rows == 8 ? 2 : 1;
}

size_t paged_stream_state(const PagedParams& p, int rows) {
  return static_cast<size_t>(p.ctas) * 2 * rows;
}

cudaError_t launch_paged_stream(const PagedParams& p, int rows, int dev, cudaStream_t stream) {
  using Launch = cudaError_t (*)(const PagedParams&, int, cudaStream_t);
  static const Launch table[2][2][2] = {
      {{launch_stream<64, false, 1>, launch_stream<64, false, 2>},
       {launch_stream<64, true, 1>, launch_stream<64, true, 2>}},
      {{launch_stream<128, false, 1>, launch_stream<128, false, 2>},
       {launch_stream<128, true, 1>, launch_stream<128, true, 2>}}};
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  return table[p.c.D == 128][p.c.quant][rows == 16](p, dev, stream);
}

}  // namespace attn
