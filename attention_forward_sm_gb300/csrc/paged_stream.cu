// Attention of a few new tokens of each request over its paged cache: single tokens
// (decode) and a handful of drafted ones.
//
// The rows of a (request, KV head) are its new tokens times the G query heads that
// share the head, at most 8 NT per block of rows; all of them use every key that is
// read, so a call is bound by reading the cache once.  The keys of all blocks,
// 64 to a unit, make one long sequence of units, which is dealt out evenly among the
// CTAs (one per SM): a request of any length among any others costs its bytes.  A
// block that ends up in several CTAs has a partial state (maximum, sum, O) in each;
// paged_merge_kernel joins them.
//
// A CTA is one loading warp and eight computing warps around a ring of stages, one
// unit each: K and V of 64 keys by tensor copies, a box per page.  A unit belongs to
// four of the computing warps, 16 keys each, every other unit to the other four.
// Rows are few, so the keys are the rows of the products (mma.sync m16n8k16):
//   S^T [16 keys, 8 rows] = K [16, D] Q^T,   O^T [D, 8 rows] += V^T [D, 16] P^T.
// A tcgen05.mma has at least 64 rows of one operand in shared memory or TMEM and
// would take the keys through either; here they go from shared memory straight into
// registers, where e4m3 codes become bf16 on the way.  Which key and which
// dimension a thread's piece of an operand stands for is free as long as both
// operands agree, and chosen so that every load is 16 bytes of a swizzled row
// without bank conflicts: row i of a 16-key block is key kKey(i), and a thread
// has whole 16-byte pieces of the keys' rows.  P^T is S^T transposed within a warp
// (movmatrix).
#include <math_constants.h>

#include <atomic>

#include "../../include/attn.h"
#include "fwd_tile.cuh"
#include "paged_plan.cuh"

namespace attn {
namespace {

constexpr int kWarps = 8;  // computing
constexpr int kThreads = (kWarps + 1) * 32;

// One unit in the ring, as the loading warp describes it.
struct Unit {
  int flags, b, h, block;  // of kUnit..; request, KV head, block of rows
  int key0, len, slot;     // first key; tokens in the cache; partial state, -1: none
  int row0, rows;          // first row of the dense tensors; new tokens
};
constexpr int kUnitFirst = 1, kUnitLast = 2, kUnitEnd = 4;  // of the block's part here; no unit

template <int D, bool kQuant, int NT>
struct StreamCfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kRowBytes = kQuant ? D : 2 * D;
  static constexpr int kTile = kUnitKeys * kRowBytes;  // K or V of a unit
  static constexpr int kScales = kQuant ? 2 * kUnitKeys : 0;
  static constexpr int kMerge = kWarps * kRows * D * 4;
  // as many stages as fit beside the buffer for merging, 128 KB of copies in flight at most
  static constexpr int kRoom = 226 * 1024 - 1024 - kMerge;
  static constexpr int kFit = kRoom / (2 * kTile + kScales);
  static constexpr int kWant = 196 * 1024 / (2 * kTile);
  static constexpr int kStages = kFit < kWant ? kFit : kWant;
  static constexpr int kOffMerge = kStages * 2 * kTile;
  static constexpr int kOffScales = kOffMerge + kMerge;
  static constexpr int kSmem = kOffScales + kStages * kScales + 1024;  // + alignment
  static_assert(kStages >= 3, "shared memory");
};

template <int kStages, int kRows>
struct StreamShared {
  uint64_t full[kStages], empty[kStages];
  uint64_t merge_full, merge_empty;
  Unit unit[kStages];
  float2 ml[kWarps][kRows];
  PlanShared plan;
  int abort_flag;
};

__device__ __forceinline__ void mma_16n8k16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void lds128(uint32_t (&x)[4], uint32_t addr) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void lds64(uint32_t (&x)[4], uint32_t addr) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t x;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
  return x;
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
// bytes (tiles of wider rows are two such tiles), 64-byte rows by 64.
template <int kRowBytes>
__device__ __forceinline__ uint32_t swizzled(int row, int at) {
  if constexpr (kRowBytes == 64)
    return static_cast<uint32_t>(row * 64 + (at ^ ((row >> 1 & 3) << 4)));
  else
    return static_cast<uint32_t>((at >> 7) * (kUnitKeys * 128) + row * 128 +
                                 ((at & 127) ^ ((row & 7) << 4)));
}

template <int D, bool kQuant, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    paged_stream_kernel(const __grid_constant__ PagedParams p) {
  using C = StreamCfg<D, kQuant, NT>;
  constexpr int kStages = C::kStages, kRows = C::kRows, kRowBytes = C::kRowBytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ StreamShared<kStages, kRows> ms;
  static_assert(C::kSmem + sizeof(ms) <= 227 * 1024, "shared memory");
  const uint32_t abort_flag = smem_u32(&ms.abort_flag);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ms.full[s], 1);
      mbar_init(&ms.empty[s], kWarps);
    }
    mbar_init(&ms.merge_full, kWarps);
    mbar_init(&ms.merge_empty, kWarps);
    ms.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tmap_k);
    tma_prefetch_desc(&p.tmap_v);
  }
  const StreamPlan plan(p.c, p.G, kRows);
  // (its barriers also publish the mbarriers)
  const PlanPlace at = plan.place<kThreads>(ms.plan, blockIdx.x, p.ctas);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == kWarps) {
    // ---- loading warp
    const int box = min(p.c.page, kUnitKeys);
    const uint64_t policy = l2_policy_evict_first();
    uint32_t s = 0;
    bool ok = true;
    int b = at.b;
    uint32_t in_request = at.in_request;  // unit within the request
    for (uint32_t u = at.first; u < at.end && b < p.c.B && ok;) {
      const Rows rows = request_rows(p.c, b);
      const int len = clamp_len(p.c, b);
      const uint32_t tiles = plan.tiles(len), units = plan.units(rows.n, len);
      const int blocks = plan.blocks(rows.n);
      int pbase = -64, ids = 0;
      while (in_request < units && u < at.end && ok) {
        // a block's part that lies in this CTA
        const uint32_t item = in_request / tiles, tile0 = in_request % tiles;
        const uint32_t n = min(tiles - tile0, at.end - u);
        const int h = static_cast<int>(item) / blocks, block = static_cast<int>(item) % blocks;
        const int slot = n == tiles ? -1 : 2 * static_cast<int>(blockIdx.x) + (tile0 == 0);
        for (uint32_t i = 0; i < n; ++i, ++s) {
          const int key0 = static_cast<int>(tile0 + i) * kUnitKeys;
          const uint32_t st = s % kStages;
          // pages of this unit: lane l holds entry pbase + l of the table's row
          const int page0 = key0 / p.c.page;
          const int n_box = max(0, min(kUnitKeys, len - key0) + box - 1) / box;
          const int page1 = (key0 + max(n_box - 1, 0) * box) / p.c.page;
          if (page0 < pbase || page1 >= pbase + 32) {
            pbase = page0;
            ids = pbase + lane < p.c.M ? p.c.table[static_cast<size_t>(b) * p.c.M + pbase + lane]
                                       : -1;
          }
          const int key = key0 + lane * box;
          const int id = __shfl_sync(0xFFFFFFFFu, ids, (key / p.c.page - pbase) & 31);
          if (!warp_all(mbar_wait(&ms.empty[st], ((s / kStages) & 1u) ^ 1u, abort_flag, p.err,
                                  kErrWaitLoad, p.wait_limit_ns))) {
            ok = false;
            break;
          }
          const bool good = static_cast<unsigned>(id) < static_cast<unsigned>(p.c.P);
          const uint32_t bad = __ballot_sync(0xFFFFFFFFu, lane < n_box && !good);
          uint8_t* scales = smem + C::kOffScales + st * C::kScales + lane * box;
          if (bad) {
            // a page of zeros: the copies fill with them; its scales are written here
            if (lane == 0) atomicOr(p.err, kErrPage);
            if (kQuant && (bad >> lane & 1u))
              for (int i = 0; i < 2 * box; ++i)
                scales[(i < box ? 0 : kUnitKeys) + i % box] = 127;
            __syncwarp();
          }
          if (lane == 0) {
            ms.unit[st] = Unit{(i == 0 ? kUnitFirst : 0) | (i == n - 1 ? kUnitLast : 0),
                               b, h, block, key0, len, slot, rows.first, rows.n};
            mbar_arrive_expect_tx(
                &ms.full[st],
                static_cast<uint32_t>(2 * box * (n_box * kRowBytes +
                                                 (kQuant ? n_box - __popc(bad) : 0))));
          }
          __syncwarp();
          if (lane < n_box) {
            const int z = good ? id * p.c.Hkv + h : p.c.P * p.c.Hkv;
            const int y = key % p.c.page;
            uint8_t* dst = smem + st * (2 * C::kTile) + lane * box * (kRowBytes < 128 ? 64 : 128);
            constexpr int kPieces = kRowBytes / 128 > 0 ? kRowBytes / 128 : 1;
            constexpr int kElems = kQuant ? 128 : 64;  // of a 128-byte piece
#pragma unroll
            for (int c = 0; c < kPieces; ++c) {
              tma_load_3d(dst + c * (kUnitKeys * 128), &p.tmap_k, &ms.full[st], c * kElems, y, z,
                          policy);
              tma_load_3d(dst + C::kTile + c * (kUnitKeys * 128), &p.tmap_v, &ms.full[st],
                          c * kElems, y, z, policy);
            }
            if (kQuant && good) {
              const size_t from = static_cast<size_t>(z) * p.c.page + y;
              bulk_copy(scales, p.c.kscale + from, box, &ms.full[st], policy);
              bulk_copy(scales + kUnitKeys, p.c.vscale + from, box, &ms.full[st], policy);
            }
          }
        }
        u += n;
        in_request += n;
      }
      ++b;
      in_request = 0;
    }
    if (ok) {
      const uint32_t st = s % kStages;
      if (warp_all(mbar_wait(&ms.empty[st], ((s / kStages) & 1u) ^ 1u, abort_flag, p.err,
                             kErrWaitLoad, p.wait_limit_ns)) &&
          lane == 0) {
        ms.unit[st].flags = kUnitEnd;
        mbar_arrive(&ms.full[st]);
      }
    }
    if (abort_set(abort_flag))  // copies in flight land before the CTA leaves
      for (uint32_t i = s > kStages ? s - kStages : 0u; i < s; ++i)
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
  uint32_t qf[NT][2 * kSteps];
  float o[NT][kSteps][4], m[NT][2], l[NT][2];
  int vis[NT][2], first_vis = 0;
  uint32_t merges = 0;
  for (uint32_t s = 0;; ++s) {
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
        const bool real = r < n_rows;
        const uint8_t* q =
            static_cast<const uint8_t*>(p.q) +
            2 * (static_cast<size_t>(un.row0 + row / p.G) * p.q_stride +
                 static_cast<size_t>(un.h * p.G + row % p.G) * D);
        // the elements that go with those of K that the thread loads: piece 4c + t
        // of a row, its 16-bit pairs in order (bf16) or its bytes 0 2 1 3 of each word
#pragma unroll
        for (int c = 0; c < kRowBytes / 64; ++c) {
          uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
          if (real) {
            const uint4* src = reinterpret_cast<const uint4*>(q + (4 * c + t) * (kQuant ? 32 : 16));
            x[0] = src[0];
            if constexpr (kQuant) x[1] = src[1];
          }
          if constexpr (kQuant) {
            const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              qf[nt][8 * c + 2 * i] = __byte_perm(w[2 * i], w[2 * i + 1], 0x5410);
              qf[nt][8 * c + 2 * i + 1] = __byte_perm(w[2 * i], w[2 * i + 1], 0x7632);
            }
          } else {
            qf[nt][4 * c] = x[0].x;
            qf[nt][4 * c + 1] = x[0].y;
            qf[nt][4 * c + 2] = x[0].z;
            qf[nt][4 * c + 3] = x[0].w;
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int row_of = (un.block * kRows + nt * 8 + 2 * t + k) / p.G;
          vis[nt][k] = p.causal ? min(un.len, before + row_of + 1) : un.len;
          m[nt][k] = -CUDART_INF_F;
          l[nt][k] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[nt][i][k] = 0.f;
      }
      first_vis = p.causal ? min(un.len, before + un.block * kRows / p.G + 1) : un.len;
    }

    const int k0 = un.key0 + my_key;
    if ((s & 1u) == static_cast<uint32_t>(warp >> 2) && k0 < un.len) {
      const uint32_t ktile = smem_u32(smem) + st * (2 * C::kTile), vtile = ktile + C::kTile;
      float x[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) x[nt][k] = 0.f;
      [[maybe_unused]] uint32_t f_lo = 0, f_hi = 0, scales = 0;
      float by_lo = p.scale_log2, by_hi = p.scale_log2;
      if constexpr (kQuant) {
        scales = smem_u32(smem) + C::kOffScales + st * C::kScales;
        const uint32_t lo = lds8(scales + row_lo), hi = lds8(scales + row_hi);
        f_lo = e4m3_factor(lo);
        f_hi = e4m3_factor(hi);
        by_lo *= e4m3_rest(lo);
        by_hi *= e4m3_rest(hi);
      }
#pragma unroll
      for (int c = 0; c < kRowBytes / 64; ++c) {
        uint32_t a[4], e[4];
        lds128(a, ktile + swizzled<kRowBytes>(row_lo, (4 * c + t) * 16));
        lds128(e, ktile + swizzled<kRowBytes>(row_hi, (4 * c + t) * 16));
        if constexpr (kQuant) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = e4m3_pair(a[i] << 8, f_lo), a2 = e4m3_pair(a[i], f_lo);
            const uint32_t a1 = e4m3_pair(e[i] << 8, f_hi), a3 = e4m3_pair(e[i], f_hi);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_16n8k16(x[nt], a0, a1, a2, a3, qf[nt][8 * c + 2 * i], qf[nt][8 * c + 2 * i + 1]);
          }
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_16n8k16(x[nt], a[0], e[0], a[1], e[1], qf[nt][4 * c], qf[nt][4 * c + 1]);
            mma_16n8k16(x[nt], a[2], e[2], a[3], e[3], qf[nt][4 * c + 2], qf[nt][4 * c + 3]);
          }
        }
      }
      // scores in log2 units, unseen ones -inf
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) x[nt][k] *= k < 2 ? by_lo : by_hi;
      if (k0 + 16 > first_vis) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (un.key0 + (k < 2 ? row_lo : row_hi) >= vis[nt][k & 1]) x[nt][k] = -CUDART_INF_F;
      }
      // The maximum moves only when a score is above it by more than 2^8: a stale one
      // is as good (the sum has the same), and the vote is cheaper than the maximum.
      bool above = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) above = above || x[nt][k] > m[nt][k & 1] + 8.f;
      if (__any_sync(0xFFFFFFFFu, above)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float top = fmaxf(x[nt][k], x[nt][k + 2]);
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
            if (top > m[nt][k] + 8.f) {
              const float alpha = ex2_approx(m[nt][k] - top);  // 0 the first time
              m[nt][k] = top;
              l[nt][k] *= alpha;
#pragma unroll
              for (int i = 0; i < kSteps; ++i) {
                o[nt][i][k] *= alpha;
                o[nt][i][k + 2] *= alpha;
              }
            }
          }
      }
      // V: rows behind the last token may hold anything, and 0 * NaN is none
      const bool tail = k0 + 16 > un.len;
      uint32_t pf[NT][2];
      [[maybe_unused]] float rest_lo = 1.f, rest_hi = 1.f;
      if constexpr (kQuant) {
        rest_lo = e4m3_rest(lds8(scales + kUnitKeys + row_lo));
        rest_hi = e4m3_rest(lds8(scales + kUnitKeys + row_hi));
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = x[nt][k] == -CUDART_INF_F ? 0.f : ex2_approx(x[nt][k] - m[nt][k & 1]);
        l[nt][0] += w[0] + w[2];
        l[nt][1] += w[1] + w[3];
        if constexpr (kQuant) {
          w[0] *= rest_lo;
          w[1] *= rest_lo;
          w[2] *= rest_hi;
          w[3] *= rest_hi;
        }
        // bf16 for the product, as V is
        pf[nt][0] = transpose_8x8(pack_bf16x2(w[0], w[1]));
        pf[nt][1] = transpose_8x8(pack_bf16x2(w[2], w[3]));
      }
      const int keys[4] = {vkey, vkey1, vkey + 8, vkey1 + 8};
      constexpr int kVBytes = kQuant ? D / 8 : 16;  // a thread's piece of a row
      [[maybe_unused]] uint32_t f[2];
      if constexpr (kQuant) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t by[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            by[k] = lds8(scales + kUnitKeys + keys[2 * i + k]);
            if (tail && un.key0 + keys[2 * i + k] >= un.len) by[k] = 127;
          }
          f[i] = e4m3_factors(by[0], by[1]);
        }
      }
#pragma unroll
      for (int half = 0; half < (kQuant ? 1 : D / 64); ++half) {
        uint32_t v[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t from = vtile + swizzled<kRowBytes>(keys[i], half * 128 + g * kVBytes);
          if constexpr (kVBytes == 16)
            lds128(v[i], from);
          else
            lds64(v[i], from);
          if (tail && un.key0 + keys[i] >= un.len)
#pragma unroll
            for (int k = 0; k < kVBytes / 4; ++k) v[i][k] = 0;
        }
#pragma unroll
        for (int i = 0; i < kVBytes / 4; ++i) {
          if constexpr (kQuant) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {  // bytes 2k, 2k + 1 of the word
              const uint32_t s0 = 0x4000 + 0x2020 * k, s1 = s0 + 0x1010;
              uint32_t a[4];
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                a[2 * j] = e4m3_pair(__byte_perm(v[2 * j][i], v[2 * j + 1][i], s0), f[j]);
                a[2 * j + 1] = e4m3_pair(__byte_perm(v[2 * j][i], v[2 * j + 1][i], s1), f[j]);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_16n8k16(o[nt][2 * i + k], a[0], a[1], a[2], a[3], pf[nt][0], pf[nt][1]);
            }
          } else {
            const uint32_t a0 = __byte_perm(v[0][i], v[1][i], 0x5410);
            const uint32_t a1 = __byte_perm(v[0][i], v[1][i], 0x7632);
            const uint32_t a2 = __byte_perm(v[2][i], v[3][i], 0x5410);
            const uint32_t a3 = __byte_perm(v[2][i], v[3][i], 0x7632);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_16n8k16(o[nt][half * 4 + i], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&ms.empty[st]);
    if (!(un.flags & kUnitLast)) continue;

    // ---- the warps' states of the block, joined through shared memory
    float* merge = reinterpret_cast<float*>(smem + C::kOffMerge);
    if (!warp_all(mbar_wait(&ms.merge_empty, (merges & 1u) ^ 1u, abort_flag, p.err, kErrWaitCorr,
                            p.wait_limit_ns)))
      return;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int d = 4; d < 32; d *= 2) l[nt][k] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][k], d);
        const int r = nt * 8 + 2 * t + k;
        if (g == 0) ms.ml[warp][r] = make_float2(m[nt][k], l[nt][k]);
        float* row = merge + (warp * kRows + r) * D;
#pragma unroll
        for (int i = 0; i < kSteps; i += 2) {
          // four elements of the row: the thread's tiles i and i + 1
          const int d = kQuant ? g * (D / 8) + 2 * i : (i / 4) * 64 + g * 8 + 2 * (i % 4);
          *reinterpret_cast<float4*>(row + d) =
              make_float4(o[nt][i][k], o[nt][i][k + 2], o[nt][i + 1][k], o[nt][i + 1][k + 2]);
        }
      }
    __syncwarp();
    if (lane == 0) mbar_arrive(&ms.merge_full);
    if (!warp_all(mbar_wait(&ms.merge_full, merges & 1u, abort_flag, p.err, kErrWaitCorr,
                            p.wait_limit_ns)))
      return;
    for (int r = warp; r < min(kRows, n_rows); r += kWarps) {
      State<D> sum;
      float top = -CUDART_INF_F;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) top = fmaxf(top, ms.ml[i][r].x);
#pragma unroll
      for (int i = 0; i < kWarps; ++i)
        sum.add(ms.ml[i][r], top, merge + (i * kRows + r) * D, lane);
      const int row = un.block * kRows + r;
      if (un.slot < 0) {
        sum.finish(p, un.row0 + row / p.G, un.h * p.G + row % p.G, top, lane);
      } else {
        const size_t to = static_cast<size_t>(un.slot) * kRows + r;
        sum.store(p.part_o + to * D, lane);
        if (lane == 0) p.part_ml[to] = make_float2(top, sum.l);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&ms.merge_empty);
    ++merges;
  }
}

// W warps join the partial states of a (row, query head) whose keys several CTAs
// had; the others' results are there already.  The plan, which needs no result
// of the kernel before, is found ahead of the wait for it.
template <int D, int W>
__global__ void __launch_bounds__(256) paged_merge_kernel(const __grid_constant__ PagedParams p,
                                                          int block_rows) {
  __shared__ PlanShared shared;
  __shared__ uint32_t starts_of[256];
  __shared__ alignas(16) float sums[8][D];
  __shared__ float2 tops[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % W;
  const StreamPlan plan(p.c, p.G, block_rows);
  const long long row = static_cast<long long>(blockIdx.x) * (8 / W) + warp / W;
  const int t = static_cast<int>(row / p.Hq), hq = static_cast<int>(row % p.Hq);
  const int b = row < static_cast<long long>(p.c.T) * p.Hq ? find_request(p.c, t, lane) : -1;
  const uint32_t before = plan.before<256>(shared, starts_of, b);
  int first = 0, n = 0, r = 0;
  bool starts = false;
  if (b >= 0) {
    const Rows rows = request_rows(p.c, b);
    const int len = clamp_len(p.c, b);
    const int in_head = (t - rows.first) * p.G + hq % p.G;
    const uint32_t tiles = plan.tiles(len);
    const uint32_t u0 = before + (static_cast<uint32_t>(hq / p.G) * plan.blocks(rows.n) +
                                  static_cast<uint32_t>(in_head / block_rows)) * tiles;
    r = in_head % block_rows;
    const Deal deal(shared.total, p.ctas);
    if (t - rows.first < rows.n && u0 + tiles <= shared.total) {
      first = static_cast<int>(deal.run_of(u0));
      n = static_cast<int>(deal.run_of(u0 + tiles - 1)) - first + 1;
      starts = deal.start(first) <= u0;
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  auto state = [&](int i) {
    return (static_cast<size_t>(first + i) * 2 + (i == 0 && starts ? 1 : 0)) * block_rows + r;
  };
  State<D> sum;
  float top = -CUDART_INF_F;
  if (n > 1) {
    for (int i = part + W * lane; i < n; i += 32 * W) top = fmaxf(top, p.part_ml[state(i)].x);
#pragma unroll
    for (int d = 1; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
#pragma unroll 4
    for (int i = part; i < n; i += W) sum.add(p.part_ml[state(i)], top, p.part_o + state(i) * D, lane);
  }
  if constexpr (W > 1) {
    sum.store(sums[warp], lane);
    if (lane == 0) tops[warp] = make_float2(top, sum.l);
    __syncthreads();
    if (part > 0) return;
    State<D> all;
#pragma unroll
    for (int i = 0; i < W; ++i) top = fmaxf(top, tops[warp + i].x);
#pragma unroll
    for (int i = 0; i < W; ++i) all.add(tops[warp + i], top, sums[warp + i], lane);
    sum = all;
  }
  if (n > 1) sum.finish(p, t, hq, top, lane);
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
  paged_stream_kernel<D, kQuant, NT><<<p.ctas, kThreads, C::kSmem, stream>>>(p);
  return cudaGetLastError();
}

template <int D, int W>
cudaError_t launch_merge(const PagedParams& p, int rows, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const long long all = static_cast<long long>(p.c.T) * p.Hq;
  cfg.gridDim = dim3(static_cast<unsigned>((all + 8 / W - 1) / (8 / W)));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel<D, W>, p, rows);
}

}  // namespace

size_t paged_stream_scratch(const PagedParams& p, int rows, size_t* ml_at) {
  *ml_at = static_cast<size_t>(p.ctas) * 2 * rows * p.c.D * sizeof(float);
  return *ml_at + static_cast<size_t>(p.ctas) * 2 * rows * sizeof(float2);
}

cudaError_t launch_paged_stream(const PagedParams& p, int rows, int dev, cudaStream_t stream) {
  using Launch = cudaError_t (*)(const PagedParams&, int, cudaStream_t);
  static const Launch table[2][2][2] = {
      {{launch_stream<64, false, 1>, launch_stream<64, false, 2>},
       {launch_stream<64, true, 1>, launch_stream<64, true, 2>}},
      {{launch_stream<128, false, 1>, launch_stream<128, false, 2>},
       {launch_stream<128, true, 1>, launch_stream<128, true, 2>}}};
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  cudaError_t e = table[p.c.D == 128][p.c.quant][rows == 16](p, dev, stream);
  if (e != cudaSuccess) return e;
  const bool wide = static_cast<long long>(p.c.T) * p.Hq <= 4096;
  if (p.c.D == 128)
    return wide ? launch_merge<128, 4>(p, rows, stream) : launch_merge<128, 1>(p, rows, stream);
  return wide ? launch_merge<64, 4>(p, rows, stream) : launch_merge<64, 1>(p, rows, stream);
}

}  // namespace attn
