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
//     query tiles an interval of its own), found by the load warp and handed to
//     the other roles through shared memory.  Documents far from a row cost it
//     nothing, and an item that sees nothing is not loaded at all.
//   * Two spare warps clear the rows of V that lie outside of the item's
//     visible span in its first and last tile before the MMA reads them: their
//     weights are 0, but 0 * NaN in a cache's unused tail would not be.
//   * Prefill (kSplit = false): an item is (batch, head, 256 query rows), handed
//     out by cluster launch control.
//   * Decode (kSplit = true): the rows of an item are the query heads that share
//     a KV head: those of 128 / G requests per tile for the shared prefix, of
//     one request for its own keys.  The key tiles of all items, laid end to
//     end, are cut into equal runs, one per CTA, whatever the lengths are; an
//     item cut by a run's end leaves fp32 partial states that a second kernel
//     merges through their log-sum-exp.  A prefix tile is read once for 256
//     rows, and at fewer than ~300 rows its bytes cost more than its products.
#pragma once

#include <cuda_bf16.h>
#include <limits.h>
#include <math_constants.h>

#include <atomic>

#include "fwd_tile.cuh"
#include "score_mod.cuh"

namespace attn {
namespace {

constexpr int kModThreads = 640;  // 16 softmax warps, load, MMA, 2 warps that clear V edges
constexpr int kModWarpLoad = 16, kModWarpMma = 17, kModWarpEdge = 18;
constexpr int kWorkReaders = 19;  // everyone but the load warp
// setmaxnreg split of the 61440 registers the launch gets (640 threads x 96)
constexpr uint32_t kModRegSoftmax = 104, kModRegOther = 64;
static_assert(4 * 128 * kModRegSoftmax + 128 * kModRegOther <= 640 * 96, "register split");

// One work item, written by the load warp.  Key tiles are relative to tile0.
struct Work {
  int n;          // key tiles to load (0: no row sees any key); -1: no more work
  int tile0;      // first key tile
  int a[2], b[2]; // query tile t uses tiles [a[t], b[t])
  int edges;      // bit 0 / 1: V rows outside [lo, hi) in the first / last tile to clear
  int lo, hi;     // visible span of the item
  int id;         // prefill: batch * Hq + head; decode: KV head
  int q0;         // prefill: first query row; decode: first request of tile 0
  int kind;       // decode: 0 shared prefix, 1 own keys
  int slot;       // decode: where its partial states go
};

struct ModMisc {
  uint64_t q_full, q_empty, unit_done;
  uint64_t s_full[2], s_read[2], p_full[2], o_done[2];
  uint64_t mma_done;
  uint64_t edge_next;     // the next V tile of the ring is an edge tile (one phase each)
  uint64_t v_edge;        // it is cleared (one phase each)
  uint64_t kv_full[8], kv_empty[8];
  uint64_t clc_full;      // the answer to the request for more work arrived
  uint64_t work_full[2], work_empty[2];
  uint4 clc_resp;
  Work work[2];           // item k in slot k % 2
  uint32_t tmem_base;
  int abort_flag;
};

// What the softmax warps know about a row: it sees keys [lo, hi) of the item's
// K/V, and with a bias key j gets -slope * (|pos - j| - ref), pos and j counted
// alike.
struct RowInfo {
  int lo, hi, pos, ref;
  float slope;  // times log2(e)
};

// Packed 2^... helpers ------------------------------------------------------

// tanh_poly of score_mod.cuh on two values, times cap_out, minus m.
struct CapCoef {
  uint64_t c[6];
};
__device__ __forceinline__ CapCoef cap_coef(float out) {
  const float c[6] = {0x1.ffffecp-1f, -0x1.5549d8p-2f, 0x1.0ffd3ap-3f,
                      -0x1.a697a8p-5f, 0x1.11f45ap-6f, -0x1.90d924p-9f};
  CapCoef r;
#pragma unroll
  for (int i = 0; i < 6; ++i) r.c[i] = f32x2(c[i] * out, c[i] * out);
  return r;
}
__device__ __forceinline__ uint64_t cap2(const CapCoef& k, uint64_t x, uint64_t add) {
  const uint64_t y = mul_f32x2(x, x);
  uint64_t t = fma_f32x2(y, k.c[5], k.c[4]);
#pragma unroll
  for (int i = 3; i >= 0; --i) t = fma_f32x2(y, t, k.c[i]);
  return fma_f32x2(x, t, add);
}

// The pass over one tile of 64 scores of a thread (half a row): from raw
// products s to weights, in place.  Returns by reference the tile's maximum
// for the row (both halves) in `mx` and leaves s in log2 units (kCap && !kBias:
// still raw; the cap is applied with the exponential).
template <bool kCap, bool kBias>
struct Scores {
  // kb: key of s[0].  masked: some of the warp's rows do not see all 128 keys.
  __device__ static __forceinline__ float prepare(float (&s)[64], const ModKernelParams& p,
                                                  const RowInfo& row, int kb, bool masked,
                                                  bool& poly) {
    poly = true;
    if constexpr (kCap) {
      // the polynomial holds while |x| <= 1; garbage in unseen keys only
      // chooses the slower path
      float a0 = 0.f, a1 = 0.f;
#pragma unroll
      for (int i = 0; i < 64; i += 4) {
        a0 = max3f(a0, fabsf(s[i]), fabsf(s[i + 1]));
        a1 = max3f(a1, fabsf(s[i + 2]), fabsf(s[i + 3]));
      }
      poly = __all_sync(0xFFFFFFFFu, fmaxf(a0, a1) * p.mod.cap_in <= 1.f);
    }
    if constexpr (kBias) {
      if constexpr (kCap) {
        if (poly) {
          const CapCoef c = cap_coef(p.mod.cap_out);
          const uint64_t in2 = f32x2(p.mod.cap_in, p.mod.cap_in), zero = f32x2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 64; i += 2)
            unpack_f32x2(cap2(c, mul_f32x2(f32x2(s[i], s[i + 1]), in2), zero), s[i], s[i + 1]);
        } else {
#pragma unroll
          for (int i = 0; i < 64; ++i) s[i] = tanh_any(s[i] * p.mod.cap_in) * p.mod.cap_out;
        }
      }
      const uint64_t mul = kCap ? f32x2(1.f, 1.f) : f32x2(p.scale_log2, p.scale_log2);
      // |pos - j| is linear in j over the keys that the row sees, but where
      // they lie on both sides of pos
      const bool left = row.hi - 1 <= row.pos || kb + 63 <= row.pos;
      const bool right = row.lo >= row.pos || kb >= row.pos;
      if (__all_sync(0xFFFFFFFFu, left || right)) {
        const float sl = left ? row.slope : -row.slope;
        // bias = sl * (j - c0), c0 = pos - ref (left) or pos + ref (right);
        // the difference is small whatever its terms are
        const unsigned c0 = static_cast<unsigned>(row.pos) +
                            static_cast<unsigned>(left ? -row.ref : row.ref);
        const float rel = static_cast<float>(static_cast<int>(static_cast<unsigned>(kb) - c0));
        uint64_t off[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) off[i] = f32x2(sl * (2 * i), sl * (2 * i + 1));
#pragma unroll
        for (int g = 0; g < 64; g += 8) {
          const float b0 = sl * (rel + g);
          const uint64_t b2 = f32x2(b0, b0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = g + 2 * i;
            unpack_f32x2(fma_f32x2(f32x2(s[e], s[e + 1]), mul, add_f32x2(b2, off[i])), s[e],
                         s[e + 1]);
          }
        }
      } else {
        const unsigned d0 = static_cast<unsigned>(row.pos) - static_cast<unsigned>(kb);
        float m1, unused;
        unpack_f32x2(mul, m1, unused);
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          const int dist = abs(static_cast<int>(d0 - i)) - row.ref;
          s[i] = fmaf(s[i], m1, -row.slope * static_cast<float>(dist));
        }
      }
    }
    if (masked) {
      const int from = row.lo - kb, to = row.hi - kb;  // columns [from, to) seen
#pragma unroll
      for (int i = 0; i < 64; ++i)
        if (i < from || i >= to) s[i] = -CUDART_INF_F;
    }
    float a0 = fmaxf(s[0], s[1]), a1 = fmaxf(s[2], s[3]);
    float a2 = fmaxf(s[4], s[5]), a3 = fmaxf(s[6], s[7]);
#pragma unroll
    for (int i = 8; i < 64; i += 8) {
      a0 = max3f(a0, s[i], s[i + 1]);
      a1 = max3f(a1, s[i + 2], s[i + 3]);
      a2 = max3f(a2, s[i + 4], s[i + 5]);
      a3 = max3f(a3, s[i + 6], s[i + 7]);
    }
    float mx = max3f(a0, a1, fmaxf(a2, a3));
    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));  // the row's other half
    if (mx == -CUDART_INF_F) return mx;
    if constexpr (kBias) return mx;
    // the cap is monotone: the largest raw score is the largest capped one
    if constexpr (kCap) return tanh_any(mx * p.mod.cap_in) * p.mod.cap_out;
    return mx * p.scale_log2;
  }

  // pk = 2^(score - m) as bf16 pairs, low key first; returns their sum in
  // fp32 before the rounding to bf16 (2^-9 of a weight on average: its effect
  // on O is that of the rounding of O itself).  Unseen keys are exactly 0.
  __device__ static __forceinline__ float weights(const float (&s)[64], const ModKernelParams& p,
                                                  float neg_m, bool masked, bool poly,
                                                  uint32_t (&pk)[32]) {
    const uint64_t negm2 = f32x2(neg_m, neg_m);
    uint64_t acc0 = f32x2(0.f, 0.f), acc1 = acc0;
    auto emit = [&](int i, uint64_t x01, uint64_t x23) {
      float x0, x1, x2, x3;
      unpack_f32x2(x01, x0, x1);
      unpack_f32x2(x23, x2, x3);
      float p0 = ex2_approx(x0), p1 = ex2_approx(x1), p2 = ex2_approx(x2), p3 = ex2_approx(x3);
      if (masked) {  // an unseen score is -inf, but what became of it need not be
        p0 = s[i] == -CUDART_INF_F ? 0.f : p0;
        p1 = s[i + 1] == -CUDART_INF_F ? 0.f : p1;
        p2 = s[i + 2] == -CUDART_INF_F ? 0.f : p2;
        p3 = s[i + 3] == -CUDART_INF_F ? 0.f : p3;
      }
      acc0 = add_f32x2(acc0, f32x2(p0, p1));
      acc1 = add_f32x2(acc1, f32x2(p2, p3));
      pk[i / 2] = pack_bf16x2(p0, p1);
      pk[i / 2 + 1] = pack_bf16x2(p2, p3);
    };
    if constexpr (kBias) {
#pragma unroll
      for (int i = 0; i < 64; i += 4)
        emit(i, add_f32x2(f32x2(s[i], s[i + 1]), negm2), add_f32x2(f32x2(s[i + 2], s[i + 3]), negm2));
    } else if constexpr (kCap) {
      if (poly) {
        const CapCoef c = cap_coef(p.mod.cap_out);
        const uint64_t in2 = f32x2(p.mod.cap_in, p.mod.cap_in);
#pragma unroll
        for (int i = 0; i < 64; i += 4)
          emit(i, cap2(c, mul_f32x2(f32x2(s[i], s[i + 1]), in2), negm2),
               cap2(c, mul_f32x2(f32x2(s[i + 2], s[i + 3]), in2), negm2));
      } else {
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          float x[4];
#pragma unroll
          for (int v = 0; v < 4; ++v)
            x[v] = fmaf(tanh_any(s[i + v] * p.mod.cap_in), p.mod.cap_out, neg_m);
          emit(i, f32x2(x[0], x[1]), f32x2(x[2], x[3]));
        }
      }
    } else {
      const uint64_t scale2 = f32x2(p.scale_log2, p.scale_log2);
#pragma unroll
      for (int i = 0; i < 64; i += 4)
        emit(i, fma_f32x2(f32x2(s[i], s[i + 1]), scale2, negm2),
             fma_f32x2(f32x2(s[i + 2], s[i + 3]), scale2, negm2));
    }
    float u0, u1;
    unpack_f32x2(add_f32x2(acc0, acc1), u0, u1);
    return u0 + u1;
  }
};

// Everything below indexes a warp's loop over work items: item k is in slot
// k % 2 from work_full (phase k / 2) until every reader arrived on work_empty.
__device__ __forceinline__ bool work_wait(ModMisc& ms, const ModKernelParams& p, int k,
                                          uint32_t abort_flag, uint32_t site) {
  return warp_all(mbar_wait(&ms.work_full[k & 1], (k >> 1) & 1, abort_flag, p.err, site,
                            p.wait_limit_ns));
}
__device__ __forceinline__ void work_done(ModMisc& ms, int k, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(&ms.work_empty[k & 1]);
}

// Prefill item u (warp-wide): the query rows, and the key tiles they see.
__device__ __forceinline__ Work plan_unit(const ModKernelParams& p, int u, int lane) {
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
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int first = w.q0 + t * kBM;
    lo[t] = INT_MAX;
    hi[t] = 0;
    if (p.ranges) {
      const int2* rg = reinterpret_cast<const int2*>(p.ranges) +
                       static_cast<size_t>(bh / p.Hq) * p.Nq;
#pragma unroll
      for (int i = 0; i < kBM / 32; ++i) {
        const int row = first + i * 32 + lane;
        if (row < p.Nq) {
          const int2 r = rg[row];
          const int l = max(r.x, 0);
          int h = min(r.y, p.Nk);
          if (p.causal) h = min(h, p.q_offset + row + 1);
          if (l < h) {
            lo[t] = min(lo[t], l);
            hi[t] = max(hi[t], h);
          }
        }
      }
      lo[t] = __reduce_min_sync(0xFFFFFFFFu, lo[t]);
      hi[t] = __reduce_max_sync(0xFFFFFFFFu, hi[t]);
    } else if (first < p.Nq) {
      lo[t] = 0;
      hi[t] = p.causal ? min(p.Nk, p.q_offset + min(first + kBM, p.Nq)) : p.Nk;
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

__device__ __forceinline__ int request_len(const ModKernelParams& p, int b) {
  return p.lens ? min(max(p.lens[b], 0), p.Nk) : p.Nk;
}
__device__ __forceinline__ int key_tiles(int keys) { return (keys + kBN - 1) / kBN; }

// Inclusive sum over the warp's lanes.
__device__ __forceinline__ int warp_scan(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += up;
  }
  return x;
}

// Decode: walks the key tiles [x, end) of this CTA through the items (warp-wide).
struct SplitPlan {
  long long x, end;    // tiles of all items, laid end to end: shared prefix first
  long long prefix;    // tiles of the shared prefix's items
  long long before;    // own-key tiles of the requests in front of block b0, per KV head
  int b0;              // first of the 32 requests that the lanes hold
  int tiles, scan;     // this lane's request: its tiles and their inclusive sum

  __device__ __forceinline__ void load_block(const ModKernelParams& p, int lane) {
    tiles = b0 + lane < p.B ? key_tiles(request_len(p, b0 + lane)) : 0;
    scan = warp_scan(tiles, lane);
  }
  __device__ __forceinline__ void start(const ModKernelParams& p, int lane) {
    long long own = 0;
    for (int b = lane; b < p.B; b += 32) own += key_tiles(request_len(p, b));
#pragma unroll
    for (int d = 16; d >= 1; d /= 2) own += __shfl_xor_sync(0xFFFFFFFFu, own, d);
    prefix = static_cast<long long>(p.Hkv) * p.row_blocks * p.prefix_tiles;
    const long long total = prefix + own * p.Hkv;
    const long long run = split_run(total, gridDim.x);
    x = min(run * blockIdx.x, total);
    end = min(x + run, total);
    before = 0;
    b0 = 0;
    load_block(p, lane);
  }
  __device__ __forceinline__ Work next(const ModKernelParams& p, int lane) {
    Work w;
    w.n = -1;
    w.edges = 0;
    w.a[0] = w.a[1] = w.b[0] = w.b[1] = 0;
    w.lo = 0;
    if (x >= end) return w;
    if (x < prefix) {
      const int item = static_cast<int>(x / p.prefix_tiles);
      w.tile0 = static_cast<int>(x % p.prefix_tiles);
      w.n = static_cast<int>(min(static_cast<long long>(p.prefix_tiles - w.tile0), end - x));
      w.kind = 0;
      w.id = item / p.row_blocks;
      w.q0 = (item % p.row_blocks) * 2 * p.per_tile;
      w.hi = p.Np;
      w.slot = item + static_cast<int>(blockIdx.x);
      w.b[0] = w.n;
      w.b[1] = w.q0 + p.per_tile < p.B ? w.n : 0;
    } else {
      long long y = x - prefix;
      for (;;) {  // the block of 32 requests that holds tile y
        const long long block = static_cast<long long>(__shfl_sync(0xFFFFFFFFu, scan, 31)) * p.Hkv;
        if (y < before + block) break;
        before += block;
        b0 += 32;
        load_block(p, lane);
      }
      y -= before;
      const unsigned behind =
          __ballot_sync(0xFFFFFFFFu, y < static_cast<long long>(scan) * p.Hkv);
      const int at = __ffs(behind) - 1;
      const int nt = __shfl_sync(0xFFFFFFFFu, tiles, at);
      y -= static_cast<long long>(__shfl_sync(0xFFFFFFFFu, scan, at) - nt) * p.Hkv;
      w.id = static_cast<int>(y / nt);
      w.tile0 = static_cast<int>(y % nt);
      w.n = static_cast<int>(min(static_cast<long long>(nt - w.tile0), end - x));
      w.kind = 1;
      w.q0 = b0 + at;
      w.hi = request_len(p, w.q0);
      w.slot = w.q0 * p.Hkv + w.id + static_cast<int>(blockIdx.x);
      w.b[0] = w.n;
      if (w.hi < min((w.tile0 + w.n) * kBN, p.Nk)) w.edges = 2;
    }
    x += w.n;
    return w;
  }
};

template <int D, bool kSplit, bool kCap, bool kBias>
__global__ void __launch_bounds__(kModThreads, 1)
    mod_attn_kernel(const __grid_constant__ ModKernelParams p) {
  using C = Cfg<D, false>;
  constexpr uint32_t kS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ ModMisc ms;
  const uint32_t abort_flag = smem_u32(&ms.abort_flag);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- setup: barriers (load warp), TMEM (MMA warp)
  if (warp == kModWarpLoad && lane == 0) {
    mbar_init(&ms.q_full, 1);
    mbar_init(&ms.q_empty, 1);
    mbar_init(&ms.unit_done, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&ms.s_full[t], 1);
      mbar_init(&ms.s_read[t], 8);
      mbar_init(&ms.p_full[t], 8);
      mbar_init(&ms.o_done[t], 1);
      mbar_init(&ms.work_full[t], 1);
      mbar_init(&ms.work_empty[t], kWorkReaders);
    }
    mbar_init(&ms.mma_done, 1);
    mbar_init(&ms.edge_next, 1);
    mbar_init(&ms.v_edge, 2);
    mbar_init(&ms.clc_full, 1);
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

  if (warp < 16) {
    // =====================================================================
    // softmax + epilogue: warps 8t .. 8t + 7 serve query tile t; a warp has 16
    // rows, threads i and i + 16 the two 64-key halves of row i (the layout of
    // fwd_sm103a.cu).
    // =====================================================================
    reg_alloc<kModRegSoftmax>();
    const int t = warp >> 3;
    const int lbase = (warp & 3) * 32 + ((warp >> 2) & 1) * 16;  // first TMEM lane of the warp
    const int r = lbase + (lane & 15);                           // row within the tile
    const int c = lane >> 4;                                     // column half of the row
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(lbase) << 16);
    const uint32_t s_addr = lane_addr + (t ? C::kColS1 : C::kColS0);
    const uint32_t o_addr = lane_addr + (t ? C::kColO1 : C::kColO0);
    uint32_t step = 0;   // tiles done by this query tile: phase of s_full
    uint32_t units = 0;  // items that this query tile took part in: phase of o_done
    for (int k = 0;; ++k) {
      if (!work_wait(ms, p, k, abort_flag, kErrWaitSoftmax)) break;
      const Work& w = ms.work[k & 1];
      const int n_all = w.n, tile0 = w.tile0, ja = w.a[t], jb = w.b[t];
      const int id = w.id, q0 = w.q0, kind = w.kind, slot = w.slot, wlo = w.lo, whi = w.hi;
      work_done(ms, k, lane);
      if (n_all < 0) break;
      // the row: which query, which keys
      RowInfo row;
      bool valid;
      size_t out = 0;  // its row in the outputs
      int head = 0;
      row.lo = wlo;
      row.hi = whi;
      if constexpr (kSplit) {
        const int G = p.G;
        const int req = kind ? 0 : r / G;
        const int b = q0 + (kind ? 0 : t * p.per_tile) + req;
        const int g = r - req * G;
        valid = jb > 0 && (kind ? r < G : req < p.per_tile) && b < p.B;
        head = id * G + g;
        row.pos = 0;
        if constexpr (kBias) {
          // positions count from the item's first key
          if (valid) row.pos = (kind ? whi : p.Np + request_len(p, b)) - 1;
        }
        out = kind ? static_cast<size_t>(slot) * G + r
                   : static_cast<size_t>(slot) * p.pre_rows + t * kBM + r;
      } else {
        const int i = q0 + t * kBM + r;
        valid = i < p.Nq;
        head = id % p.Hq;
        row.pos = p.q_offset + i;
        out = static_cast<size_t>(id) * p.Nq + i;
        if (valid) {
          row.lo = 0;
          row.hi = p.Nk;
          if (p.ranges) {
            const int2 rg = reinterpret_cast<const int2*>(
                p.ranges)[static_cast<size_t>(id / p.Hq) * p.Nq + i];
            row.lo = max(rg.x, 0);
            row.hi = min(rg.y, p.Nk);
          }
          if (p.causal) row.hi = min(row.hi, row.pos + 1);
          if (row.lo >= row.hi) row.lo = row.hi = 0;
        }
      }
      row.slope = 0.f;
      row.ref = 0;
      if constexpr (kBias) {
        if (valid) {
          row.slope = p.mod.slopes[head] * kLog2e;
          if constexpr (kSplit) {
            // nearest: the query's own position; farthest: the first key of all
            if (row.slope < 0.f) row.ref = (kind ? p.Np : 0) + row.pos;
          } else if (row.lo < row.hi) {
            row.ref = bias_ref(row.slope, row.pos, row.lo, row.hi);
          }
        }
      }
      const bool live = __any_sync(0xFFFFFFFFu, valid && row.lo < row.hi);
      float m = -CUDART_INF_F, l = 0.f;  // l: sum over this thread's half of the row
      bool ok = true;
      for (int j = ja; j < jb; ++j, ++step) {
        if (!warp_all(mbar_wait(&ms.s_full[t], step & 1, abort_flag, p.err, kErrWaitSoftmax,
                                p.wait_limit_ns))) {
          ok = false;
          break;
        }
        const int kt = (tile0 + j) * kBN;  // first key of the tile
        if (!live || !__any_sync(0xFFFFFFFFu, row.lo < kt + kBN && row.hi > kt)) {
          // no row of the warp sees a key of this tile
          if (live) {
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) pk[i] = 0;
            tc_fence_after();
            tmem_st_pair32<32>(s_addr, pk);
            tmem_st_wait();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (C::kSplitS) mbar_arrive(&ms.s_read[t]);
            mbar_arrive(&ms.p_full[t]);
          }
          continue;
        }
        tc_fence_after();
        float s[64];
        {
          uint32_t sr[64];
          tmem_ld_pair64<64>(s_addr, sr);
#pragma unroll
          for (int i = 0; i < 64; ++i) s[i] = __uint_as_float(sr[i]);
        }
        const bool masked =
            __any_sync(0xFFFFFFFFu, row.lo > kt || row.hi < kt + kBN);
        bool poly;
        const float m_tile =
            Scores<kCap, kBias>::prepare(s, p, row, kt + c * 64, masked, poly);
        if constexpr (C::kSplitS) {
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
        const float rsum = Scores<kCap, kBias>::weights(s, p, neg_m, masked, poly, pk);
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
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.p_full[t]);
      }
      if (!ok) break;
      if (jb > ja) {
        ok = warp_all(mbar_wait(&ms.o_done[t], units & 1, abort_flag, p.err, kErrWaitCorr,
                                p.wait_limit_ns));
        ++units;
        if (!ok) break;
      }
      if (kSplit && !live) continue;
      tc_fence_after();
      // ---- epilogue: O / l and the LSE; a row that saw nothing gives 0 and -inf
      const float l_row = l + __shfl_xor_sync(0xFFFFFFFFu, l, 16);
      const bool none = l_row == 0.f;
      const float inv = none ? 0.f : 1.f / l_row;
      const float lse2 = none ? -CUDART_INF_F : m + __log2f(l_row);
#pragma unroll
      for (int kk = 0; kk < D / 64; ++kk) {
        uint32_t v[32];  // columns c * D / 2 + [32 kk, 32 kk + 32) of the row
        if (jb > ja) {
          tmem_ld_pair32<D / 2>(o_addr + kk * 32, v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0;
        }
        if constexpr (kSplit) {
          float4* dst = reinterpret_cast<float4*>((kind ? p.part_o : p.pre_o) + out * D +
                                                  c * (D / 2) + kk * 32);
          if (valid) {
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              float4 x;
              x.x = none ? 0.f : __uint_as_float(v[4 * g]) * inv;
              x.y = none ? 0.f : __uint_as_float(v[4 * g + 1]) * inv;
              x.z = none ? 0.f : __uint_as_float(v[4 * g + 2]) * inv;
              x.w = none ? 0.f : __uint_as_float(v[4 * g + 3]) * inv;
              dst[g] = x;
            }
          }
        } else {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + out * D +
                                                c * (D / 2)) + kk * 4;
          uint32_t o2[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            o2[i] = none ? 0u
                         : pack_bf16x2(__uint_as_float(v[2 * i]) * inv,
                                       __uint_as_float(v[2 * i + 1]) * inv);
          if (valid) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
              st_global_v4_evict_first(dst + g, o2[4 * g], o2[4 * g + 1], o2[4 * g + 2],
                                       o2[4 * g + 3]);
          }
        }
      }
      if (valid && c == 0) {
        if constexpr (kSplit)
          (kind ? p.part_lse : p.pre_lse)[out] = lse2;
        else
          p.lse[out] = (lse2 - row.slope * static_cast<float>(row.ref)) * kLn2;
      }
    }
  } else if (warp == kModWarpLoad) {
    // =====================================================================
    // TMA loader and planner.  Ring items run on across work items: the item's
    // tile j is ring items 2 (j + tiles before), + 1 (K, then V).
    // =====================================================================
    reg_dealloc<kModRegOther>();
    uint32_t g = 0;         // next ring item
    uint32_t q_loads = 0;   // Q loads issued
    bool clc_pending = false, ok = true;
    uint32_t clc_done = 0;  // answers read
    SplitPlan plan;
    Work w;
    if constexpr (kSplit) {
      plan.start(p, lane);
      w = plan.next(p, lane);
    } else {
      w = plan_unit(p, static_cast<int>(blockIdx.x), lane);
    }
    for (int k = 0; ok; ++k) {
      if (k >= 2 && !warp_all(mbar_wait(&ms.work_empty[k & 1], ((k >> 1) + 1) & 1, abort_flag,
                                        p.err, kErrWaitLoad, p.wait_limit_ns)))
        break;
      if (lane == 0) {
        ms.work[k & 1] = w;
        mbar_arrive(&ms.work_full[k & 1]);
      }
      if (w.n < 0) break;
      const CUtensorMap* mk = &p.tmap_k;
      const CUtensorMap* mv = &p.tmap_v;
      int bhkv;
      uint64_t policy;
      if constexpr (kSplit) {
        if (w.kind == 0) {
          mk = &p.tmap_kp;
          mv = &p.tmap_vp;
        }
        bhkv = w.kind ? w.q0 * p.Hkv + w.id : w.id;
        // a request's own keys are read once, the prefix once per row block
        policy = w.kind || p.row_blocks == 1 ? l2_policy_evict_first() : l2_policy_evict_last();
      } else {
        bhkv = (w.id / p.Hq) * p.Hkv + (w.id % p.Hq) / p.G;
        policy = l2_policy_evict_last();
      }
      for (int it = 0; it < 2 * w.n; ++it, ++g) {
        const uint32_t s = g % kS;
        if (!warp_all(mbar_wait(&ms.kv_empty[s], ((g / kS) & 1u) ^ 1u, abort_flag, p.err,
                                kErrWaitLoad, p.wait_limit_ns))) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx_elect(&ms.kv_full[s], C::kTileBytes);
        uint8_t* dst = smem + C::kOffKV + s * C::kTileBytes;
        const CUtensorMap* map = (it & 1) ? mv : mk;
        for (int ch = 0; ch < C::kChunks; ++ch)
          tma_load_3d_elect(dst + ch * (kBM * 128), map, &ms.kv_full[s], ch * C::kAtomElems,
                            (w.tile0 + (it >> 1)) * kBN, bhkv, policy);
        if (it == 0) {
          // Q, once the previous item's last Q K^T (or copy to TMEM) read it
          if (q_loads > 0 &&
              !warp_all(mbar_wait(&ms.q_empty, (q_loads - 1) & 1, abort_flag, p.err, kErrWaitLoad,
                                  p.wait_limit_ns))) {
            ok = false;
            ++g;
            break;
          }
          const bool two = w.b[1] > w.a[1];
          if constexpr (kSplit) {
            const uint32_t rows = (w.kind ? 1 : p.per_tile) * p.G;
            mbar_arrive_expect_tx_elect(&ms.q_full, (two ? 2 : 1) * C::kChunks * rows * 128);
            for (int t = 0; t < (two ? 2 : 1); ++t)
              for (int ch = 0; ch < C::kChunks; ++ch)
                tma_load_4d_elect(smem + C::kOffQ + t * C::kTileBytes + ch * (kBM * 128),
                                  w.kind ? &p.tmap_q1 : &p.tmap_q, &ms.q_full,
                                  ch * C::kAtomElems, 0, w.id, w.q0 + t * p.per_tile,
                                  l2_policy_evict_last());
          } else {
            mbar_arrive_expect_tx_elect(&ms.q_full, 2 * C::kTileBytes);
            for (int t = 0; t < 2; ++t)
              for (int ch = 0; ch < C::kChunks; ++ch)
                tma_load_3d_elect(smem + C::kOffQ + t * C::kTileBytes + ch * (kBM * 128),
                                  &p.tmap_q, &ms.q_full, ch * C::kAtomElems, w.q0 + t * kBM, w.id,
                                  l2_policy_evict_first());
          }
          ++q_loads;
        }
      }
      if (!ok) break;
      if constexpr (kSplit) {
        w = plan.next(p, lane);
      } else {
        // everything of this item is on its way: ask for the next one
        mbar_arrive_expect_tx_elect(&ms.clc_full, 16);
        clc_try_cancel_elect(smem_u32(&ms.clc_resp), &ms.clc_full);
        clc_pending = true;
        if (!warp_all(mbar_wait(&ms.clc_full, clc_done & 1, abort_flag, p.err, kErrWaitLoad,
                                p.wait_limit_ns)))
          break;
        clc_pending = false;
        ++clc_done;
        const int nu = clc_response_ctaid_x(smem_u32(&ms.clc_resp));
        fence_proxy_async_smem();
        __syncwarp();
        if (nu < 0)
          w.n = -1;
        else
          w = plan_unit(p, nu, lane);
      }
    }
    if (abort_set(abort_flag)) {
      // let the copies still in flight land before the CTA exits
      if (q_loads > 0) drain_wait(&ms.q_full, (q_loads - 1) & 1);
      if (clc_pending) drain_wait(&ms.clc_full, clc_done & 1);
      for (uint32_t it = g > kS ? g - kS : 0u; it < g; ++it)
        drain_wait(&ms.kv_full[it % kS], (it / kS) & 1u);
    }
  } else if (warp == kModWarpMma) {
    // =====================================================================
    // MMA issuer (warp-wide, one elected thread per instruction).  Step j of an
    // item issues, per query tile, O_t += P_t V_{j-1} and S_t = Q_t K_j^T.
    // =====================================================================
    reg_dealloc<kModRegOther>();
    constexpr uint32_t kTileDesc = C::kTileBytes >> 4;
    const uint32_t desc_k = sdesc_sw128_lo(smem_u32(smem + C::kOffKV), 16);
    constexpr uint32_t kQFromK = static_cast<uint32_t>((C::kOffKV - C::kOffQ) >> 4);
    constexpr uint32_t kVFromK = static_cast<uint32_t>(((kBM * 128) >> 4) - 1) << 16;
    static_assert((kS & (kS - 1)) == 0, "ring depth must be a power of two");
    constexpr uint32_t kQ0 = 0u - kQFromK, kQ1 = kQ0 + kTileDesc;
    constexpr uint32_t kTQ0 = C::kQInTmem ? C::kColQ0 : 0, kTQ1 = C::kQInTmem ? C::kColQ1 : 0;
    // S_t = Q_t K^T: all keys, or (kHalf) the lower / upper 64
    auto issue_s = [&](int t, uint32_t b0, int half) {
      if (t) {
        if (half == 0)
          issue_s_steps<D, false, C::kColS1, kQ1, 0, kTQ1>(tmem, desc_k, b0);
        else if (half == 1)
          issue_s_steps<D, false, C::kColS1, kQ1, 1, kTQ1>(tmem, desc_k, b0);
        else
          issue_s_steps<D, false, C::kColS1, kQ1, 2, kTQ1>(tmem, desc_k, b0);
      } else {
        if (half == 0)
          issue_s_steps<D, false, C::kColS0, kQ0, 0, kTQ0>(tmem, desc_k, b0);
        else if (half == 1)
          issue_s_steps<D, false, C::kColS0, kQ0, 1, kTQ0>(tmem, desc_k, b0);
        else
          issue_s_steps<D, false, C::kColS0, kQ0, 2, kTQ0>(tmem, desc_k, b0);
      }
    };
    auto issue_pv = [&](int t, uint32_t b0, uint32_t acc) {
      if (t)
        issue_pv_steps<D, false, C::kColO1, C::kColS1, kVFromK>(tmem, b0, acc);
      else
        issue_pv_steps<D, false, C::kColO0, C::kColS0, kVFromK>(tmem, b0, acc);
    };
    auto wait = [&](uint64_t* bar, uint32_t phase) {
      return warp_all(mbar_wait(bar, phase & 1u, abort_flag, p.err, kErrWaitMma, p.wait_limit_ns));
    };
    uint32_t items = 0;          // items with keys so far
    uint32_t tiles = 0;          // key tiles so far: ring items 2 tiles ..
    uint32_t edge = 0;           // edge tiles so far
    uint32_t steps0 = 0, steps1 = 0;  // S_0, S_1 issued so far
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!work_wait(ms, p, k, abort_flag, kErrWaitMma)) break;
      const Work& w = ms.work[k & 1];
      const int n = w.n, edges = w.edges;
      const int a0 = w.a[0], a1 = w.a[1], b0 = w.b[0], b1 = w.b[1];
      work_done(ms, k, lane);
      if (n < 0) break;
      if (n == 0) continue;
      ok = wait(&ms.q_full, items);
      if constexpr (C::kQInTmem) {
        // Q_0, Q_1 into TMEM once every MMA of the previous item retired (see
        // fwd_sm103a.cu)
        if (ok && items > 0) ok = wait(&ms.unit_done, items - 1);
        if (ok) {
          tc_fence_after();
          const uint32_t q0 = desc_k + kQ0, q1 = desc_k + kQ1;
          tmem_cp_128x256b<C::kColQ0 + 0, 0>(tmem, q0);
          tmem_cp_128x256b<C::kColQ0 + 8, 2>(tmem, q0);
          tmem_cp_128x256b<C::kColQ0 + 16, 4>(tmem, q0);
          tmem_cp_128x256b<C::kColQ0 + 24, 6>(tmem, q0);
          tmem_cp_128x256b<C::kColQ1 + 0, 0>(tmem, q1);
          tmem_cp_128x256b<C::kColQ1 + 8, 2>(tmem, q1);
          tmem_cp_128x256b<C::kColQ1 + 16, 4>(tmem, q1);
          tmem_cp_128x256b<C::kColQ1 + 24, 6>(tmem, q1);
          mma_commit(&ms.q_empty);
        }
      }
      for (int j = 0; ok && j <= n; ++j) {
        const uint32_t ik = 2u * (tiles + j), iv = ik - 1u;
        const uint32_t bk = desc_k + (ik % kS) * kTileDesc, bv = desc_k + (iv % kS) * kTileDesc;
        if (j < n) ok = wait(&ms.kv_full[ik % kS], ik / kS);
        if (ok && j > 0) {
          ok = wait(&ms.kv_full[iv % kS], iv / kS);
          if (ok && (((edges & 1) && j == 1) || ((edges & 2) && j == n)))
            ok = wait(&ms.v_edge, edge++);
        }
        if (!ok) break;
        tc_fence_after();
        for (int t = 0; t < 2 && ok; ++t) {
          const int a = t ? a1 : a0, b = t ? b1 : b0;
          const bool pv = j > a && j <= b, qk = j >= a && j < b;
          const uint32_t last = (t ? steps1 : steps0) - 1u;  // the step whose P V is due
          if (pv) {
            if constexpr (C::kSplitS) {
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
            if (C::kSplitS && qk) issue_s(t, bk, 1);
          }
          if (qk) {
            if (!(C::kSplitS && pv)) issue_s(t, bk, 0);
            mma_commit(&ms.s_full[t]);
            if (t)
              ++steps1;
            else
              ++steps0;
          }
        }
        if (!ok) break;
        if (j < n) mma_commit(&ms.kv_empty[ik % kS]);
        if (j > 0) mma_commit(&ms.kv_empty[iv % kS]);
        if (!C::kQInTmem && j == n - 1) mma_commit(&ms.q_empty);
        // V_j is an edge tile: have it cleared while the softmax works on S_j.
        // Asked for here, its slot's barrier is in V_j's own phase: a warp
        // that waited for it from afar could take an earlier tile for it.
        if (j < n && (((edges & 1) && j == 0) || ((edges & 2) && j == n - 1)) && lane == 0)
          mbar_arrive(&ms.edge_next);
      }
      if (!ok) break;
      if (C::kQInTmem) mma_commit(&ms.unit_done);
      ++items;
      tiles += n;
    }
    // all issued MMAs retire before the CTA releases TMEM
    mma_commit(&ms.mma_done);
    drain_wait(&ms.mma_done, 0);
  } else {
    // =====================================================================
    // V edges: clear the rows of V that no row of the item sees
    // =====================================================================
    reg_dealloc<kModRegOther>();
    if constexpr (kSplit) {
      // CTA 0 leaves the merge kernel where every request's tiles begin
      if (blockIdx.x == 0 && warp == kModWarpEdge + 1) {
        long long before = 0;
        for (int b = 0; b < p.B; b += 32) {
          const int nt = b + lane < p.B ? key_tiles(request_len(p, b + lane)) : 0;
          const int scan = warp_scan(nt, lane);
          if (b + lane < p.B) p.plan[b + lane] = before + scan - nt;
          before += __shfl_sync(0xFFFFFFFFu, scan, 31);
        }
        if (lane == 0) p.plan[p.B] = before;
      }
    }
    uint32_t tiles = 0, asked = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!work_wait(ms, p, k, abort_flag, kErrWaitLoad)) break;
      const Work& w = ms.work[k & 1];
      const int n = w.n, edges = w.edges;
      const int from = w.lo - w.tile0 * kBN;  // rows [from, to) are seen, from the first tile on
      const int to = w.hi - w.tile0 * kBN;
      work_done(ms, k, lane);
      if (n < 0) break;
      for (int e = 0; e < 2 && ok; ++e) {
        const int j = e ? n - 1 : 0;
        const bool here = e ? (edges & 2) && !(n == 1 && (edges & 1)) : (edges & 1) != 0;
        if (!here) continue;
        const uint32_t iv = 2u * (tiles + j) + 1u;
        ok = warp_all(mbar_wait(&ms.edge_next, asked++ & 1u, abort_flag, p.err, kErrWaitLoad,
                                p.wait_limit_ns)) &&
             warp_all(mbar_wait(&ms.kv_full[iv % kS], (iv / kS) & 1u, abort_flag, p.err,
                                kErrWaitLoad, p.wait_limit_ns));
        if (!ok) break;
        uint8_t* v = smem + C::kOffKV + (iv % kS) * C::kTileBytes;
        const int r0 = from - j * kBN, r1 = to - j * kBN;
        for (int i = (warp - kModWarpEdge) * 32 + lane; i < kBN * C::kChunks * 8; i += 64) {
          const int row = (i >> 3) & (kBN - 1);
          if (row < r0 || row >= r1) reinterpret_cast<uint4*>(v)[i] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.v_edge);
      }
      tiles += n;
    }
  }

  if constexpr (kSplit) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (warp == kModWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D, bool kSplit, bool kCap, bool kBias>
cudaError_t launch_one(const ModKernelParams& p, unsigned grid, cudaStream_t stream) {
  using C = Cfg<D, false>;
  auto kernel = mod_attn_kernel<D, kSplit, kCap, kBias>;
  // the shared-memory opt-in is a per-device property of the function
  static std::atomic<bool> attr_done[64];  // zero-initialised: false
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    attr_done[dev].store(true, std::memory_order_release);
  }
  kernel<<<grid, kModThreads, C::kSmemBytes, stream>>>(p);
  return cudaGetLastError();
}

// The variant is the caller's request alone: what is not asked for is not computed.
template <int D, bool kSplit>
cudaError_t launch_variant(const ModKernelParams& p, unsigned grid, cudaStream_t stream) {
  const bool cap = p.mod.cap_out > 0.f, bias = p.mod.slopes != nullptr;
  if (cap && bias) return launch_one<D, kSplit, true, true>(p, grid, stream);
  if (cap) return launch_one<D, kSplit, true, false>(p, grid, stream);
  if (bias) return launch_one<D, kSplit, false, true>(p, grid, stream);
  return launch_one<D, kSplit, false, false>(p, grid, stream);
}

}  // namespace
}  // namespace attn
