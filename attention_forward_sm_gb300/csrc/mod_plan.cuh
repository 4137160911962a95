// The plan of a decode with modified scores: which CTA and query tile has which key
// tiles, where the partial states go, and where the merge finds a row's.  Integers and
// warp votes only, so that the host can compile it too (tests/mod_plan_host.cpp).
#pragma once

#include "internal.h"

namespace attn {
namespace {

constexpr int kKeyTile = 128;  // keys

// One work item, written by a planning warp, once for each query tile (a decode's
// own-key items: for the one that has it).  Key tiles are relative to tile0.
struct Work {
  int n;          // key tiles to load (0: no row sees any key); -1: no more work
  int tile0;      // first key tile
  int a[2], b[2]; // query tile t uses tiles [a[t], b[t])
  int edges;      // bit 0 / 1: V rows outside [lo, hi) in the first / last tile to clear
  int lo, hi;     // visible span of the item
  int id;         // prefill: batch * Hq + head; decode: KV head
  int q0;         // prefill: first query row; decode: first request of tile 0
  int kind;       // decode: 0 shared prefix, 1 own keys, 2 end of the prefix items
  int slot;       // decode: where its partial states go
  uint32_t v_first, v_last;  // ring items of V in the first and the last tile; own
                             // keys: ring items of the prefix, number of the first tile
};

__device__ __forceinline__ int request_len(const ModKernelParams& p, int b) {
  return p.lens ? min(max(p.lens[b], 0), p.Nk) : p.Nk;
}
__device__ __forceinline__ int key_tiles(int keys) { return (keys + kKeyTile - 1) / kKeyTile; }

// Inclusive sum over the warp's lanes.
__device__ __forceinline__ int warp_scan(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += up;
  }
  return x;
}

// Decode: the prefix tiles of this CTA's run, [x, end), item by item.
struct PrefixPlan {
  uint32_t begin, x, end;
  Pieces pieces = Pieces(0, 1);
  __device__ __forceinline__ void start(const ModKernelParams& p, uint32_t share) {
    const uint32_t total = prefix_total(p);
    const uint32_t runs = min(total, gridDim.x - share);
    begin = x = end = 0;
    if (blockIdx.x < runs) {
      x = run_start(total, runs, blockIdx.x);
      end = run_start(total, runs, blockIdx.x + 1);
      begin = x;
      pieces = Pieces(total, runs);
    }
  }
  __device__ __forceinline__ bool next(const ModKernelParams& p, Work& w) {
    if (x >= end) return false;
    const uint32_t tiles = p.prefix_tiles, item = x / tiles;
    w.tile0 = static_cast<int>(x - item * tiles);
    w.n = static_cast<int>(min(tiles - w.tile0, end - x));
    if (pieces.per_run > 1)
      w.n = min(w.n, static_cast<int>(pieces.tiles - (x - begin) % pieces.tiles));
    w.kind = 0;
    w.edges = 0;
    w.id = static_cast<int>(item) / p.row_blocks;
    w.q0 = (static_cast<int>(item) - w.id * p.row_blocks) * 2 * p.per_tile;
    w.lo = 0;
    w.hi = p.Np;
    w.slot = static_cast<int>(item + pieces.of(blockIdx.x, x - begin));
    w.a[0] = w.a[1] = 0;
    w.b[0] = w.n;
    w.b[1] = w.q0 + p.per_tile < p.B ? w.n : 0;
    x += w.n;
    return true;
  }
};

// Decode: query tile t's run of the requests' own key tiles (warp-wide).  Run
// r of 2 x CTAs belongs to query tile r / CTAs; the CTAs (those that have own keys)
// count from the other end than those of the prefix.  The tiles of all items are laid
// end to end, request by request, KV head by KV head.
struct OwnPlan {
  int left;        // tiles left of the run
  int run;
  Pieces pieces = Pieces(0, 1);
  int b0, at;      // request b0 + at, of a block of 32 that the lanes hold
  int id, tile0;   // KV head, tile within the item
  int len, tiles;  // this lane's request: its keys and key tiles
  uint32_t mine;   // tiles of this run

  __device__ __forceinline__ void load_block(const ModKernelParams& p, int lane) {
    len = b0 + lane < p.B ? request_len(p, b0 + lane) : 0;
    tiles = key_tiles(len);
  }
  // false: behind the last request, with tiles left: the lengths are not those that the
  // total came from, which is the caller's mistake.  The run ends here.
  __device__ __forceinline__ bool next_block(const ModKernelParams& p, int lane) {
    b0 += 32;
    if (b0 >= p.B) {
      if (lane == 0) atomicOr(p.err, kErrLens);
      left = 0;
      return false;
    }
    load_block(p, lane);
    return true;
  }
  // How many tiles there are of all requests; the first ones stay in the lanes.
  __device__ __forceinline__ uint32_t total_tiles(const ModKernelParams& p, int lane) {
    b0 = 0;
    load_block(p, lane);
    uint32_t own = tiles;
#pragma unroll 4
    for (int b = 32 + lane; b < p.B; b += 32) own += key_tiles(request_len(p, b));
    return __reduce_add_sync(0xFFFFFFFFu, own) * p.Hkv;
  }
  __device__ __forceinline__ void start(const ModKernelParams& p, int t, int lane,
                                        uint32_t total, uint32_t share) {
    const uint32_t ctas = share ? share : gridDim.x;
    const uint32_t runs = min(total, 2 * ctas);
    const uint32_t cta = gridDim.x - 1 - blockIdx.x, r = t * ctas + cta;
    uint32_t x = 0;
    mine = 0;
    if (cta < ctas && r < runs) {
      x = run_start(total, runs, r);
      mine = run_start(total, runs, r + 1) - x;
    }
    run = static_cast<int>(r);
    pieces = Pieces(total, runs);
    left = static_cast<int>(mine);
    at = id = tile0 = 0;
    if (left == 0) return;
    for (;;) {  // the block, the request and the KV head that hold tile x
      const int scan = warp_scan(tiles, lane);
      const uint32_t block = static_cast<uint32_t>(__shfl_sync(0xFFFFFFFFu, scan, 31)) * p.Hkv;
      if (x < block) {
        at = __ffs(__ballot_sync(0xFFFFFFFFu, x < static_cast<uint32_t>(scan) * p.Hkv)) - 1;
        const int nt = __shfl_sync(0xFFFFFFFFu, tiles, at);
        x -= static_cast<uint32_t>(__shfl_sync(0xFFFFFFFFu, scan, at) - nt) * p.Hkv;
        id = static_cast<int>(x / nt);
        tile0 = static_cast<int>(x - static_cast<uint32_t>(id) * nt);
        return;
      }
      x -= block;
      if (!next_block(p, lane)) return;
    }
  }
  // The next item; ring0: ring items of the prefix tiles before.
  __device__ __forceinline__ bool next(const ModKernelParams& p, int t, int lane, uint32_t ring0,
                                       Work& w) {
    if (left == 0) return false;
    const int nt = __shfl_sync(0xFFFFFFFFu, tiles, at);
    w.hi = __shfl_sync(0xFFFFFFFFu, len, at);
    w.id = id;
    w.tile0 = tile0;
    const uint32_t done = mine - left;
    w.n = min(nt - tile0, left);
    if (pieces.per_run > 1) w.n = min(w.n, static_cast<int>(pieces.tiles - done % pieces.tiles));
    w.kind = 1;
    w.q0 = b0 + at;
    w.lo = 0;
    w.slot = w.q0 * p.Hkv + id + static_cast<int>(pieces.of(run, done));
    w.a[0] = w.a[1] = 0;
    w.b[0] = t ? 0 : w.n;
    w.b[1] = t ? w.n : 0;
    w.edges = w.hi < (tile0 + w.n) * kKeyTile ? 2 : 0;
    w.v_first = ring0;
    w.v_last = done;
    left -= w.n;
    tile0 += w.n;
    if (left > 0 && tile0 == nt) {
      tile0 = 0;
      if (++id == p.Hkv) {
        id = 0;
        for (;;) {  // the next request that has keys
          const unsigned some = __ballot_sync(0xFFFFFFFFu, tiles > 0 && lane > at);
          if (some) {
            at = __ffs(some) - 1;
            break;
          }
          at = -1;
          if (!next_block(p, lane)) break;
        }
      }
    }
    return true;
  }
};

// A decode's planning warp for query tile t (warp-wide): its items, one by one, in w for
// publish(), which returns false if the wait for a free slot ran out.
template <class Publish>
__device__ __forceinline__ void plan_decode(const ModKernelParams& p, int t, int lane, Work& w,
                                            Publish&& publish) {
  bool ok = true;
  uint32_t ring = 0;  // ring items so far
  OwnPlan own;
  uint32_t total = 0, share = 0;
  // (else every CTA has both)
  const bool shared = prefix_total(p) >= gridDim.x;
  if (shared) {
    total = own.total_tiles(p, lane);
    share = own_share(gridDim.x, prefix_total(p), total, p.prefix_cost, p.own_cost);
  }
  if (p.prefix_tiles > 0) {
    PrefixPlan plan;
    plan.start(p, share);
    while (ok && plan.next(p, w)) {
      w.v_first = w.v_last = 0;  // no edges
      ring += 2 * w.n;
      ok = publish();
    }
    w.n = 0;
    w.kind = 2;
    w.a[0] = w.a[1] = w.b[0] = w.b[1] = 0;
    ok = ok && publish();
  }
  if (!shared) total = own.total_tiles(p, lane);
  own.start(p, t, lane, total, share);
  while (ok && own.next(p, t, lane, ring, w)) ok = publish();
  w.n = -1;
  ok = ok && publish();
  // CTA 0 leaves the merge kernel where every request's tiles begin, and the share, whose
  // rounding another kernel need not repeat
  if (blockIdx.x == 0 && t == 1) {
    uint32_t before = 0;
    for (int b = 0; b < p.B; b += 32) {
      const int nt = b + lane < p.B ? key_tiles(request_len(p, b + lane)) : 0;
      const int scan = warp_scan(nt, lane);
      if (b + lane < p.B) p.plan[b + lane] = before + scan - nt;
      before += __shfl_sync(0xFFFFFFFFu, scan, 31);
    }
    if (lane == 0) {
      p.plan[p.B] = before;
      p.plan[p.B + 1] = share;
    }
  }
}

// What the merge needs of ModKernelParams (a launch copies its parameters).
struct CombineParams {
  void* o;
  float* lse;
  const int* lens;
  const float* slopes;
  const float* pre_o;
  const float* pre_lse;
  const float* part_o;
  const float* part_lse;
  const uint32_t* plan;
  int B, Hq, Hkv, G, Nk, Np, row_blocks, per_tile, prefix_tiles, pre_rows;
  uint32_t prefix_total, ctas;
};

// The partial states of a row (request b, query head g of KV head hkv): count and first
// row of those of the shared prefix [0] and of the request's own keys [1], rows of
// either one slot apart.
struct RowParts {
  long long first[2] = {0, 0};
  int count[2] = {0, 0};
  __device__ __forceinline__ void prefix(const CombineParams& p, int b, int hkv, int g,
                                         uint32_t share) {
    const uint32_t all = p.prefix_total, runs = min(all, p.ctas - share);
    const int item = hkv * p.row_blocks + b / (2 * p.per_tile);
    const uint32_t t0 = static_cast<uint32_t>(item) * p.prefix_tiles;
    const Pieces pieces(all, runs);
    const uint32_t r0 = piece_of(all, runs, pieces, t0);
    count[0] = static_cast<int>(piece_of(all, runs, pieces, t0 + p.prefix_tiles - 1) - r0) + 1;
    const int in_tile = b % p.per_tile, tile = (b / p.per_tile) & 1;
    first[0] = static_cast<long long>(item + r0) * p.pre_rows + tile * 128 + in_tile * p.G + g;
  }
  // CTAs are shared out by the lengths where there are enough tiles of the prefix
  __device__ __forceinline__ static bool shared(const CombineParams& p) {
    return p.prefix_total >= p.ctas;
  }
  // What needs no result of the split kernel; then, behind it, the rest.
  __device__ __forceinline__ void before(const CombineParams& p, int b, int hkv, int g) {
    if (p.prefix_tiles > 0 && !shared(p)) prefix(p, b, hkv, g, 0);
  }
  __device__ __forceinline__ void after(const CombineParams& p, int b, int hkv, int g) {
    const uint32_t front = p.plan[b], nt = p.plan[b + 1] - front, own = p.plan[p.B] * p.Hkv;
    const uint32_t share = p.plan[p.B + 1];
    if (shared(p)) prefix(p, b, hkv, g, share);
    if (nt > 0) {
      const uint32_t runs = min(own, 2 * (share ? share : p.ctas));
      const uint32_t t0 = front * p.Hkv + hkv * nt;
      const Pieces pieces(own, runs);
      const uint32_t r0 = piece_of(own, runs, pieces, t0);
      count[1] = static_cast<int>(piece_of(own, runs, pieces, t0 + nt - 1) - r0) + 1;
      first[1] = (static_cast<long long>(b) * p.Hkv + hkv + r0) * p.G + g;
    }
  }
};

}  // namespace
}  // namespace attn
