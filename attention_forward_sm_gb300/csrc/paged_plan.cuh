// How the split attention kernels over a paged cache share out their work, and the
// partial states they leave.
#pragma once

#include <math_constants.h>

#include <type_traits>

#include "paged.cuh"

namespace attn {
namespace {

constexpr int kUnitKeys = 64;  // keys of a unit of work of the kernel for few rows

// `total` units dealt out in runs, as equal as they can be.
struct Deal {
  uint32_t runs, each, more;  // the first `more` runs have each + 1
  __device__ Deal(uint32_t total, uint32_t ctas)
      : runs(min(total, ctas)), each(runs ? total / runs : 0), more(runs ? total % runs : 0) {}
  __device__ uint32_t start(uint32_t r) const { return r * each + min(r, more); }
  __device__ uint32_t run_of(uint32_t x) const {
    const uint32_t cut = more * (each + 1);
    return x < cut ? x / (each + 1) : min(more + (x - cut) / each, runs - 1);
  }
};

struct PlanShared {
  uint32_t warp_sum[16];
  int b;
  uint32_t in_request;
  Rows rows;
  int len;
};
struct PlanPlace {
  uint32_t total;       // units of all
  uint32_t first, end;  // of this CTA
  int b;                // request that holds the first one,
  uint32_t in_request;  // and which of its units that is
  Rows rows;            // of that request, and its tokens
  int len;
};

// What a block of rows costs besides its keys, in units: its queries, and joining and
// storing what the warps have.  32 requests of 16 to 12000 tokens, bf16, 8 rows: 45.1 us
// with 2, 43.2 with 3, 43.5 with 4; 16 rows 70, 58, 49.8, and 50.1 with 6.  Quantised, whose
// units are half the bytes, 64 requests, 8 rows: 54.2 with 3, 50.8 with 4, 50.8 with 6; 16
// rows 123 with 4, 78 with 8, 81 with 16.
__host__ __device__ constexpr uint32_t block_cost(bool quant, int block_rows) {
  return quant && block_rows == 16 ? 8 : 4;
}

// An item is a block of rows of one KV head; it is worth its key tiles (one where there
// is no key, so that the rows' results are written) and block_cost, which comes first.
struct StreamPlan {
  const PagedArrays& c;
  int G, block_rows;
  uint32_t block_cost;
  __device__ StreamPlan(const PagedArrays& c, int G, int block_rows)
      : c(c), G(G), block_rows(block_rows), block_cost(attn::block_cost(c.quant, block_rows)) {}
  __device__ uint32_t tiles(int len) const {
    return static_cast<uint32_t>(max(1, (len + kUnitKeys - 1) / kUnitKeys));
  }
  __device__ int blocks(int n) const {  // of 8 or 16 rows
    return static_cast<int>((static_cast<long long>(n) * G + block_rows - 1) >>
                            (block_rows == 8 ? 3 : 4));
  }
  __device__ uint32_t units(int n, int len) const {
    return static_cast<uint32_t>(c.Hkv) * static_cast<uint32_t>(blocks(n)) *
           (tiles(len) + block_cost);
  }
  __device__ uint32_t units_of(int b) const {
    const int len = clamp_len(c, b);  // (its load beside the others)
    const Rows rows = request_rows(c, b);
    return rows.n > 0 ? units(rows.n, len) : 0;
  }
  // Where CTA `cta` of `ctas` begins and ends; all kThreads threads call this.
  template <int kThreads>
  __device__ PlanPlace place(PlanShared& sh, uint32_t cta, uint32_t ctas) const {
    const int per = (c.B + kThreads - 1) / kThreads;
    const int lo = min(static_cast<int>(threadIdx.x) * per, c.B), hi = min(lo + per, c.B);
    uint32_t own = 0;
    for (int b = lo; b < hi; ++b) own += units_of(b);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t sum = own;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += up;
    }
    if (lane == 31) sh.warp_sum[warp] = sum;
    if (threadIdx.x == 0) sh.b = c.B;
    __syncthreads();
    uint32_t before = sum - own, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += sh.warp_sum[w];
      total += sh.warp_sum[w];
    }
    PlanPlace at = {total, 0, 0, c.B, 0, {0, 0}, 0};
    const Deal deal(total, ctas);
    if (cta < deal.runs) {
      at.first = deal.start(cta);
      at.end = deal.start(cta + 1);
      if (at.first >= before && at.first - before < own) {
        int b = lo;
        uint32_t rest = at.first - before;
        for (; b < hi; ++b) {
          const uint32_t u = units_of(b);
          if (rest < u) break;
          rest -= u;
        }
        sh.b = b;
        sh.in_request = rest;
        sh.rows = request_rows(c, b);
        sh.len = clamp_len(c, b);
      }
    }
    __syncthreads();
    at.b = sh.b;
    at.in_request = sh.in_request;
    at.rows = sh.rows;
    at.len = sh.len;
    return at;
  }
};

// ---------------------------------------------------------------- the kernel for many rows
//
// An item is 2 * (128 / G) tokens of one KV head; its cost is the keys that its last
// token sees, and kItemCost for what every item takes besides (the products fill and drain,
// the epilogue).  The costs of a request's items are in arithmetic progression, so
// their sums have closed forms and nothing about them is stored.
constexpr int kTileKeys = 128;
constexpr int kItemCost = 512;
// A CTA's share of the line at least: what an item that is cut costs its CTAs (partial
// states of 128 KB, one after the other) is several key tiles, and no CTA may be left without
// one of an item that reaches into the next.  Item cost and least share of 256 and 512,
// 512 and 1024, 512 and 2048: requests of 1 to 500 tokens behind 64 to 6000 38, 35.5, 48 us;
// of 77 to 700, D 64, 29.1, 28.3, 36.9; long chunks all the same.
constexpr int kLeastShare = 1024;

struct CostShared {
  long long warp_sum[32];
  long long rest;
  int b;
};
// The line of all costs in `runs` equal stretches.
struct CostDeal {
  long long each;
  unsigned runs, more;
  __device__ CostDeal() {}
  __device__ CostDeal(long long total, unsigned ctas) {
    runs = total >= static_cast<long long>(ctas) * kLeastShare
               ? ctas
               : max(1u, static_cast<unsigned>(total) / kLeastShare);
    each = total / runs;
    more = static_cast<unsigned>(total - each * runs);
  }
  __device__ long long start(unsigned r) const { return each * r + more * r / runs; }
};
struct CostPlace {
  CostDeal deal;
  long long first, end;  // of this CTA
  long long rest;        // first's distance from the start of request b, which holds it
  int b;
};
struct CostItem {
  long long x0, cost;  // where it starts on the line, how long it is
  int row0, left, before, len;
  int h, j, n_kv;
};

struct CostPlan {
  const PagedArrays& c;
  int tokens, causal;  // of an item
  __device__ CostPlan(const PagedArrays& c, int G, int causal)
      : c(c), tokens(2 * (128 / G)), causal(causal) {}
  __device__ int items(int n) const { return (n + tokens - 1) / tokens; }
  // costs of the first j items of a KV head, j < items(n); of item j; of all
  __device__ long long before(int n, int len, int j) const {
    if (!causal) return static_cast<long long>(j) * (len + kItemCost);
    return static_cast<long long>(j) * (max(len - n, 0) + kItemCost) +
           static_cast<long long>(tokens) * (static_cast<long long>(j) * (j + 1) / 2);
  }
  __device__ long long cost(int n, int len, int j) const {
    return kItemCost + (!causal || j == items(n) - 1
                            ? len
                            : max(len - n, 0) + static_cast<long long>(j + 1) * tokens);
  }
  __device__ long long head(int n, int len) const {
    const int last = items(n) - 1;
    return before(n, len, last) + cost(n, len, last);
  }
  __device__ long long request(int b) const {
    const Rows rows = request_rows(c, b);
    return rows.n > 0 ? c.Hkv * head(rows.n, clamp_len(c, b)) : 0;
  }
  // Where CTA `cta` of `ctas` begins and ends; all kThreads threads call this.
  template <int kThreads>
  __device__ CostPlace place(CostShared& sh, unsigned cta, unsigned ctas) const {
    const int per = (c.B + kThreads - 1) / kThreads;
    const int lo = min(static_cast<int>(threadIdx.x) * per, c.B), hi = min(lo + per, c.B);
    long long own = 0;
    for (int b = lo; b < hi; ++b) own += request(b);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long sum = own;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const long long up = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += up;
    }
    if (lane == 31) sh.warp_sum[warp] = sum;
    if (threadIdx.x == 0) sh.b = c.B;
    __syncthreads();
    long long in_front = sum - own, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) in_front += sh.warp_sum[w];
      total += sh.warp_sum[w];
    }
    CostPlace at;
    at.deal = CostDeal(total, ctas);
    at.first = at.deal.start(cta);
    at.end = at.deal.start(cta + 1);
    if (cta < at.deal.runs && at.first >= in_front && at.first - in_front < own) {
      long long rest = at.first - in_front;
      int b = lo;
      for (; b < hi; ++b) {
        const long long x = request(b);
        if (rest < x) break;
        rest -= x;
      }
      sh.b = b;
      sh.rest = rest;
    }
    __syncthreads();
    at.b = sh.b;
    at.rest = sh.rest;
    return at;
  }
  // Item (h, j) of request b, at x0 on the line.
  __device__ CostItem make(int b, int h, int j, long long x0) const {
    const Rows rows = request_rows(c, b);
    const int len = clamp_len(c, b);
    CostItem i;
    i.x0 = x0;
    i.cost = cost(rows.n, len, j);
    i.row0 = rows.first + j * tokens;
    i.left = rows.n - j * tokens;
    i.before = len - rows.n + j * tokens;
    i.len = len;
    i.h = h;
    i.j = j;
    const int seen = causal ? min(len, i.before + min(i.left, tokens)) : len;
    i.n_kv = max(1, (seen + kTileKeys - 1) / kTileKeys);
    return i;
  }
  // The item that holds a CTA's first point.
  __device__ CostItem item(const CostPlace& at) const {
    const Rows rows = request_rows(c, at.b);
    const int len = clamp_len(c, at.b);
    const long long per_head = head(rows.n, len);
    const int h = static_cast<int>(at.rest / per_head);
    const long long rest = at.rest % per_head;
    int lo = 0, hi = items(rows.n) - 1;  // the last j with before(j) <= rest
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (before(rows.n, len, mid) <= rest)
        lo = mid;
      else
        hi = mid - 1;
    }
    return make(at.b, h, lo, at.first - rest + before(rows.n, len, lo));
  }
  // The first key tile of what lies behind point y of an item.
  __device__ int cut(const CostItem& i, long long y) const {
    if (y <= 0) return 0;
    if (y >= i.cost) return i.n_kv;
    return static_cast<int>(min(max(y - kItemCost, 0ll) / kTileKeys,
                                static_cast<long long>(i.n_kv)));
  }
};

// A state (maximum, sum, O) of one row that states are added to; a lane holds
// D / 32 consecutive elements of O (quantised, times 2^kWeightLift).  The maximum of a state
// that saw nothing is -inf, its sum and O 0; a NaN among the scores leaves them NaN.
template <int D, bool kQuant>
struct State {
  static constexpr int E = D / 32;
  float l = 0.f, o[E];
  __device__ State() {
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
  }
  using Vec = std::conditional_t<E == 4, float4, float2>;
  // ml: its maximum and sum; top: the largest maximum of all
  __device__ void add(float2 ml, float top, const Vec& x) {
    const float2 f = ex2_factors<kQuant>(ml.x == -CUDART_INF_F ? 0.f : ml.x - top);
    const float w = f.x * f.y;
    l = fmaf(f.x, ml.y * f.y, l);
    o[0] = fmaf(w, x.x, o[0]);
    o[1] = fmaf(w, x.y, o[1]);
    if constexpr (E == 4) {
      o[2] = fmaf(w, x.z, o[2]);
      o[3] = fmaf(w, x.w, o[3]);
    }
  }
  // Adds up `parts` states that other CTAs stored, the k-th one in row state(k) (read in
  // L2, where they are), four at a time; returns the largest maximum.
  template <class F>
  __device__ float join(const PagedParams& p, int parts, int lane, F state) {
    float top = -CUDART_INF_F;
    for (int k0 = 0; k0 < parts; k0 += 4) {
      float2 ml[4];
      Vec x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ml[i] = make_float2(-CUDART_INF_F, 0.f);
        x[i] = Vec{};
        if (k0 + i >= parts) continue;
        const size_t row = state(k0 + i);
        ml[i] = __ldcg(&p.part_ml[row]);
        x[i] = __ldcg(reinterpret_cast<const Vec*>(p.part_o + row * D) + lane);
      }
      float most = top;
#pragma unroll
      for (int i = 0; i < 4; ++i) most = fmaxf(most, ml[i].x);
      const float2 f = ex2_factors<kQuant>(top == -CUDART_INF_F ? 0.f : top - most);
      top = most;
      l = l * f.x * f.y;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= f.x * f.y;
#pragma unroll
      for (int i = 0; i < 4; ++i) add(ml[i], top, x[i]);
    }
    return top;
  }
  __device__ void store(float* to, int lane) const {
    if constexpr (E == 4)
      reinterpret_cast<float4*>(to)[lane] = make_float4(o[0], o[1], o[2], o[3]);
    else
      reinterpret_cast<float2*>(to)[lane] = make_float2(o[0], o[1]);
  }
  // O and LSE of row t, query head hq
  __device__ void finish(const PagedParams& p, int t, int hq, float top, int lane) const {
    const size_t row = static_cast<size_t>(t) * p.Hq + hq;
    const float inv = l == 0.f ? 0.f : (kQuant ? kWeightUnit : 1.f) / l;
    uint32_t* dst = static_cast<uint32_t*>(p.o) + row * (D / 2) + lane * (E / 2);
    if constexpr (E == 4)
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    else
      *dst = pack_bf16x2(o[0] * inv, o[1] * inv);
    if (lane == 0)
      p.lse[row] = l == 0.f ? -CUDART_INF_F : (top + log2f(l)) * 0.69314718055994530942f;
  }
};

// The next call's counts (all of them: that call may have more CTAs).
__device__ __forceinline__ void clear_counts(const PagedParams& p) {
  for (uint32_t i = blockIdx.x * blockDim.x + threadIdx.x; i < kPagedCounts;
       i += gridDim.x * blockDim.x)
    p.clear[i] = 0;
}

// Says that a warp's stores of a part are done, of the rows counted in *count of the lanes
// that have one; which of these lanes' rows have all `parts` of them stored now, so that
// this warp, the last one, joins them.
__device__ __forceinline__ uint32_t last_to_arrive(uint32_t* count, int parts, bool has) {
  __syncwarp();
  uint32_t before = 0;
  if (has) {
    __threadfence();
    before = atomicAdd(count, 1u);
    __threadfence();
  }
  return __ballot_sync(0xFFFFFFFFu, has && before + 1 == static_cast<uint32_t>(parts));
}

// Launches a kernel that may start while the one before it ends, and waits for that one
// itself (griddepcontrol.wait) before it reads or writes anything but its parameters.
template <class... Args>
cudaError_t launch_overlapped(void (*kernel)(Args...), dim3 grid, int threads, size_t smem,
                              cudaStream_t stream, std::common_type_t<Args>... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace
}  // namespace attn
