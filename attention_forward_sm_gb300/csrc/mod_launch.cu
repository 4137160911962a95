// Host side of mod_attn_kernel: tensor maps, the plan of a decode, its scratch,
// and the kernel that merges a decode's partial states.
#include <cuda_bf16.h>
#include <limits.h>
#include <math_constants.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "../../include/attn.h"
#include "mod_plan.cuh"
#include "score_mod.cuh"

namespace attn {
namespace {

// W warps per (request, query head), 1, 2 or 8: they merge the row's partial states,
//   L = log2 sum_c 2^(lse_c),  O = sum_c 2^(lse_c - L) O_c,
// those of the shared prefix's item and those of the request's own item.  The
// runs of key tiles give every item's first and last run, and with it its
// slots.  A lane holds D / 32 consecutive elements of O; the states are
// few and in L2, so the loads of up to four of them are in flight at once and
// nothing else is shared.  Bound by latency: 1.5 to 3 us behind the split kernel, of
// which its plan (of the prefix, where that needs no lengths) and the launch are
// hidden behind that kernel's end, and the first states come with the lse.
template <int D, int W>
__global__ void __launch_bounds__(256) mod_combine_kernel(const CombineParams p) {
  constexpr int E = D / 32;
  // programmatic dependent launch: what needs no result of the split kernel goes in
  // front of the wait for it, beside that kernel's last CTAs
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5, part = warp % W;
  const uint32_t row = blockIdx.x * (8 / W) + warp / W;
  // (no row: whole rows of warps leave, and a barrier does not count them)
  if (row >= static_cast<uint32_t>(p.B) * p.Hq) return;
  const int b = static_cast<int>(row / p.Hq), h = static_cast<int>(row % p.Hq);
  const int hkv = h / p.G, g = h % p.G;

  RowParts parts;
  parts.before(p, b, hkv, g);
  const int len = p.lens ? min(max(p.lens[b], 0), p.Nk) : p.Nk;
  const float slope = p.slopes ? p.slopes[h] : 0.f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  parts.after(p, b, hkv, g);
  const int(&count)[2] = parts.count;
  const long long(&first)[2] = parts.first;
  // this warp's parts: every W-th
  const int all_parts = count[0] + count[1];
  const int total = all_parts > part ? (all_parts - part + W - 1) / W : 0;
  auto lse_of = [&](int j) {
    const int i = part + W * j;
    return i < count[0] ? p.pre_lse[first[0] + static_cast<long long>(i) * p.pre_rows]
                        : p.part_lse[first[1] + static_cast<long long>(i - count[0]) * p.G];
  };
  using Vec = std::conditional_t<E == 4, float4, float2>;
  auto state_of = [&](int j) {
    const int i = part + W * j;
    const float* src = i < count[0]
                           ? p.pre_o + (first[0] + static_cast<long long>(i) * p.pre_rows) * D
                           : p.part_o + (first[1] + static_cast<long long>(i - count[0]) * p.G) * D;
    return reinterpret_cast<const Vec*>(src)[lane];
  };
  // the first states come in together with the lse
  constexpr int kAhead = 4;
  Vec ahead[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (i < total) ahead[i] = state_of(i);
  // the largest lse, as integers of the same order; a NaN state stays one
  int top = INT_MIN;
  for (int i = lane; i < total; i += 32) {
    const float x = lse_of(i);
    const int y = __float_as_int(x);
    top = max(top, x != x ? INT_MAX : y ^ ((y >> 31) & INT_MAX));
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  float m = total > 0 ? __int_as_float(top ^ ((top >> 31) & INT_MAX)) : -CUDART_INF_F;
  bool none = m == -CUDART_INF_F;
  float sum = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  if (!none) {
    for (int i0 = 0; i0 < total; i0 += 32) {
      const float w_lane = i0 + lane < total ? ex2_approx(lse_of(i0 + lane) - m) : 0.f;
      const int n = min(32, total - i0);
      auto add = [&](int i, const Vec& x) {
        const float w = __shfl_sync(0xFFFFFFFFu, w_lane, i);
        sum += w;
        o[0] = fmaf(w, x.x, o[0]);
        o[1] = fmaf(w, x.y, o[1]);
        if constexpr (E == 4) {
          o[2] = fmaf(w, x.z, o[2]);
          o[3] = fmaf(w, x.w, o[3]);
        }
      };
      int i = 0;
      if (i0 == 0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (k < total) add(k, ahead[k]);
        i = min(kAhead, total);
      }
#pragma unroll 4
      for (; i < n; ++i) add(i, state_of(i0 + i));
    }
  }
  if constexpr (W > 1) {
    // the row's warps through shared memory; the first one goes on
    __shared__ float sums[8][D], tops[8][2];
#pragma unroll
    for (int e = 0; e < E; ++e) sums[warp][lane * E + e] = o[e];
    if (lane == 0) {
      tops[warp][0] = m;
      tops[warp][1] = sum;
    }
    __syncthreads();
    if (part > 0) return;
    for (int i = 1; i < W; ++i) {
      const float x = tops[warp + i][0];
      m = x != x || m != m ? x + m : fmaxf(m, x);
    }
    none = m == -CUDART_INF_F;
    sum = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float x = tops[warp + i][0];
      const float w = none || x == -CUDART_INF_F ? 0.f : ex2_approx(x - m);
      sum = fmaf(w, tops[warp + i][1], sum);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(w, sums[warp + i][lane * E + e], o[e]);
    }
  }
  const float inv = none ? 0.f : 1.f / sum;
  uint32_t out[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; ++e) out[e] = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
  uint32_t* dst = static_cast<uint32_t*>(p.o) + static_cast<size_t>(row) * (D / 2) + lane * (E / 2);
  if constexpr (E == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
  else
    *dst = out[0];
  if (lane == 0) {
    float lse = none ? -CUDART_INF_F : (m + __log2f(sum)) * kLn2;
    // a negative slope is relative to the farthest key
    if (slope < 0.f && !none) lse -= slope * static_cast<float>(p.Np + len - 1);
    p.lse[row] = lse;
  }
}

template <int D, int W>
cudaError_t launch_combine(const ModKernelParams& p, unsigned ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const long long rows = static_cast<long long>(p.B) * p.Hq;
  cfg.gridDim = dim3(static_cast<unsigned>((rows + 8 / W - 1) / (8 / W)));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const CombineParams c = {p.o,        p.lse,      p.lens,     p.mod.slopes, p.pre_o,
                           p.pre_lse,  p.part_o,   p.part_lse, p.plan,       p.B,
                           p.Hq,       p.Hkv,      p.G,        p.Nk,         p.Np,
                           p.row_blocks, p.per_tile, p.prefix_tiles, p.pre_rows,
                           prefix_total(p), ctas};
  return cudaLaunchKernelEx(&cfg, mod_combine_kernel<D, W>, c);
}

void common_params(ModKernelParams* k, const ScoreMod& mod, const DeviceInfo& di) {
  k->mod = mod;
  // Never 0: an unseen score is -inf and has to stay it.  1e-37 times any product
  // below 1e30 is 0 next to a score's fp32 roundings.
  k->scale_log2 = std::max(mod.scale * kLog2e, 1e-37f);
  k->err = di.err_word;
  k->wait_limit_ns = wait_limit_ns();
}

struct DecodeLaunch {
  ModKernelParams* k;
  int D, dev;
  unsigned ctas;
  int merge_warps;  // per row: 1, 2 or 8
  size_t pre_o, pre_lse, part_o, part_lse;  // offsets into the scratch; plan at 0
};

int launch_decode(void* ctx, void* scratch, cudaStream_t stream) {
  const DecodeLaunch& d = *static_cast<DecodeLaunch*>(ctx);
  char* base = static_cast<char*>(scratch);
  d.k->plan = reinterpret_cast<uint32_t*>(base);
  d.k->pre_o = reinterpret_cast<float*>(base + d.pre_o);
  d.k->pre_lse = reinterpret_cast<float*>(base + d.pre_lse);
  d.k->part_o = reinterpret_cast<float*>(base + d.part_o);
  d.k->part_lse = reinterpret_cast<float*>(base + d.part_lse);
  using Launch = cudaError_t (*)(const ModKernelParams&, unsigned, int, cudaStream_t);
  static const Launch split[2][3] = {
      {launch_mod_split_d64_h4, launch_mod_split_d64_h8, launch_mod_split_d64_h0},
      {launch_mod_split_d128_h4, launch_mod_split_d128_h8, launch_mod_split_d128_h0}};
  // Own keys with the keys as rows (h4, h8: heads a thread holds) or, above 8
  // heads, the heads.  Measured with 64 requests of up to 4096 / 256 keys, Hkv 8,
  // D 128: 4 heads 85.8 / 19.7 us (heads as rows 91.4 / 22.4), 8 heads 103.6 /
  // 21.4 (104.3 / 22.7), 16 heads 100.1 / 27.6 (98.2 / 23.5).
  const int G = d.k->G, heads = G <= 4 ? 0 : (G <= 8 ? 1 : 2);
  cudaError_t e = split[d.D == 128][heads](*d.k, d.ctas, d.dev, stream);
  if (e == cudaSuccess)
    e = (d.D == 128 ? (d.merge_warps == 8   ? launch_combine<128, 8>
                       : d.merge_warps == 2 ? launch_combine<128, 2>
                                            : launch_combine<128, 1>)
                    : (d.merge_warps == 8   ? launch_combine<64, 8>
                       : d.merge_warps == 2 ? launch_combine<64, 2>
                                            : launch_combine<64, 1>))(*d.k, d.ctas, stream);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

// The keys [key0, key0 + nk) of a prefill.
int launch_fwd(const ModFwdParams& p, const DeviceInfo& di, int key0, int nk,
               cudaStream_t stream) {
  ModKernelParams k = {};
  if (int rc = encode_rows(&k.tmap_q, p.q, p.D, p.Nq, static_cast<long long>(p.B) * p.Hq, 128))
    return rc;
  const long long heads = static_cast<long long>(p.B) * p.Hkv;
  const size_t skip = static_cast<size_t>(key0) * p.D * 2;
  if (int rc = encode_rows(&k.tmap_k, static_cast<const char*>(p.k) + skip, p.D, nk, heads, 128,
                           p.Nk))
    return rc;
  if (int rc = encode_rows(&k.tmap_v, static_cast<const char*>(p.v) + skip, p.D, nk, heads, 128,
                           p.Nk))
    return rc;
  k.o = p.o;
  k.lse = p.lse;
  k.ranges = p.ranges;
  k.B = p.B;
  k.Hq = p.Hq;
  k.Hkv = p.Hkv;
  k.G = p.Hq / p.Hkv;
  k.Nq = p.Nq;
  k.Nk = nk;
  k.causal = p.causal;
  k.q_offset = p.q_offset - key0;
  k.key0 = key0;
  // Rows that see different keys: items of later rows, as a rule the longer
  // ones, first, in groups of heads whose K and V take about a third of the
  // L2 (as in fwd_sm103a.cu).
  k.longest_first = p.causal || p.ranges;
  const double kv_bytes = 4.0 * nk * p.D;
  const int kv_heads = std::max(1, std::min(static_cast<int>(40.0e6 / kv_bytes), p.B * p.Hkv));
  k.group_heads = kv_heads * k.G;
  k.o_sectors = (reinterpret_cast<uintptr_t>(p.o) & 31u) == 0;
  common_params(&k, p.mod, di);
  const unsigned grid =
      static_cast<unsigned>((p.Nq + 255ll) / 256 * p.B * p.Hq);
  const cudaError_t e = p.D == 128 ? launch_mod_fwd_d128(k, grid, di.dev, stream)
                                   : launch_mod_fwd_d64(k, grid, di.dev, stream);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

// Adds a segment's result (O, LSE of the output tensors) to the sum of those before,
//   acc = sum_i e^(LSE_i - T) O_i,  state = (T, sum_i e^(LSE_i - T)),
// T the largest LSE so far.  The first segment starts the sum, the last one leaves
// O = acc / sum and LSE = T + ln sum in the output.  A warp per row and turn; 10
// bytes read and written per element, next to 2^18 keys a row.
template <int D>
__global__ void __launch_bounds__(256)
    segment_merge_kernel(__nv_bfloat16* o, float* lse, float* acc, float2* states, long long rows,
                         bool first, bool last) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long warps = static_cast<long long>(gridDim.x) * 8;
  for (long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); row < rows;
       row += warps) {
    const float2 before = first ? make_float2(-CUDART_INF_F, 0.f) : states[row];
    const float x = lse[row];
    // (a NaN stays one)
    const float top = x != x || before.x != before.x ? x + before.x : fmaxf(x, before.x);
    const bool none = top == -CUDART_INF_F;
    const float wa = none ? 0.f : expf(before.x - top), ws = none ? 0.f : expf(x - top);
    const float sum = fmaf(before.y, wa, ws);
    const float out = last ? (none ? 0.f : 1.f / sum) : 1.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const long long at = row * D + i * 32 + lane;
      // (a weight of 0 takes nothing, not even from a NaN that stands there)
      float v = first || wa == 0.f ? 0.f : wa * acc[at];
      if (ws != 0.f) v = fmaf(ws, __bfloat162float(o[at]), v);
      if (last)
        o[at] = __float2bfloat16_rn(v * out);
      else
        acc[at] = v;
    }
    __syncwarp();
    if (lane == 0) {
      if (last)
        lse[row] = none ? top : top + logf(sum);
      else
        states[row] = make_float2(top, sum);
    }
  }
}

struct SegmentsLaunch {
  const ModFwdParams* p;
  const DeviceInfo* di;
  int count;  // segments that some row can see
  long long rows;
  size_t states;  // offset into the scratch
};

int launch_segments(void* ctx, void* scratch, cudaStream_t stream) {
  const SegmentsLaunch& d = *static_cast<SegmentsLaunch*>(ctx);
  const ModFwdParams& p = *d.p;
  float* acc = static_cast<float*>(scratch);
  float2* states = reinterpret_cast<float2*>(static_cast<char*>(scratch) + d.states);
  const unsigned grid =
      static_cast<unsigned>(std::min<long long>((d.rows + 7) / 8, 8ll * d.di->sms));
  for (int i = 0; i < d.count; ++i) {
    const int key0 = i * kSegmentKeys;
    if (int rc = launch_fwd(p, *d.di, key0, std::min(kSegmentKeys, p.Nk - key0), stream)) return rc;
    const bool first = i == 0, last = i == d.count - 1;
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o);
    if (p.D == 128)
      segment_merge_kernel<128><<<grid, 256, 0, stream>>>(o, p.lse, acc, states, d.rows, first,
                                                           last);
    else
      segment_merge_kernel<64><<<grid, 256, 0, stream>>>(o, p.lse, acc, states, d.rows, first,
                                                           last);
    if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_LAUNCH;
  }
  return ATTN_OK;
}

}  // namespace

int mod_fwd(const ModFwdParams& p, cudaStream_t stream) {
  DeviceInfo di;
  if (int rc = device_info(&di)) return rc;
  // without ranges, causal rows see no key behind the last one's position
  const long long seen =
      p.causal ? std::min<long long>(p.Nk, static_cast<long long>(p.q_offset) + p.Nq) : p.Nk;
  if (p.Nk <= kSegmentKeys) return launch_fwd(p, di, 0, p.Nk, stream);
  if (seen <= kSegmentKeys) return launch_fwd(p, di, 0, static_cast<int>(seen), stream);
  SegmentsLaunch d = {&p, &di, static_cast<int>((seen + kSegmentKeys - 1) / kSegmentKeys),
                      static_cast<long long>(p.B) * p.Hq * p.Nq, 0};
  d.states = static_cast<size_t>(d.rows) * p.D * sizeof(float);
  return with_own_scratch(d.states + static_cast<size_t>(d.rows) * sizeof(float2), stream,
                          launch_segments, &d);
}

int mod_decode(const ModDecodeParams& p, cudaStream_t stream) {
  DeviceInfo di;
  if (int rc = device_info(&di)) return rc;
  ModKernelParams k = {};
  k.G = p.Hq / p.Hkv;
  k.per_tile = 128 / k.G;
  if (int rc = encode_queries(&k.tmap_q1, p.q, p.D, k.G, p.Hkv, p.B, 1)) return rc;
  const long long heads = static_cast<long long>(p.B) * p.Hkv;
  if (int rc = encode_rows(&k.tmap_k, p.kcache, p.D, p.Ncap, heads, 32)) return rc;
  if (int rc = encode_rows(&k.tmap_v, p.vcache, p.D, p.Ncap, heads, 32)) return rc;
  k.row_blocks = (p.B + 2 * k.per_tile - 1) / (2 * k.per_tile);
  if (p.Np > 0) {
    if (int rc = encode_queries(&k.tmap_q, p.q, p.D, k.G, p.Hkv, p.B, k.per_tile)) return rc;
    if (int rc = encode_rows(&k.tmap_kp, p.kprefix, p.D, p.Np, p.Hkv, 128)) return rc;
    if (int rc = encode_rows(&k.tmap_vp, p.vprefix, p.D, p.Np, p.Hkv, 128)) return rc;
    k.prefix_tiles = (p.Np + 127) / 128;
  }
  k.pre_rows = p.B <= k.per_tile ? p.B * k.G : 256;
  k.o = p.o;
  k.lse = p.lse;
  k.lens = p.lens;
  k.B = p.B;
  k.Hq = p.Hq;
  k.Hkv = p.Hkv;
  k.Nk = p.Ncap;
  k.Np = p.Np;
  // What a key tile costs a CTA in us: of the prefix, 256 rows, as measured in a
  // prefill; of own keys, where the shares that follow made the call fastest, with
  // what short requests cost besides their keys.  Shares against all CTAs doing both:
  // serving sizes (64 requests of up to 1024 keys behind 16384, D 128, 4 heads per KV
  // head) 38.5 us, 42.8; 8 heads 34.7, 41.0; 1 head, 256 requests 62.6, 71.2; capped,
  // 256 behind 8192 75.0, 80.3; D 64, 128 requests 49.5, 51.2.
  const bool cap = p.mod.cap_out > 0.f, bias = p.mod.slopes != nullptr;
  k.prefix_cost = (p.D == 128 ? 1.5f : 1.2f) + (cap ? 0.6f : 0.f) + (bias ? 0.5f : 0.f);
  // The whole call at own costs of 0.45, 0.6, 0.75, 0.9, 1.2, 1.7, 64 requests as above:
  // D 64, 4 heads 32.1, 30.9, 31.5, 32.4, 31.7, 37.8, capped 41.0, 39.8, 40.0, 41.9,
  // 43.3, 47.2, 8 heads (4 KV heads) 36.8, 32.5, 28.3, 29.7, 30.6, 32.7, capped 49.7,
  // 42.1, 39.8, 36.9, 38.2, 40.7; 256 behind 8192, D 64, 4 heads 55.6, 49.4, 50.9, 53.7,
  // 60.0, 70.1, capped 72.2, 66.7, 69.5, 72.4, 80.2, 90.5; 128 behind 8192, D 64, 1
  // head, capped and biased 35.7, 32.8, 31.1, 30.0, 32.5, 35.7; 256 behind 8192, D 128
  // 90.9, 78.5, 71.4, 67.1, 65.3, 74.8, capped 114.7, 96.6, 84.9, 78.3, 75.6, 84.2,
  // biased 108.6, 91.9, 82.5, 75.7, 75.6, 83.7: no matter of caps or heads at D 128.
  if (p.D == 128)
    k.own_cost = 1.15f;
  else if (k.G <= 4)
    k.own_cost = cap ? 0.75f : 0.6f;
  else
    k.own_cost = cap ? 1.1f : 0.8f;
  common_params(&k, p.mod, di);
  const long long prefix_items =
      p.Np > 0 ? static_cast<long long>(p.Hkv) * k.row_blocks : 0;
  const long long most_tiles = prefix_items * k.prefix_tiles + heads * ((p.Ncap + 127ll) / 128);
  DecodeLaunch d = {};
  d.k = &k;
  d.D = p.D;
  d.dev = di.dev;
  d.ctas = static_cast<unsigned>(std::min<long long>({di.sms, most_tiles, kMostCtas}));
  // The merge takes more warps per row where rows with many parts are few.  Measured,
  // the whole call in us with 8, 2, 1 warps: 64 rows of 76 parts 17, -, 38; 256 of 5
  // 84, -, 90; 768 of 20 23.5, -, 26; 800 of 5 15.8, -, 14.7; 2048 of 20 43.8, 37.9,
  // 39.8; 8192 of 6 105, 81, 78.
  const long long own_runs = std::min(2ll * d.ctas, most_tiles);
  const long long parts =
      std::max((own_runs + heads - 1) / heads,
               p.Np > 0 ? (std::min<long long>(d.ctas, prefix_items * k.prefix_tiles) +
                           prefix_items - 1) / prefix_items
                        : 0);
  const long long rows = static_cast<long long>(p.B) * p.Hq;
  d.merge_warps = rows <= 4ll * di.sms && parts >= 4    ? 8
                  : rows <= 8ll * di.sms && parts >= 8  ? 8
                  : rows <= 16ll * di.sms && parts >= 8 ? 2
                                                        : 1;
  // slot of a state: its item's number + its piece's
  // (n runs of `tiles` in all have at most tiles / kPieceTiles + 2 n pieces)
  const size_t pre_tiles = prefix_total(k), own_tiles = heads * ((p.Ncap + 127ll) / 128);
  const size_t pre = p.Np > 0 ? (prefix_items + pre_tiles / kPieceTiles + 2ull * d.ctas) * k.pre_rows
                              : 0;
  const size_t own = (heads + own_tiles / kPieceTiles + 4ull * d.ctas) * k.G;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  d.pre_o = up((static_cast<size_t>(p.B) + 2) * sizeof(uint32_t));
  d.pre_lse = d.pre_o + up(pre * p.D * sizeof(float));
  d.part_o = d.pre_lse + up(pre * sizeof(float));
  d.part_lse = d.part_o + up(own * p.D * sizeof(float));
  const size_t bytes = d.part_lse + up(own * sizeof(float));
  return with_scratch(bytes, di.dev, stream, launch_decode, &d);
}

}  // namespace attn
