// attn_cache_write, attn_cache_read: new tokens' K and V into the pages of their
// requests, and back out as dense rows.
//
// Quantised, a row x of D values with largest magnitude a has the scale 2^e, e the
// least integer with a <= 448 * 2^e, and the codes e4m3(x / 2^e).  A power of two
// loses nothing against a / 448: e4m3 is a floating-point format, so the scale only
// decides where its subnormals begin, one binade earlier at worst.  In return
// x / 2^e and code * 2^e are exact (the code has 4 significant bits, bf16 holds 8),
// and a scale is a byte, e + 127, not four.  e stays within +-100, so that every
// code * 2^e is a normal bf16 number.  A row that holds a NaN has the scale byte 255
// and comes back as NaN.
//
// A lane moves 16 elements of a row (a row is one run of whole sectors on either side) and
// D / 16 lanes a row; a CTA takes up to kTokens tokens, whose pages are looked up once, by
// a warp each, ahead of the rows.  A lane keeps its head and goes through tokens, so that a
// row costs little more than its loads and stores: with 8 elements a lane, and the row's
// token and head found by division, instructions were the bound.  Long reads are bound by
// memory: 152709 tokens of 8 heads, D 128, quantised, 148 us, 93% of the measured copy.
// Writes wait for their loads, one row a lane behind the look-up of its page, more than half of
// the time: 26424 of these tokens 35 us on data that is not in L2, 69% (DRAM busy 52%,
// issue slots 61%; 29 us over and over on the same data), bf16 42, 75%.
#include "../../include/attn.h"
#include "paged.cuh"

namespace attn {
namespace {

constexpr int kThreads = 128;
constexpr int kTokens = 8;  // tokens per CTA, at most

__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 x;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "l"(p));
  return x;
}

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// A row of D values, 16 per lane, D / 16 consecutive lanes.
template <int D>
__device__ __forceinline__ uint4 quantise_row(const uint4 (&x)[2], uint32_t* scale) {
  const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
  uint32_t a = w[0] & 0x7FFF7FFFu;
#pragma unroll
  for (int i = 1; i < 8; ++i) a = max_nan_bf16x2(a, w[i] & 0x7FFF7FFFu);
#pragma unroll
  for (int d = 1; d < D / 16; d *= 2) a = max_nan_bf16x2(a, __shfl_xor_sync(0xFFFFFFFFu, a, d));
  a = max_nan_bf16x2(a, a << 16) & 0xFFFF0000u;  // of both halves, as a float's bits
  // a = 1.m * 2^E, 448 = 1.75 * 2^8
  int e = static_cast<int>(a >> 23) - 127 - 8 + ((a & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = a ? min(max(e, -100), 100) : 0;
  *scale = a > 0x7F800000u ? kScaleNan : 127 + e;
  const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = pack_e4m3x4(bf16_lo(w[2 * i]) * inv, bf16_hi(w[2 * i]) * inv,
                       bf16_lo(w[2 * i + 1]) * inv, bf16_hi(w[2 * i + 1]) * inv);
  return make_uint4(q[0], q[1], q[2], q[3]);
}
__device__ __forceinline__ void dequantise(uint4 (&x)[2], uint32_t scale) {
  uint32_t y[8];
  e4m3_row16(x[0], e4m3_factor(scale), y);
  if (scale > kScaleMost && scale != kScaleNan) {
    const uint32_t rest = ((scale - kScaleMost + 127u) << 7) * 0x10001u;
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(y[i]) : "r"(rest));
  }
  x[0] = make_uint4(y[0], y[1], y[2], y[3]);
  x[1] = make_uint4(y[4], y[5], y[6], y[7]);
}

template <int D, bool kQuant, bool kRead>
__global__ void __launch_bounds__(kThreads)
    cache_rows_kernel(const PagedArrays c, const CacheRows r, int tokens) {
  constexpr int kLanes = D / 16;              // of a row
  constexpr int kGroups = kThreads / kLanes;  // rows at a time
  constexpr int kAhead = kQuant && kRead ? 2 : 1;  // of them in flight (more: fewer CTAs)
  // of every token: the row in the pages of its first head; -1: none, -2: no such token
  __shared__ long long where[kTokens];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = static_cast<int>(blockIdx.x) * tokens;
  for (int i = warp; i < tokens; i += kThreads / 32) {
    const int t = t0 + i;
    long long at = -2;
    const int b = t < c.T ? find_request(c, t, lane) : -1;
    if (b >= 0) {
      const Rows rows = request_rows(c, b);
      const int pos = clamp_len(c, b) - rows.n + (t - rows.first);
      at = -1;
      if (pos >= 0 && t - rows.first < rows.n) {
        const int id = page_of(c, b, pos);
        if (id >= 0)
          at = static_cast<long long>(id) * c.Hkv * c.page + (pos & (c.page - 1));
        else if (lane == 0)
          atomicOr(r.err, kErrPage);
      }
    }
    if (lane == 0) where[i] = at;
  }
  __syncthreads();

  // heads of K, then of V; a group of lanes has a head, and of the tokens every step-th
  const int heads = 2 * c.Hkv, at_once = min(heads, kGroups);
  const int step = kGroups / at_once;
  const int group = threadIdx.x / kLanes, first = group / at_once;
  const int e0 = (threadIdx.x % kLanes) * 16;
  const bool first_lane = threadIdx.x % kLanes == 0;
  for (int h0 = 0; h0 < heads; h0 += at_once) {
    // (a warp's lanes stay together for the shuffles, also those with nothing to do)
    const int h = h0 + group % at_once;
    const bool mine = h < heads && first < step;
    const bool is_v = h >= c.Hkv;
    const int head = is_v ? h - c.Hkv : h;
    const long long stride = is_v ? r.v_stride : r.k_stride;
    const size_t dense0 = static_cast<size_t>(t0) * stride + static_cast<size_t>(head) * D + e0;
    void* const pages = is_v ? c.vpages : c.kpages;
    uint8_t* const scales = is_v ? c.vscale : c.kscale;
    for (int i0 = 0; i0 < tokens; i0 += step * kAhead) {
      uint4 x[kAhead][2];
      uint32_t scale[kAhead];
      long long at[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + first + k * step;
        const long long row = mine && i < tokens ? where[i] : -2;
        at[k] = row < 0 ? row : row + static_cast<long long>(head) * c.page;
        x[k][0] = x[k][1] = make_uint4(0, 0, 0, 0);
        scale[k] = 127;
        if (row < 0) continue;
        if constexpr (kRead && kQuant) {
          x[k][0] = ld_stream(static_cast<const uint8_t*>(pages) + at[k] * D + e0);
          scale[k] = scales[at[k]];
        } else {
          const __nv_bfloat16* from =
              kRead ? static_cast<const __nv_bfloat16*>(pages) + at[k] * D + e0
                    : static_cast<const __nv_bfloat16*>(is_v ? r.v : r.k) + dense0 + i * stride;
          x[k][0] = ld_stream(from);
          x[k][1] = ld_stream(from + 8);
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + first + k * step;
        if constexpr (!kRead && kQuant) {
          const uint4 q = quantise_row<D>(x[k], &scale[k]);
          if (at[k] >= 0) {
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(pages) + at[k] * D + e0) = q;
            if (first_lane) scales[at[k]] = static_cast<uint8_t>(scale[k]);
          }
        } else {
          if constexpr (kRead && kQuant) dequantise(x[k], scale[k]);
          if (at[k] < (kRead ? -1 : 0)) continue;
          uint4* to = reinterpret_cast<uint4*>(
              kRead ? static_cast<__nv_bfloat16*>(is_v ? r.v_out : r.k_out) + dense0 + i * stride
                    : static_cast<__nv_bfloat16*>(pages) + at[k] * D + e0);
          to[0] = x[k][0];
          to[1] = x[k][1];
        }
      }
    }
  }
}

template <int D, bool kQuant, bool kRead>
cudaError_t launch(const PagedArrays& c, const CacheRows& r, cudaStream_t stream) {
  // a few CTAs for every SM before they take more tokens each
  const int tokens = min(max(c.T / 1024, 1), kTokens);
  const unsigned grid = static_cast<unsigned>((c.T + tokens - 1) / tokens);
  cache_rows_kernel<D, kQuant, kRead><<<grid, kThreads, 0, stream>>>(c, r, tokens);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_rows(const PagedArrays& c, const CacheRows& r, bool read,
                              cudaStream_t stream) {
  using Launch = cudaError_t (*)(const PagedArrays&, const CacheRows&, cudaStream_t);
  static const Launch table[2][2][2] = {
      {{launch<64, false, false>, launch<64, false, true>},
       {launch<64, true, false>, launch<64, true, true>}},
      {{launch<128, false, false>, launch<128, false, true>},
       {launch<128, true, false>, launch<128, true, true>}}};
  return table[c.D == 128][c.quant][read](c, r, stream);
}

}  // namespace attn
