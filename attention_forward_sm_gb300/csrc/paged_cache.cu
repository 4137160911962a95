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
// Bound by memory.  A lane moves 8 elements of a row and D / 8 lanes a row, so that
// a row is one run of whole sectors on either side; a CTA takes up to kTokens tokens,
// whose pages are looked up once, by a warp each, ahead of the rows.
#include <cuda_fp16.h>

#include "../../include/attn.h"
#include "paged.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 16;  // tokens per CTA, at most

__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 x;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "l"(p));
  return x;
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t codes) {
  const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// One row of D values, 8 per lane; `lanes` = D / 8 consecutive lanes hold the row.
template <int D>
__device__ __forceinline__ uint2 quantise_row(const uint4& x, uint8_t* scale) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) a = max_nan(a, max_nan(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
#pragma unroll
  for (int d = 1; d < D / 8; d *= 2) a = max_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, d));
  const uint32_t bits = __float_as_uint(a);
  // a = 1.m * 2^E, 448 = 1.75 * 2^8
  int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = a > 0.f ? min(max(e, -100), 100) : 0;
  const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  *scale = static_cast<uint8_t>(a != a ? kScaleNan : 127 + e);
  uint2 q;
  q.x = pack_e4m3x4(bf16_lo(w[0]) * inv, bf16_hi(w[0]) * inv, bf16_lo(w[1]) * inv,
                    bf16_hi(w[1]) * inv);
  q.y = pack_e4m3x4(bf16_lo(w[2]) * inv, bf16_hi(w[2]) * inv, bf16_lo(w[3]) * inv,
                    bf16_hi(w[3]) * inv);
  return q;
}
__device__ __forceinline__ uint4 dequantise(const uint2& q, uint32_t scale) {
  const float f = scale_value(scale);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = e4m3x2_to_float2((i < 2 ? q.x : q.y) >> (16 * (i & 1)) & 0xFFFFu);
    w[i] = pack_bf16x2(x.x * f, x.y * f);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D, bool kQuant, bool kRead>
__global__ void __launch_bounds__(kThreads)
    cache_rows_kernel(const PagedArrays c, const CacheRows r, int tokens) {
  constexpr int kLanes = D / 8;               // of a row
  constexpr int kGroups = kThreads / kLanes;  // rows at a time
  constexpr int kAhead = 4;                   // of them in flight
  __shared__ int2 where[kTokens];             // (page, slot); page -1: none, -2: no such row
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = static_cast<int>(blockIdx.x) * tokens;
  for (int i = warp; i < tokens; i += kThreads / 32) {
    const int t = t0 + i;
    int2 at = make_int2(-2, 0);
    const int b = t < c.T ? find_request(c, t, lane) : -1;
    if (b >= 0) {
      const Rows rows = request_rows(c, b);
      const int pos = clamp_len(c, b) - rows.n + (t - rows.first);
      at = make_int2(-1, 0);
      if (pos >= 0 && t - rows.first < rows.n) {
        at = make_int2(page_of(c, b, pos), pos & (c.page - 1));
        if (at.x < 0 && lane == 0) atomicOr(r.err, kErrPage);
      }
    }
    if (lane == 0) where[i] = at;
  }
  __syncthreads();

  const int heads = 2 * c.Hkv;  // of K, then of V
  const int rows = min(tokens, c.T - t0) * heads;
  const int e0 = (threadIdx.x % kLanes) * 8;
  const bool first_lane = threadIdx.x % kLanes == 0;
  for (int i0 = threadIdx.x / kLanes; i0 < (rows + kGroups - 1) / kGroups * kGroups;
       i0 += kGroups * kAhead) {
    uint4 x[kAhead];
    uint32_t scale[kAhead];
    // where the row stands: in the dense tensors, and in the pages
    auto place = [&](int i, int2* at, bool* is_v, size_t* dense, size_t* paged) {
      const int token = i / heads, h = i % heads;
      *is_v = h >= c.Hkv;
      const int head = *is_v ? h - c.Hkv : h;
      *at = i < rows ? where[token] : make_int2(-2, 0);
      *dense = static_cast<size_t>(t0 + token) * (*is_v ? r.v_stride : r.k_stride) +
               static_cast<size_t>(head) * D + e0;
      *paged = (static_cast<size_t>(max(at->x, 0)) * c.Hkv + head) * c.page + at->y;
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      int2 at;
      bool is_v;
      size_t dense, paged;
      place(i0 + k * kGroups, &at, &is_v, &dense, &paged);
      x[k] = make_uint4(0, 0, 0, 0);
      scale[k] = 127;
      if (at.x < 0) continue;
      if constexpr (!kRead) {
        x[k] = ld_stream(static_cast<const __nv_bfloat16*>(is_v ? r.v : r.k) + dense);
      } else if constexpr (kQuant) {
        const uint2 q = *reinterpret_cast<const uint2*>(
            static_cast<const uint8_t*>(is_v ? c.vpages : c.kpages) + paged * D + e0);
        x[k].x = q.x;
        x[k].y = q.y;
        scale[k] = (is_v ? c.vscale : c.kscale)[paged];
      } else {
        x[k] = ld_stream(static_cast<const __nv_bfloat16*>(is_v ? c.vpages : c.kpages) +
                         paged * D + e0);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      int2 at;
      bool is_v;
      size_t dense, paged;
      place(i0 + k * kGroups, &at, &is_v, &dense, &paged);
      if constexpr (kRead) {
        if constexpr (kQuant) x[k] = dequantise(make_uint2(x[k].x, x[k].y), scale[k]);
        if (at.x != -2)
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? r.v_out : r.k_out) + dense) =
              x[k];
      } else if constexpr (kQuant) {
        uint8_t byte;
        const uint2 q = quantise_row<D>(x[k], &byte);
        if (at.x >= 0) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? c.vpages : c.kpages) + paged * D +
                                    e0) = q;
          if (first_lane) (is_v ? c.vscale : c.kscale)[paged] = byte;
        }
      } else if (at.x >= 0) {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? c.vpages : c.kpages) +
                                  paged * D + e0) = x[k];
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
