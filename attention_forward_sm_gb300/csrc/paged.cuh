// What the kernels over a paged cache share: its layout on the device, and where
// a request's new tokens and pages are.
//
// K and V stand in pages [P, Hkv, page, D], table[b][i] naming the i-th page of
// request b.  The part of a page that belongs to one KV head is one block of
// `page` rows: a box of a tensor map, and one copy.  lens[b] counts the tokens
// of request b in the cache, the new ones among them; the new ones are the rows
// offsets[b] .. offsets[b + 1] of the dense tensors.
//
// Everything on the device is taken as it comes: lengths and offsets are clamped
// and a page number out of range stands for a page of zeros that takes no
// writes (kErrPage), so that no contents of these arrays lead out of bounds.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

__device__ __forceinline__ int clamp_len(const PagedArrays& c, int b) {
  return min(max(c.lens[b], 0), c.M * c.page);
}

// The rows [first, first + n) of the dense tensors that request b's new tokens are.
struct Rows {
  int first, n;
};
__device__ __forceinline__ Rows request_rows(const PagedArrays& c, int b) {
  if (!c.offsets) return {b, 1};
  const int lo = min(max(c.offsets[b], 0), c.T);
  const int hi = min(max(c.offsets[b + 1], lo), c.T);
  return {lo, hi - lo};
}

// Request that row t belongs to, -1 if none: one past the offsets that are <= t,
// found by a whole warp, which looks at 32 of them at a time.
__device__ __forceinline__ int find_request(const PagedArrays& c, int t, int lane) {
  if (!c.offsets) return t < c.B ? t : -1;
  int lo = 0, hi = c.B;
  const int begin = c.offsets[0];
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + (lane + 1) * step - 1;
    const bool behind = i < hi && c.offsets[i + 1] <= t;
    const int k = __popc(__ballot_sync(0xFFFFFFFFu, behind));
    hi = min(hi, lo + (k + 1) * step - 1);
    lo = min(lo + k * step, hi);
  }
  return lo < c.B && t >= begin ? lo : -1;
}

// Page that holds position pos of request b, or -1.
__device__ __forceinline__ int page_of(const PagedArrays& c, int b, int pos) {
  const int id = c.table[static_cast<size_t>(b) * c.M + (pos >> c.page_bits)];
  return static_cast<unsigned>(id) < static_cast<unsigned>(c.P) ? id : -1;
}

// Contiguous global -> shared copy, completion counted in bytes on `bar`.
__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// ---------------------------------------------------------------- e4m3 codes to bf16
// A code s eeee mmm moved to bits 15 and 10 .. 4 of a bf16 is its value times 2^-120
// (the exponents' biases are 7 and 127), subnormal codes included; a product with
// 2^(120 + e) is code * 2^e, exact.  Scale bytes (e + 127) above 134 would take the
// factor out of bf16: what is above is a second one.
constexpr uint32_t kScaleNan = 255, kScaleMost = 134;
// The least scale that a row has, 2^-100; a row of zeros has 2^0.
constexpr uint32_t kScaleLeast = 27, kScaleOfZeros = 127;

// Weights of V's codes, in f16: 2^(x + e - the largest x + e there was) stands for 2^kWeightTop
// times it, and may grow by 2^kWeightRoom before the reference follows (2^15 in all, f16
// ends below 2^16).  So a weight is rounded to 11 bits down to 2^-24 of the largest, and
// many thousands of small ones beside a single large one are not lost.  The sum of weights
// is of 2^x, over 2^kSumShift times that reference: with e between -100 and 100 and up to 2^21
// keys it stays within 32 bits.  O is 2^kWeightLift times what goes with that sum.
constexpr float kWeightTop = 10.f, kWeightRoom = 5.f, kSumShift = 8.f;
constexpr float kWeightLift = kWeightTop + kSumShift, kWeightUnit = 0x1p-18f;

// 2^d in two factors.  Quantised, the references of a row's states are up to 200 apart, where
// V's scales are, and 2^d alone would be 0 next to a sum that is as much above 1.
template <bool kQuant>
__device__ __forceinline__ float2 ex2_factors(float d) {
  return kQuant ? make_float2(ex2_approx(fmaxf(d, -100.f)), ex2_approx(fminf(d + 100.f, 0.f)))
                : make_float2(ex2_approx(d), 1.f);
}

// The codes in bytes 1 and 3 of u (the others do not matter), times the factors f.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t u, uint32_t f) {
  const uint32_t x = (u >> 4 & 0x07F007F0u) | (u & 0x80008000u);
  uint32_t y;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(f));
  return y;
}
// Two codes (the lower byte first) as f16, which holds every one exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
  return h;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Bits of the larger magnitude of two bf16; both to f16, times f.
__device__ __forceinline__ uint32_t bf16x2_top(uint32_t x) {
  return max(x << 16 & 0x7FFFFFFFu, x & 0x7FFFFFFFu);
}
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t x, float f) {
  return pack_f16x2(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xFFFF0000u) * f);
}
// The two lower and the two upper of four codes.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t x) {
  return e4m3x2_to_f16x2(static_cast<uint16_t>(x));
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t x) {
  return e4m3x2_to_f16x2(static_cast<uint16_t>(x >> 16));
}
__device__ __forceinline__ uint32_t or_of(const uint4& x) { return x.x | x.y | x.z | x.w; }
// 2^e and e of a scale byte; NaN for the one that says so.
__device__ __forceinline__ float scale_value(uint32_t scale) {
  return __uint_as_float(scale == kScaleNan ? 0x7FFFFFFFu : scale << 23);
}
__device__ __forceinline__ float scale_exponent(uint32_t scale) {
  return static_cast<float>(static_cast<int>(scale) - 127);
}
// 16 codes in order, under one factor.
__device__ __forceinline__ void e4m3_row16(const uint4& x, uint32_t f, uint32_t (&y)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = e4m3_pair(__byte_perm(w[i], 0, 0x1404), f);
    y[2 * i + 1] = e4m3_pair(__byte_perm(w[i], 0, 0x3424), f);
  }
}
__device__ __forceinline__ uint32_t e4m3_factor16(uint32_t scale) {
  return scale == kScaleNan ? 0x7FFFu : (min(scale, kScaleMost) + 120u) << 7;
}
__device__ __forceinline__ uint32_t e4m3_factor(uint32_t scale) {
  return e4m3_factor16(scale) * 0x10001u;
}

}  // namespace
}  // namespace attn
