// Tile shapes, shared-memory and TMEM maps and MMA issue of the prefill kernels
// (fwd_sm103a.cu, mod_sm103a.cuh).
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kBM = 128;          // query rows per tile
constexpr int kBN = 128;          // keys per K/V tile

template <int D, bool kFp8 = false>
struct Cfg {
  static constexpr int kElemBytes = kFp8 ? 1 : 2;
  static constexpr int kTileBytes = kBM * D * kElemBytes;  // a 128 x D tile (Q, K; V or V^T)
  static constexpr int kAtomElems = 128 / kElemBytes;      // elements per 128-byte swizzle row
  static constexpr int kChunks = D * kElemBytes / 128;     // 128-byte swizzle chunks per tile row
  static constexpr int kStages = (D == 128) ? 4 : 8;       // K/V ring depth
  static constexpr int kColS0 = 0, kColS1 = 128, kColO0 = 256, kColO1 = 256 + D;
  // Q K^T in two N = 64 halves, keys [64, 128) issued while the softmax
  // still works on the previous S (see the MMA warp).  With Q in shared
  // memory each half re-reads all of Q, so the halves cost 3/4 of a full
  // MMA's time each; that pays where the tensor pipe has slack (e4m3, and
  // D = 64, whose Q moreover sits in TMEM) and not at D = 128 bf16, where
  // the pipe is already busy ~3/4 of the time.
  static constexpr bool kSplitS = (D == 64) || kFp8;
  // D = 64 (bf16) has TMEM columns to spare: Q_t is copied there once per
  // unit (kColQ0, kColQ1: D / 2 columns each) and every Q K^T reads A from
  // TMEM, so an N = 64 half reads only its 2 KB of K from shared memory per
  // k-step instead of 6 KB; Q's shared-memory buffers are free once copied.
  static constexpr bool kQInTmem = (D == 64) && !kFp8;
  static constexpr int kColQ0 = 2 * 128 + 2 * D, kColQ1 = kColQ0 + D / 2;
  static constexpr int kTmemCols = 512;
  static_assert(!kQInTmem || kColQ1 + D / 2 <= kTmemCols, "TMEM columns");
  // P = 2^(s - m + kPBias) and the running max moves when it rises by more
  // than kRescale (log2 units).  bf16 P has fp32's range: any bias works, a
  // wide threshold saves O rescales.  E4M3 P saturates at 448 < 2^9, so
  // p <= 2^(kPBias + kRescale) must stay <= 2^8; the bias lifts small
  // weights out of the subnormal range (normal E4M3 starts at 2^-6).
  static constexpr float kPBias = kFp8 ? 6.f : 0.f;
  static constexpr float kRescale = kFp8 ? 2.f : 8.f;
  // dynamic shared memory map (offsets from a 1024-byte aligned base): the
  // two Q tiles, the K/V ring (barriers are static shared memory)
  static constexpr int kOffQ = 0;
  static constexpr int kOffKV = 2 * kTileBytes;
  static constexpr int kSmemBytes = kOffKV + kStages * kTileBytes + 1024;  // + alignment slack
  static_assert(!kFp8 || D == kBN, "the FP8 V^T tile is D x 128 keys: D must be 128");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ bool warp_all(bool v) { return __all_sync(0xFFFFFFFFu, v); }

// Wait used only while tearing down after an abort: ignores the abort flag and
// gives up after a bounded number of polls (each poll suspends briefly), so
// copies and MMAs already in flight retire before the CTA exits.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  for (int spin = 0; spin < (1 << 20); ++spin)
    if (mbar_try_wait(bar, parity)) return;
}

// S = Q K^T over the head dimension into TMEM columns kColD, one MMA per 32
// bytes of a row (16 bf16 or 32 e4m3 columns); inside a 128-byte swizzle
// chunk a k-step advances the start address by 32 bytes, the next chunk
// starts 128 rows * 128 bytes further.  kOffB moves the K operand by whole
// rows: kKeyHalf selects keys [64, 128) of the tile (64 rows * 128 bytes,
// eight 1024-byte swizzle atoms).
constexpr uint32_t kKeyHalf = (64 * 128) >> 4;
// kColQ = 0: A (Q) from shared memory; otherwise A from TMEM columns
// kColQ.. (Q copied there once per unit, 8 columns per k-step).
template <bool kFp8, uint32_t kColD, uint32_t kOffA, uint32_t kColQ, uint32_t kOffB,
          uint32_t kIdesc, int KK, int NK>
__device__ __forceinline__ void issue_s_rec(uint32_t tmem, uint32_t a0, uint32_t b0) {
  if constexpr (KK < NK) {
    constexpr uint32_t off = ((KK >> 2) * (kBM * 128) + (KK & 3) * 32) >> 4;
    if constexpr (kColQ != 0)
      mma_ts<kFp8, kColD, kColQ + KK * 8, off + kOffB, kIdesc>(tmem, b0, KK > 0 ? 1u : 0u);
    else
      mma_ss<kFp8, kColD, off + kOffA, off + kOffB, kIdesc>(tmem, a0, b0, KK > 0 ? 1u : 0u);
    issue_s_rec<kFp8, kColD, kOffA, kColQ, kOffB, kIdesc, KK + 1, NK>(tmem, a0, b0);
  }
}
// N = 128 (all keys of the tile) or, with kHalf = 1 or 2, N = 64 over keys
// [0, 64) or [64, 128) into the same columns of S as the full product.  The
// A (Q) descriptor is a0 + kOffA (a constant, modulo 2^32, from the K ring's
// descriptor, so that no second descriptor register stays live), or, with
// kColQ != 0, Q is read from TMEM columns kColQ..
template <int D, bool kFp8, uint32_t kColS, uint32_t kOffA, int kHalf = 0, uint32_t kColQ = 0>
__device__ __forceinline__ void issue_s_steps(uint32_t tmem, uint32_t a0, uint32_t b0) {
  constexpr uint32_t kN = kHalf ? kBN / 2 : kBN;
  constexpr uint32_t kIdesc = kFp8 ? idesc_e4m3_f32(128, kN) : idesc_bf16_f32(128, kN, false);
  constexpr uint32_t kColD = kColS + (kHalf == 2 ? kBN / 2 : 0);
  constexpr uint32_t kOffB = kHalf == 2 ? kKeyHalf : 0;
  issue_s_rec<kFp8, kColD, kOffA, kColQ, kOffB, kIdesc, 0, D * (kFp8 ? 1 : 2) / 32>(tmem, a0,
                                                                                   b0);
}
// O (TMEM columns kColD) += P (TMEM columns kColP) V over the 128 keys of a
// tile, one MMA per 8 TMEM columns of P (16 bf16 or 32 e4m3 keys).  bf16: V
// is MN-major, a step advances 16 rows * 128 bytes.  e4m3: V^T (D rows of
// 128 keys) is K-major, a step advances 32 bytes inside the 128-byte row.
template <bool kFp8, uint32_t kColD, uint32_t kColP, uint32_t kOffB, uint32_t kIdesc, int KK>
__device__ __forceinline__ void issue_pv_rec(uint32_t tmem, uint32_t b0, uint32_t acc) {
  constexpr int kSteps = kFp8 ? kBN / 32 : kBN / 16;
  if constexpr (KK < kSteps) {
    constexpr uint32_t off = kFp8 ? ((KK * 32) >> 4) : ((KK * 16 * 128) >> 4);
    mma_ts<kFp8, kColD, kColP + KK * 8, off + kOffB, kIdesc>(tmem, b0, KK > 0 ? 1u : acc);
    issue_pv_rec<kFp8, kColD, kColP, kOffB, kIdesc, KK + 1>(tmem, b0, acc);
  }
}
template <int D, bool kFp8, uint32_t kColD, uint32_t kColP, uint32_t kOffB>
__device__ __forceinline__ void issue_pv_steps(uint32_t tmem, uint32_t b0, uint32_t acc) {
  constexpr uint32_t kIdesc = kFp8 ? idesc_e4m3_f32(128, D) : idesc_bf16_f32(128, D, true);
  issue_pv_rec<kFp8, kColD, kColP, kOffB, kIdesc, 0>(tmem, b0, acc);
}

}  // namespace
}  // namespace attn
