// Attention with modified scores, the plain way: one warp per query row walks
// the row's keys with a running maximum and sum, a lane holding D / 32
// elements of every vector.  Right for every case; nothing is shared between
// the rows that read the same keys.
#include <cuda_bf16.h>
#include <math.h>

#include "../../include/attn.h"
#include "score_mod.cuh"

namespace attn {
namespace {

template <int E>
struct RowState {
  float m, l, o[E];
};

template <int E>
__device__ __forceinline__ void load_row(const __nv_bfloat16* row, int lane, float (&x)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = __bfloat162float(row[lane * E + i]);
}

// st += other (both unnormalised, each relative to its own maximum).
template <int E>
__device__ void merge(RowState<E>& st, const RowState<E>& other) {
  const float m = fmaxf(st.m, other.m);
  if (m == -INFINITY) return;
  const float a = ex2_approx(st.m - m), b = ex2_approx(other.m - m);
  st.m = m;
  st.l = st.l * a + other.l * b;
#pragma unroll
  for (int i = 0; i < E; ++i) st.o[i] = st.o[i] * a + other.o[i] * b;
}

// Keys [lo, hi) of k / v rows, the first of them at position pos_base + lo.
// 64 keys are summed at a time, so that a sum over n keys is a chain of about
// n / 64 additions (each can lose half a digit of the whole).
template <int E>
__device__ void attend(RowState<E>& all, const float (&q)[E], const __nv_bfloat16* k,
                       const __nv_bfloat16* v, int lo, int hi, int pos_base, int pos,
                       const ScoreMod& mod, float slope, int ref, int lane) {
  constexpr int D = E * 32;
  for (int j0 = lo; j0 < hi; j0 += 64) {
    RowState<E> st = {-INFINITY, 0.f, {}};
    const int j1 = min(j0 + 64, hi);
    for (int j = j0; j < j1; ++j) {
      float x[E], s = 0.f;
      load_row<E>(k + static_cast<size_t>(j) * D, lane, x);
#pragma unroll
      for (int i = 0; i < E; ++i) s = fmaf(q[i], x[i], s);
#pragma unroll
      for (int d = 16; d >= 1; d /= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
      s = mod_score(mod, s);
      if (slope != 0.f)
        s -= slope * kLog2e * static_cast<float>(abs(pos - (pos_base + j)) - ref);
      const float m = fmaxf(st.m, s);
      if (m == -INFINITY) continue;  // a product that overflowed: weight 0
      const float old = ex2_approx(st.m - m), w = ex2_approx(s - m);
      load_row<E>(v + static_cast<size_t>(j) * D, lane, x);
      st.m = m;
      st.l = fmaf(st.l, old, w);
#pragma unroll
      for (int i = 0; i < E; ++i) st.o[i] = fmaf(st.o[i], old, w * x[i]);
    }
    merge<E>(all, st);
  }
}

template <int E>
__device__ void store_row(const RowState<E>& st, float slope, int ref, __nv_bfloat16* o,
                          float* lse, int lane) {
  const bool none = st.l == 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i)
    o[lane * E + i] = __float2bfloat16_rn(none ? 0.f : st.o[i] / st.l);
  if (lane == 0)
    *lse = none ? -INFINITY
                : (st.m + __log2f(st.l)) * kLn2 - slope * static_cast<float>(ref);
}

template <int E>
__global__ void __launch_bounds__(128) simple_fwd_kernel(const ModFwdParams p) {
  constexpr int D = E * 32;
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(p.B) * p.Hq * p.Nq) return;
  const int i = static_cast<int>(row % p.Nq);
  const int bh = static_cast<int>(row / p.Nq), b = bh / p.Hq, h = bh % p.Hq;
  const int pos = p.q_offset + i;
  int lo = 0, hi = p.Nk;
  if (p.ranges) {
    const int2 r = reinterpret_cast<const int2*>(p.ranges)[static_cast<size_t>(b) * p.Nq + i];
    lo = max(r.x, 0);
    hi = min(r.y, p.Nk);
  }
  if (p.causal) hi = min(hi, pos + 1);
  const size_t kv = (static_cast<size_t>(b) * p.Hkv + h / (p.Hq / p.Hkv)) * p.Nk * D;
  const float slope = p.mod.slopes ? p.mod.slopes[h] : 0.f;
  const int ref = lo < hi ? bias_ref(slope, pos, lo, hi) : 0;
  float q[E];
  load_row<E>(static_cast<const __nv_bfloat16*>(p.q) + row * D, lane, q);
  RowState<E> st = {-INFINITY, 0.f, {}};
  attend<E>(st, q, static_cast<const __nv_bfloat16*>(p.k) + kv,
            static_cast<const __nv_bfloat16*>(p.v) + kv, lo, hi, 0, pos, p.mod, slope, ref, lane);
  store_row<E>(st, slope, ref, static_cast<__nv_bfloat16*>(p.o) + row * D, p.lse + row, lane);
}

template <int E>
__global__ void __launch_bounds__(128) simple_decode_kernel(const ModDecodeParams p) {
  constexpr int D = E * 32;
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(p.B) * p.Hq) return;
  const int b = static_cast<int>(row / p.Hq), h = static_cast<int>(row % p.Hq);
  const int hkv = h / (p.Hq / p.Hkv);
  const int len = p.lens ? min(max(p.lens[b], 0), p.Ncap) : p.Ncap;
  const int pos = p.Np + len - 1;
  const float slope = p.mod.slopes ? p.mod.slopes[h] : 0.f;
  const int ref = pos >= 0 ? bias_ref(slope, pos, 0, pos + 1) : 0;
  float q[E];
  load_row<E>(static_cast<const __nv_bfloat16*>(p.q) + row * D, lane, q);
  RowState<E> st = {-INFINITY, 0.f, {}};
  const size_t pre = static_cast<size_t>(hkv) * p.Np * D;
  attend<E>(st, q, static_cast<const __nv_bfloat16*>(p.kprefix) + pre,
            static_cast<const __nv_bfloat16*>(p.vprefix) + pre, 0, p.Np, 0, pos, p.mod, slope, ref,
            lane);
  const size_t kv = (static_cast<size_t>(b) * p.Hkv + hkv) * p.Ncap * D;
  attend<E>(st, q, static_cast<const __nv_bfloat16*>(p.kcache) + kv,
            static_cast<const __nv_bfloat16*>(p.vcache) + kv, 0, len, p.Np, pos, p.mod, slope, ref,
            lane);
  store_row<E>(st, slope, ref, static_cast<__nv_bfloat16*>(p.o) + row * D, p.lse + row, lane);
}

}  // namespace

int mod_fwd(const ModFwdParams& p, cudaStream_t stream) {
  if (int rc = check_device()) return rc;
  const long long rows = static_cast<long long>(p.B) * p.Hq * p.Nq;
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  if (p.D == 128)
    simple_fwd_kernel<4><<<grid, 128, 0, stream>>>(p);
  else
    simple_fwd_kernel<2><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

int mod_decode(const ModDecodeParams& p, cudaStream_t stream) {
  if (int rc = check_device()) return rc;
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(p.B) * p.Hq + 3) / 4);
  if (p.D == 128)
    simple_decode_kernel<4><<<grid, 128, 0, stream>>>(p);
  else
    simple_decode_kernel<2><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

}  // namespace attn
