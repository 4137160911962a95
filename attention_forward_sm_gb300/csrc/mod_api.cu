// C entries of the attention calls with modified scores (attn_fwd_mod,
// attn_decode_varlen, attn_decode_prefix): argument checks and launches.  The
// contracts are in include/attn.h.
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/attn.h"
#include "internal.h"

namespace attn {
namespace {

bool misaligned(const void* p, unsigned to) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1u)) != 0;
}

// tanh(x) = x T(x^2): interpolations of tanh(x) / x in the Chebyshev points of
// x^2 on [0, X^2].  The nearest singularity is at x^2 = -pi^2 / 4, so a further
// coefficient gains a factor of 159 at X = 1/4, 41 at 1/2, 12 at 1; each of
// these is off by 6.1e-7 of the value at most, a few roundings of the score.
// With x = cap_in * s the powers of cap_in go into the coefficients.
void cap_polynomials(ScoreMod* m) {
  static const double x_most[3] = {0.25, 0.5, 1.0};
  static const int n[3] = {kCapN0, kCapN1, kCapN2};
  static const double c[3][6] = {
      {0x1.fffff2p-1, -0x1.55375ap-2, 0x1.06fe18p-3},
      {0x1.ffffeep-1, -0x1.5542dap-2, 0x1.0e2146p-3, -0x1.6baa52p-5},
      {0x1.ffffecp-1, -0x1.5549d8p-2, 0x1.0ffd3ap-3, -0x1.a697a8p-5, 0x1.11f45ap-6,
       -0x1.90d924p-9}};
  constexpr double kOff = 64.0;
  const double in = m->cap_in, out = m->cap_out;
  for (int i = 0; i < 3; ++i) {
    bool fits = in > 0.0;
    double power = in * out;
    for (int k = 0; k < n[i]; ++k, power *= in * in) {
      const double x = c[i][k] * power;
      m->cap_coef[i][k] = static_cast<float>(x);
      fits = fits && fabs(x) < 1e37 && fabs(x) > 1e-37;
    }
    // what is formed on the way has to fit too, up to the limit and at cap_off
    const double limit = x_most[i] / in;
    for (const double s : {limit, kOff / in}) {
      double t = 0.0;
      for (int k = n[i] - 1; fits && k >= 0; --k) {
        t = t * (s * s) + m->cap_coef[i][k];
        fits = fabs(t) < 1e37;
      }
      fits = fits && s * s < 1e37 && fabs(s * t) < 1e37;
      if (i > 0 && s != limit) fits = fits && s * t < -1e6 - 2.0 * out;
    }
    m->cap_limit[i] = fits ? static_cast<float>(limit) : -1.f;
  }
  m->cap_off = in > 0.0 ? static_cast<float>(kOff / in) : 0.f;
}

// Checks scale, softcap and slopes and fills *m.
int score_mod(float scale, float softcap, const float* slopes, ScoreMod* m) {
  if (!isfinite(scale) || scale < 0.f) return ATTN_ERR_SHAPE;
  if (!isfinite(softcap) || softcap < 0.f) return ATTN_ERR_SHAPE;
  *m = ScoreMod{};
  m->scale = scale;
  if (softcap > 0.f) {
    m->cap_in = scale / softcap;
    m->cap_out = softcap * 1.4426950408889634f;
    if (!isfinite(m->cap_in) || !isfinite(m->cap_out)) return ATTN_ERR_SHAPE;
    cap_polynomials(m);
  }
  if (misaligned(slopes, 4)) return ATTN_ERR_ALIGN;
  m->slopes = slopes;
  return ATTN_OK;
}

int decode_entry(const void* q, const void* kprefix, const void* vprefix, const void* kcache,
                 const void* vcache, const int* lens, void* o, float* lse, int B, int Hq, int Hkv,
                 int Np, int Ncap, int D, float scale, float softcap, const float* slopes,
                 cudaStream_t stream) {
  if (!q || !kcache || !vcache || !o || !lse) return ATTN_ERR_NULL;
  constexpr int kMostKeys = 1 << 30;
  if (B < 1 || Hq < 1 || Hkv < 1 || Ncap < 1 || Ncap > kMostKeys || Np < 0 || Np > kMostKeys)
    return ATTN_ERR_SHAPE;
  if (Hq % Hkv != 0 || Hq / Hkv > 128 || Hq > 65535) return ATTN_ERR_SHAPE;
  if (D != 64 && D != 128) return ATTN_ERR_SHAPE;
  if (static_cast<long long>(B) * Hkv > (1ll << 20)) return ATTN_ERR_SHAPE;
  // key tiles are numbered in 32 bits: of the caches, and of the prefix times the
  // blocks of two times 128 / G requests that share it
  const long long blocks = (B + 2ll * (128 / (Hq / Hkv)) - 1) / (2 * (128 / (Hq / Hkv)));
  if (static_cast<long long>(B) * Hkv * ((Ncap + 127ll) / 128) > kMostTiles ||
      Hkv * blocks * ((Np + 127ll) / 128) > kMostTiles)
    return ATTN_ERR_SHAPE;
  ModDecodeParams p = {};
  if (int rc = score_mod(scale, softcap, slopes, &p.mod)) return rc;
  for (const void* x : {q, kprefix, vprefix, kcache, vcache, static_cast<const void*>(o),
                        static_cast<const void*>(lse)})
    if (misaligned(x, 16)) return ATTN_ERR_ALIGN;
  if (misaligned(lens, 4)) return ATTN_ERR_ALIGN;
  p.q = q;
  p.kprefix = kprefix;
  p.vprefix = vprefix;
  p.kcache = kcache;
  p.vcache = vcache;
  p.lens = lens;
  p.o = o;
  p.lse = lse;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Np = Np;
  p.Ncap = Ncap;
  p.D = D;
  return mod_decode(p, stream);
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

int attn_fwd_mod(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
                 int Hkv, int Nq, int Nk, int D, int causal, int q_offset, float scale,
                 float softcap, const float* slopes, const int* ranges, cudaStream_t stream) {
  if (!q || !k || !v || !o || !lse) return ATTN_ERR_NULL;
  if (B < 1 || Hq < 1 || Hkv < 1 || Nq < 1 || Nk < 1 || Hq % Hkv != 0) return ATTN_ERR_SHAPE;
  if (D != 64 && D != 128) return ATTN_ERR_SHAPE;
  // the kernels form q_offset + (row within the call) + a few tiles in int
  if (q_offset < 0 || q_offset > INT_MAX - Nq - 1024 || Nk > INT_MAX - 1024) return ATTN_ERR_SHAPE;
  if (static_cast<long long>(B) * Hq * ((Nq + 255ll) / 256) >= (1ll << 31) - 65536)
    return ATTN_ERR_SHAPE;
  ModFwdParams p = {};
  if (int rc = score_mod(scale, softcap, slopes, &p.mod)) return rc;
  for (const void* x : {q, k, v, static_cast<const void*>(o), static_cast<const void*>(lse)})
    if (misaligned(x, 16)) return ATTN_ERR_ALIGN;
  if (misaligned(ranges, 8)) return ATTN_ERR_ALIGN;
  p.q = q;
  p.k = k;
  p.v = v;
  p.o = o;
  p.lse = lse;
  p.ranges = ranges;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Nq = Nq;
  p.Nk = Nk;
  p.D = D;
  p.causal = causal ? 1 : 0;
  p.q_offset = q_offset;
  return mod_fwd(p, stream);
}

int attn_decode_varlen(const void* q, const void* kcache, const void* vcache, const int* lens,
                       void* o, float* lse, int B, int Hq, int Hkv, int Ncap, int D, float scale,
                       float softcap, const float* slopes, cudaStream_t stream) {
  return decode_entry(q, nullptr, nullptr, kcache, vcache, lens, o, lse, B, Hq, Hkv, 0, Ncap, D,
                      scale, softcap, slopes, stream);
}

int attn_decode_prefix(const void* q, const void* kprefix, const void* vprefix,
                       const void* kcache, const void* vcache, const int* lens, void* o,
                       float* lse, int B, int Hq, int Hkv, int Np, int Ncap, int D, float scale,
                       float softcap, const float* slopes, cudaStream_t stream) {
  if (!kprefix || !vprefix) return ATTN_ERR_NULL;
  if (Np < 1) return ATTN_ERR_SHAPE;
  return decode_entry(q, kprefix, vprefix, kcache, vcache, lens, o, lse, B, Hq, Hkv, Np, Ncap, D,
                      scale, softcap, slopes, stream);
}

}  // extern "C"
