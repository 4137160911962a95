// C entries of the calls over a paged cache (attn_cache_write, attn_cache_read,
// attn_paged_fwd, attn_paged_decode): argument checks and launches.  The contracts
// are in include/attn.h.
#include <math.h>

#include <algorithm>
#include <initializer_list>

#include "../../include/attn.h"
#include "internal.h"

namespace attn {
namespace {

bool misaligned(const void* p, unsigned to) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1u)) != 0;
}

// Checks the arguments that describe a cache and its requests and fills *c.
int paged_arrays(const void* kpages, const void* vpages, const unsigned char* kscale,
                 const unsigned char* vscale, const int* table, const int* lens,
                 const int* offsets, int B, int T, int Hkv, int D, int page, int P, int M,
                 PagedArrays* c) {
  if (!kpages || !vpages || !table || !lens || !kscale != !vscale) return ATTN_ERR_NULL;
  if (B < 1 || B > 65536 || T < 0 || T > (1 << 24) || Hkv < 1 || Hkv > 65535 || P < 1 || M < 1)
    return ATTN_ERR_SHAPE;
  if (D != 64 && D != 128) return ATTN_ERR_SHAPE;
  if (page != 16 && page != 32 && page != 64 && page != 128) return ATTN_ERR_SHAPE;
  if (static_cast<long long>(P) * Hkv >= (1ll << 31) ||
      static_cast<long long>(M) * page > (1 << 21))
    return ATTN_ERR_SHAPE;
  for (const void* x : {kpages, vpages, static_cast<const void*>(kscale),
                        static_cast<const void*>(vscale)})
    if (misaligned(x, 16)) return ATTN_ERR_ALIGN;
  for (const int* x : {table, lens, offsets})
    if (misaligned(x, 4)) return ATTN_ERR_ALIGN;
  *c = PagedArrays{const_cast<void*>(kpages), const_cast<void*>(vpages),
                   const_cast<uint8_t*>(kscale), const_cast<uint8_t*>(vscale), table, lens, offsets,
                   B, T, Hkv, D, page, P, M, kscale != nullptr,
                   page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7};
  return ATTN_OK;
}

// A dense tensor's elements from one token to the next.
int check_stride(long long stride, int heads, int D) {
  return stride < static_cast<long long>(heads) * D || stride % 8 != 0 || stride > (1ll << 40)
             ? ATTN_ERR_SHAPE
             : ATTN_OK;
}

// Two sets of counts, in front of the partial states.
constexpr size_t kCountBytes = 2 * kPagedCounts * sizeof(uint32_t);

struct PagedLaunch {
  PagedParams* p;
  int rows, dev;  // rows: of a block of the kernel for few rows; 0: the one for many
  size_t states;  // rows of partial states
};
int launch_stream(void* ctx, void* scratch, unsigned turn, cudaStream_t stream) {
  const PagedLaunch& l = *static_cast<PagedLaunch*>(ctx);
  uint32_t* const counts = static_cast<uint32_t*>(scratch);
  l.p->part_o = reinterpret_cast<float*>(counts + 2 * kPagedCounts);
  l.p->part_ml = reinterpret_cast<float2*>(l.p->part_o + l.states * l.p->c.D);
  if (turn == 0 && cudaMemsetAsync(counts, 0, kCountBytes, stream) != cudaSuccess)
    return ATTN_ERR_CUDA;
  l.p->arrived = counts + (turn & 1) * kPagedCounts;
  l.p->clear = counts + (turn + 1 & 1) * kPagedCounts;
  return launch_paged_stream(*l.p, l.rows, l.dev, stream) == cudaSuccess ? ATTN_OK
                                                                         : ATTN_ERR_LAUNCH;
}
int launch_tile(void* ctx, void* scratch, cudaStream_t stream) {
  const PagedLaunch& l = *static_cast<PagedLaunch*>(ctx);
  l.p->part_o = static_cast<float*>(scratch);
  l.p->part_ml = reinterpret_cast<float2*>(l.p->part_o + l.states * l.p->c.D);
  l.p->cuts = reinterpret_cast<PagedCut*>(l.p->part_ml + l.states);
  return launch_paged_tile(*l.p, l.dev, stream) == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

int attend(const PagedArrays& c, const void* q, long long q_stride, void* o, float* lse, int Hq,
           int max_new, int causal, float scale, cudaStream_t stream) {
  if (!isfinite(scale) || scale < 0.f) return ATTN_ERR_SHAPE;
  if (Hq < 1 || Hq > 65535 || Hq % c.Hkv != 0 || Hq / c.Hkv > 128 || max_new < 0)
    return ATTN_ERR_SHAPE;
  if (int rc = check_stride(q_stride, Hq, c.D)) return rc;
  if (c.T == 0 || max_new == 0) return ATTN_OK;
  if (!q || !o || !lse) return ATTN_ERR_NULL;
  for (const void* x : {q, static_cast<const void*>(o), static_cast<const void*>(lse)})
    if (misaligned(x, 16)) return ATTN_ERR_ALIGN;
  PagedParams p = {};
  p.c = c;
  p.q = q;
  p.q_stride = q_stride;
  p.o = o;
  p.lse = lse;
  p.Hq = Hq;
  p.G = Hq / c.Hkv;
  p.causal = causal ? 1 : 0;
  // (never 0: an unseen score is -inf and has to stay it; 1e-37 times any product
  // below 1e30 is 0 next to a score's roundings)
  p.scale_log2 = std::max(scale * 1.4426950408889634f, 1e-37f);
  PagedLaunch l = {};
  l.p = &p;
  // Few rows share each key (up to 16): the kernel that streams the cache.  (For 17 to 32 it
  // reads it twice: 16 requests with 8 tokens of 32 heads on 8 behind 100 to 16384 75 us, the
  // other 52; e4m3 67 and 64; with 4 tokens 45 and 52.)  An accumulator of the one for many
  // rows takes kSegmentKeys keys at most, and lengths are on the device: so does a wider
  // table, at the price of reading the cache for every 16 rows (2048 tokens behind 16001,
  // 32 heads on 8, D 128: 5.0 ms for 0.36; e4m3, 1024 behind 30000, 3.1 for 0.41; a
  // prompt of 500 87 us for 32).
  const long long rows = std::min<long long>(max_new, c.T) * p.G;
  const bool many = rows > 16 && static_cast<long long>(c.M) * c.page <= kSegmentKeys;
  l.rows = many ? 0 : rows <= 8 ? 8 : 16;
  // the streaming kernel numbers its units of work in 32 bits: a block of rows has
  // M * page / 64 + 9 of them at most, less than twice what is counted here
  // (the other one counts in 64 bits)
  const long long blocks = static_cast<long long>(c.T) * p.G / 8 + c.B;
  if (!many &&
      blocks * c.Hkv * (static_cast<long long>(c.M) * c.page / 64 + 5) >= (1ll << 31))
    return ATTN_ERR_SHAPE;
  DeviceInfo di;
  if (int rc = device_info(&di)) return rc;
  const int box = many ? c.page : paged_stream_box(c);
  if (!many || !c.quant) {
    if (int rc = encode_pages(&p.tmap_k, c.kpages, c, box, !many)) return rc;
    if (int rc = encode_pages(&p.tmap_v, c.vpages, c, box, !many)) return rc;
  }
  if (many)
    if (int rc = encode_queries(&p.tmap_q, q, c.D, p.G, c.Hkv, c.T, 128 / p.G, q_stride)) return rc;
  p.ctas = std::min(static_cast<unsigned>(di.sms), kMostCtas);
  if (!many) p.ctas *= paged_stream_ctas(p, l.rows);
  p.err = di.err_word;
  p.wait_limit_ns = wait_limit_ns();
  l.dev = di.dev;
  l.states = many ? paged_tile_state(p) : paged_stream_state(p, l.rows);
  const size_t bytes = l.states * (c.D * sizeof(float) + sizeof(float2));
  return many ? with_scratch(bytes + p.ctas * sizeof(PagedCut), di.dev, stream, launch_tile, &l)
              : with_turns(bytes + kCountBytes, di.dev, stream, launch_stream, &l);
}

int cache_rows(const PagedArrays& c, CacheRows r, bool read, cudaStream_t stream) {
  if (int rc = check_stride(r.k_stride, c.Hkv, c.D)) return rc;
  if (int rc = check_stride(r.v_stride, c.Hkv, c.D)) return rc;
  if (c.T == 0) return ATTN_OK;
  const void* k = read ? r.k_out : r.k;
  const void* v = read ? r.v_out : r.v;
  if (!k || !v) return ATTN_ERR_NULL;
  if (misaligned(k, 16) || misaligned(v, 16)) return ATTN_ERR_ALIGN;
  DeviceInfo di;
  if (int rc = device_info(&di)) return rc;
  r.err = di.err_word;
  return launch_cache_rows(c, r, read, stream) == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

int attn_cache_write(const void* k, const void* v, long long k_stride, long long v_stride,
                     void* kpages, void* vpages, unsigned char* kscale, unsigned char* vscale,
                     const int* table, const int* lens, const int* offsets, int B, int T, int Hkv,
                     int D, int page, int P, int M, cudaStream_t stream) {
  PagedArrays c;
  if (int rc = paged_arrays(kpages, vpages, kscale, vscale, table, lens, offsets, B, T, Hkv, D,
                            page, P, M, &c))
    return rc;
  return cache_rows(c, CacheRows{k, v, nullptr, nullptr, k_stride, v_stride, nullptr}, false,
                    stream);
}

int attn_cache_read(const void* kpages, const void* vpages, const unsigned char* kscale,
                    const unsigned char* vscale, const int* table, const int* lens,
                    const int* offsets, void* k, void* v, int B, int T, int Hkv, int D, int page,
                    int P, int M, cudaStream_t stream) {
  PagedArrays c;
  if (int rc = paged_arrays(kpages, vpages, kscale, vscale, table, lens, offsets, B, T, Hkv, D,
                            page, P, M, &c))
    return rc;
  const long long stride = static_cast<long long>(Hkv) * D;
  return cache_rows(c, CacheRows{nullptr, nullptr, k, v, stride, stride, nullptr}, true, stream);
}

int attn_paged_fwd(const void* q, long long q_stride, const void* kpages, const void* vpages,
                   const unsigned char* kscale, const unsigned char* vscale, const int* table,
                   const int* lens, const int* offsets, void* o, float* lse, int B, int T,
                   int max_new, int Hq, int Hkv, int D, int page, int P, int M, int causal,
                   float scale, cudaStream_t stream) {
  if (!offsets) return ATTN_ERR_NULL;
  PagedArrays c;
  if (int rc = paged_arrays(kpages, vpages, kscale, vscale, table, lens, offsets, B, T, Hkv, D,
                            page, P, M, &c))
    return rc;
  return attend(c, q, q_stride, o, lse, Hq, max_new, causal, scale, stream);
}

int attn_paged_decode(const void* q, long long q_stride, const void* kpages, const void* vpages,
                      const unsigned char* kscale, const unsigned char* vscale, const int* table,
                      const int* lens, void* o, float* lse, int B, int Hq, int Hkv, int D,
                      int page, int P, int M, float scale, cudaStream_t stream) {
  PagedArrays c;
  if (int rc = paged_arrays(kpages, vpages, kscale, vscale, table, lens, nullptr, B, B, Hkv, D,
                            page, P, M, &c))
    return rc;
  return attend(c, q, q_stride, o, lse, Hq, 1, 0, scale, stream);
}

}  // extern "C"
