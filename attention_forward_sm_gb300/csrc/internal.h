// Host-side interface between the C ABI (api.cu) and the kernel translation
// units (fwd_sm103a.cu, decode_sm103a.cu).  Not part of the public header.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace attn {

// Bits of the device error word (also listed in include/attn.h).
enum : unsigned int {
  kErrWaitLoad = 1u << 0,     // loader gave up waiting for a free K/V slot
  kErrWaitMma = 1u << 1,      // MMA issuer gave up waiting for data / P / correction
  kErrWaitSoftmax = 1u << 2,  // softmax gave up waiting for S
  kErrWaitCorr = 1u << 3,     // correction / epilogue gave up waiting
  kErrSelfTest = 1u << 4,     // the wait self-test ran out, as intended
  kErrLens = 1u << 5,         // a decode's lengths changed while it was planned
  kErrPage = 1u << 6,         // a page number out of range
};

// Forward (prefill) launch parameters.  Tensor maps are 3-D views with a
// 128-byte swizzle: bf16 [B*H, N, D] with box {64, 128, 1}; for FP8, e4m3
// Q and K [B*H, N, D] with box {128, 128, 1} and V^T [B*Hkv, D, Nk] with box
// {128 keys, 128 rows, 1}.
struct FwdParams {
  CUtensorMap tmap_q, tmap_k, tmap_v;
  void* o;             // [B, Hq, Nq, D] bf16
  float* lse;          // [B, Hq, Nq] fp32
  int B, Hq, Hkv, Nq, Nk, D;
  int causal;
  int q_offset;        // causal: row i of this call is row q_offset + i of the problem
  int fp8;             // e4m3 Q, K, V^T
  int group_heads;     // causal unit order: query heads per group (a multiple of Hq/Hkv)
  float scale_log2;    // scale * log2(e) (FP8: times q_scale * k_scale)
  float o_scale;       // O multiplier (FP8: v_scale; bf16: 1)
  unsigned int* err;   // device error word
  uint64_t wait_limit_ns;
};

// Split-KV decode launch parameters.
struct DecodeParams {
  const void* q;       // [B, Hq, D] bf16
  const void* k;       // [B, Hkv, Nk, D] bf16
  const void* v;       // [B, Hkv, Nk, D] bf16
  void* o;             // [B, Hq, D] bf16 (unless o_state is set)
  float* o_state;      // optional [B, Hq, D] fp32 output instead of o
  float* lse;          // [B, Hq] fp32
  float* ws_o;         // [B, Hq, nsplit, D] fp32 partial outputs (normalised per chunk)
  float* ws_lse;       // [B, Hq, nsplit] fp32 partial lse (natural log)
  int B, Hq, Hkv, Nk, D, nsplit;
  float scale_log2;
  unsigned int* err;   // device error word
  uint64_t wait_limit_ns;
};

// Score modifications (see include/attn.h).  x = scale * <q, k>; capped:
// tanh(x / softcap) * softcap = tanh(cap_in * <q, k>) * cap_out in log2 units.
struct ScoreMod {
  float scale;
  float cap_in;         // scale / softcap; 0: no cap
  float cap_out;        // softcap * log2(e)
  const float* slopes;  // [Hq], or NULL: no distance bias
  // s T(s^2) = the capped score for a raw product |s| <= cap_limit[i] (ascending;
  // -1: not usable), T of kCapN<i> coefficients.  At s = cap_off the last two, whose
  // leading coefficients are negative, are below any score by more than 10^6.
  float cap_off;
  float cap_limit[3];
  float cap_coef[3][6];
};
constexpr int kCapN0 = 3, kCapN1 = 4, kCapN2 = 6;

// Keys that one accumulator in tensor memory takes at most.  The tensor cores cut
// products to 26 bits below the accumulator's highest: n equal terms are 2^-27 n of
// their sum short, 2^-9 (half a step of bf16) for 2^18.
constexpr int kSegmentKeys = 1 << 18;

// Prefill with modified scores.
struct ModFwdParams {
  const void* q;      // [B, Hq, Nq, D] bf16
  const void* k;      // [B, Hkv, Nk, D] bf16
  const void* v;
  void* o;            // [B, Hq, Nq, D] bf16
  float* lse;         // [B, Hq, Nq]
  const int* ranges;  // [B, Nq, 2] visible keys [lo, hi) of every row, or NULL: all
  int B, Hq, Hkv, Nq, Nk, D;
  int causal, q_offset;
  ScoreMod mod;
};

// Decode with a length per request, behind a shared prefix if Np > 0.
struct ModDecodeParams {
  const void* q;        // [B, Hq, D] bf16
  const void* kprefix;  // [Hkv, Np, D] bf16
  const void* vprefix;
  const void* kcache;   // [B, Hkv, Ncap, D] bf16
  const void* vcache;
  const int* lens;      // [B], or NULL: Ncap each
  void* o;              // [B, Hq, D] bf16
  float* lse;           // [B, Hq]
  int B, Hq, Hkv, Np, Ncap, D;
  ScoreMod mod;
};

// Launch parameters of mod_attn_kernel (mod_sm103a.cuh), prefill and decode.
struct ModKernelParams {
  // K and V: [BH, N, D], box {64, 128, 1}.  Q: prefill the same; decode
  // [B, Hkv, G, D] with box {64, G, 1, per_tile} (tmap_q) or {64, G, 1, 1}
  // (tmap_q1).  128-byte swizzle.
  // Prefix: tmap_kp, tmap_vp; a decode's caches have boxes {64, 32, 1}.
  CUtensorMap tmap_q, tmap_q1, tmap_k, tmap_v, tmap_kp, tmap_vp;
  void* o;
  float* lse;
  const int* ranges;
  const int* lens;
  int B, Hq, Hkv, G, Nq, Nk;  // Nk: keys (prefill) or the caches' capacity (decode)
  int causal, q_offset;  // (q_offset: relative to the first key here, may be negative)
  int key0;              // prefill: keys in front of the first one here
  int longest_first, group_heads;  // prefill: order of the work items
  int o_sectors;                   // prefill: o is 32-byte aligned (stores of whole
                                   // sectors: packed documents 77 us, else 83)
  int Np, prefix_tiles;            // shared prefix: keys, key tiles
  int row_blocks, per_tile;        // its items per KV head; requests per query tile
  int pre_rows;                    // rows of a prefix item's partial states
  float prefix_cost, own_cost;     // what a key tile of either costs a CTA
  float* pre_o;                    // partial states of prefix items: [slot, pre_rows, D]
  float* pre_lse;                  // (log2 units, bias relative to its reference)
  float* part_o;                   // of the requests' own keys: [slot, G, D]
  float* part_lse;
  uint32_t* plan;                  // [B + 2] own-key tiles in front of every request, of
                                   // all; the CTAs that have own keys alone
  float scale_log2;
  ScoreMod mod;
  unsigned int* err;
  uint64_t wait_limit_ns;
};

// Tiles of all shared prefix items.
__host__ __device__ inline uint32_t prefix_total(const ModKernelParams& p) {
  return static_cast<uint32_t>(p.Hkv) * p.row_blocks * p.prefix_tiles;
}
// `total` tiles dealt out in `runs` <= total runs, as equal as they can be:
// the first tile of run r, and the run that holds tile x.  Totals are at most
// kMostTiles, so that the products fit 32 bits (a 64-bit division takes a warp
// hundreds of cycles, and the planning of a short decode is most of it).
constexpr uint32_t kMostTiles = 12000000, kMostCtas = 178;
static_assert(2ull * kMostCtas * kMostTiles < (1ull << 32), "32-bit products");
__host__ __device__ inline uint32_t run_start(uint32_t total, uint32_t runs, uint32_t r) {
  return r * total / runs;
}
__host__ __device__ inline uint32_t run_of(uint32_t total, uint32_t runs, uint32_t x) {
  return ((x + 1) * runs - 1) / total;
}
// Of `ctas` CTAs, how many have own keys alone, the others then being left to the
// shared prefix; 0: all have both, one after the other.  Apart, the products of the
// one run beside the loads of the other, and no CTA goes from one to the other.
// Either kind needs a tile for each CTA at least, and a share of eight CTAs, that the
// rounding of the shares does not cost more.
__host__ __device__ inline uint32_t own_share(uint32_t ctas, uint32_t prefix, uint32_t own,
                                              float prefix_cost, float own_cost) {
  if (prefix < ctas || own < ctas) return 0;
  const float o = own_cost * static_cast<float>(own);
  const float share = o / (o + prefix_cost * static_cast<float>(prefix));
  const uint32_t n = static_cast<uint32_t>(static_cast<float>(ctas) * share + 0.5f);
  return n < 8 || n + 8 > ctas ? 0 : n;
}
// Runs of more than kSegmentKeys keys are cut into pieces, equally many per run; an
// item's part in each has a partial state of its own.
constexpr uint32_t kPieceTiles = kSegmentKeys / 128;
struct Pieces {
  uint32_t per_run = 1, tiles = 0xFFFFFFFFu;  // tiles of one
  __host__ __device__ Pieces(uint32_t total, uint32_t runs) {
    if (total <= runs * kPieceTiles) return;
    const uint32_t most = (total + runs - 1) / runs;
    per_run = (most + kPieceTiles - 1) / kPieceTiles;
    tiles = (most + per_run - 1) / per_run;
  }
  // the piece that holds tile `at` of run r
  __host__ __device__ uint32_t of(uint32_t r, uint32_t at) const {
    return per_run == 1 ? r : r * per_run + at / tiles;
  }
};
// The piece that holds tile x.
__host__ __device__ inline uint32_t piece_of(uint32_t total, uint32_t runs, const Pieces& pieces,
                                             uint32_t x) {
  const uint32_t r = run_of(total, runs, x);
  return pieces.per_run == 1 ? r : pieces.of(r, x - run_start(total, runs, r));
}

// One launch each, by head size and modifications.
// (`dev`: the current device.)
cudaError_t launch_mod_fwd_d64(const ModKernelParams& p, unsigned grid, int dev,
                               cudaStream_t stream);
cudaError_t launch_mod_fwd_d128(const ModKernelParams& p, unsigned grid, int dev,
                               cudaStream_t stream);
cudaError_t launch_mod_split_d64_h0(const ModKernelParams& p, unsigned grid, int dev,
                               cudaStream_t stream);
cudaError_t launch_mod_split_d64_h4(const ModKernelParams& p, unsigned grid, int dev,
                               cudaStream_t stream);
cudaError_t launch_mod_split_d64_h8(const ModKernelParams& p, unsigned grid, int dev,
                               cudaStream_t stream);
cudaError_t launch_mod_split_d128_h0(const ModKernelParams& p, unsigned grid, int dev,
                               cudaStream_t stream);
cudaError_t launch_mod_split_d128_h4(const ModKernelParams& p, unsigned grid, int dev,
                               cudaStream_t stream);
cudaError_t launch_mod_split_d128_h8(const ModKernelParams& p, unsigned grid, int dev,
                               cudaStream_t stream);

// 3-D bf16 view [BH, N, D], box {64, rows, 1}; 4-D view [B, Hkv, G, D] of the
// queries of a decode, box {64, G, 1, requests}.  Return an ATTN_* status.
int encode_rows(CUtensorMap* map, const void* base, int D, int N, long long BH, int rows,
                int stride = 0);  // rows from one [N, D] to the next; 0: N
int encode_queries(CUtensorMap* map, const void* base, int D, int G, int Hkv, int B, int requests,
                   long long stride = 0);  // elements from one to the next; 0: G Hkv D

// Device scratch of `bytes` for the kernels that launch(ctx, scratch, stream)
// queues on `stream`: the stream's cached buffer or, during capture, one of the
// graph's own.  Returns launch's status or an ATTN_ERR_*.
// `dev`: the current device.
int with_scratch(size_t bytes, int dev, cudaStream_t stream,
                 int (*launch)(void* ctx, void* scratch, cudaStream_t stream), void* ctx);
// The same with a buffer that is allocated for the call alone.
int with_own_scratch(size_t bytes, cudaStream_t stream, int (*launch)(void*, void*, cudaStream_t),
                     void* ctx);

// As with_scratch, for kernels that keep something in the buffer from one call to the
// next: turn counts the calls that have used it, 0 where its contents are unknown (a new
// buffer, one after a failed call, every captured call).
int with_turns(size_t bytes, int dev, cudaStream_t stream,
               int (*launch)(void* ctx, void* scratch, unsigned turn, cudaStream_t stream),
               void* ctx);

// Check the device and queue the kernels; arguments are checked before.
// Return an ATTN_* status.
int mod_fwd(const ModFwdParams& p, cudaStream_t stream);
int mod_decode(const ModDecodeParams& p, cudaStream_t stream);

// A paged cache (see paged.cuh).
struct PagedArrays {
  void* kpages;        // [P, Hkv, page, D] bf16, or e4m3 codes (quant)
  void* vpages;
  uint8_t* kscale;     // [P, Hkv, page] scale bytes (quant), else NULL
  uint8_t* vscale;
  const int* table;    // [B, M] page numbers
  const int* lens;     // [B] tokens in the cache, the new ones among them
  const int* offsets;  // [B + 1] rows of the new tokens; NULL: row b is request b's one
  int B, T, Hkv, D, page, P, M;  // T: rows of the dense tensors
  int quant;
  int page_bits;  // page = 1 << page_bits: the loading warps have no time for divisions
};
// Dense rows that go into the cache (k, v) or come out of it (k_out, v_out, [T, Hkv, D]).
struct CacheRows {
  const void* k;
  const void* v;
  void* k_out;
  void* v_out;
  long long k_stride, v_stride;  // elements from one token to the next
  unsigned int* err;
};
cudaError_t launch_cache_rows(const PagedArrays& c, const CacheRows& r, bool read,
                              cudaStream_t stream);

// An item of the kernel for many rows that was cut, written by the CTA that has its first
// part: the parts are that CTA's state 1 and state 0 of the `parts` - 1 CTAs behind it.
struct PagedCut {
  int parts;       // 0: none begins in this CTA
  int row0, left;  // first dense row; tokens of the request from there on
  int h;           // KV head
};

// Attention of new tokens over a paged cache.
constexpr uint32_t kPagedCounts = 16 * 2 * kMostCtas;
struct PagedParams {
  CUtensorMap tmap_k, tmap_v;  // pages as [P * Hkv, pieces, page, 128 bytes]
  CUtensorMap tmap_q;          // [T, Hkv, G, D], box {64, G, 1, 128 / G} (many rows)
  PagedArrays c;
  const void* q;       // [T, Hq, D] bf16, q_stride elements from one token to the next
  long long q_stride;
  void* o;             // [T, Hq, D] bf16
  float* lse;          // [T, Hq]
  int Hq, G, causal;
  float scale_log2;
  unsigned ctas;       // of the split kernel
  float* part_o;       // partial states: [slot, rows of a block, D], and their
  float2* part_ml;     // maximum (log2 units) and sum
  PagedCut* cuts;      // of every CTA (many rows)
  // Few rows: for each CTA that has an item's first part, and 16 shares of its rows: how many of
  // the parts' CTAs have stored theirs.  Two sets that calls use in turn, each call
  // clearing the other one, so that a call that failed leaves nothing behind.
  uint32_t* arrived;   // [kPagedCounts]
  uint32_t* clear;
  unsigned int* err;
  uint64_t wait_limit_ns;
};
// The kernel for few rows, and what its scratch takes.
int paged_stream_box(const PagedArrays& c);                 // rows of a page per copy
unsigned paged_stream_ctas(const PagedParams& p, int rows);  // per SM
size_t paged_stream_state(const PagedParams& p, int rows);  // rows of partial states
cudaError_t launch_paged_stream(const PagedParams& p, int rows, int dev, cudaStream_t stream);
// The kernel for many rows, likewise.
size_t paged_tile_state(const PagedParams& p);
cudaError_t launch_paged_tile(const PagedParams& p, int dev, cudaStream_t stream);
// Tensor map over pages; a copy is `rows` rows of a page, 128 bytes of them or all.
int encode_pages(CUtensorMap* map, const void* base, const PagedArrays& c, int rows, bool all);

// ATTN_OK when the current device is an sm_103, else the status to return; and
// what a launch needs to know of it, asked for once.
struct DeviceInfo {
  int dev, sms;
  unsigned int* err_word;
};
int check_device();
int device_info(DeviceInfo* out);

// Device error word of the current device (one-time per-device set-up);
// nullptr when the current device is unusable.
unsigned int* device_error_word();
uint64_t wait_limit_ns();

cudaError_t launch_fwd(const FwdParams& p, cudaStream_t stream);
size_t fwd_smem_bytes(int D, bool fp8);

// Checks the arguments of a split-KV decode on the host (exactly one of o /
// o_state is used; the other may be NULL) and fills every field of *p but the
// scratch pointers and the error word.  Returns an ATTN_* status.
int decode_prepare(const void* q, const void* kcache, const void* vcache, void* o, float* o_state,
                   float* lse, int B, int Hq, int Hkv, int Nk, int D, int nsplit,
                   DecodeParams* p);
// Checks the current device (sm_103) and sets p->err to its error word.
int decode_bind_device(DecodeParams* p);
// Bytes of partial-state scratch a decode needs; *o_bytes = the partial
// outputs' share (the partial lse follow them).
size_t decode_scratch_bytes(const DecodeParams& p, size_t* o_bytes);

// Binds the device, takes the partial-state scratch from the per-stream cache
// (or, during stream capture, from the stream-ordered allocator) and queues
// the split and combine kernels.  Returns an ATTN_* status.
int decode_with_cached_scratch(DecodeParams& p, cudaStream_t stream);
cudaError_t launch_decode_split(const DecodeParams& p, cudaStream_t stream);
cudaError_t launch_decode_combine(const DecodeParams& p, cudaStream_t stream);
bool decode_supported(int G, int D);

}  // namespace attn
