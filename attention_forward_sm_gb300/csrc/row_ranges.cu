// attn_row_ranges: the key range [lo, hi) of every row of a batch whose rows
// hold packed documents, from the documents' lengths.
//
// A token at position i belongs to the document with the first end > i, ends
// being the running sum of the lengths (cut at N).  It sees that document
// [s, e), under a causal mask [s, max(i + 1, min(s + prefix, e))).
//
// 8 bytes written per token and 4 or 8 read per document: the work is too
// small to be bound by memory (8 x 131072 tokens: 8.4 MB), so it is one
// launch with no intermediate: a CTA takes kTokens tokens of one row, scans
// the lengths 1024 at a time up to its last token, and each thread finds its
// first token's document by bisection in the scanned ends in shared memory; the
// next three are in the same one or search behind it.  Bound by the latency of
// those steps and by instructions (a search per token: 65% of the issue slots):
// 4 x 4096 tokens 2.3 us, 8 x 131072 of 513 documents 6.6 us (7.4).
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/attn.h"
#include "internal.h"

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 4;                   // tokens and documents per thread
constexpr int kTokens = kThreads * kPer;  // tokens per CTA, documents per scan

__global__ void __launch_bounds__(kThreads)
    row_ranges_kernel(const int* __restrict__ doc_lens, const int* __restrict__ prefix_lens,
                      int2* __restrict__ ranges, int N, int M, int causal) {
  __shared__ int ends[kTokens];
  __shared__ int warp_sum[kThreads / 32];
  __shared__ int2 staged[kTokens];
  const int b = blockIdx.y;
  const int t0 = blockIdx.x * kTokens;
  const int last = min(t0 + kTokens, N) - 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int* lens = doc_lens + static_cast<size_t>(b) * M;
  int2 out[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) out[i] = make_int2(0, 0);

  int carry = 0;  // end of the documents scanned so far
  // sums saturate at N <= 2^30: min(x + y, N) of x, y <= N fits an int and is
  // associative, so the scan may group it as it likes
  for (int m0 = 0; m0 < M && carry <= last; m0 += kTokens) {
    int e[kPer], sum = 0;
    const int m = m0 + threadIdx.x * kPer;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int len = m + i < M ? min(max(lens[m + i], 0), N) : 0;
      sum = min(sum + len, N);
      e[i] = sum;
    }
    int scan = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int up = __shfl_up_sync(0xFFFFFFFFu, scan, d);
      if (lane >= d) scan = min(scan + up, N);
    }
    __syncthreads();  // ends and warp_sum of the previous turn are read
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    int before = carry, total = carry;  // ends before this thread's documents, and of all
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before = min(before + warp_sum[w], N);
      total = min(total + warp_sum[w], N);
    }
    const int up = __shfl_up_sync(0xFFFFFFFFu, scan, 1);
    if (lane > 0) before = min(before + up, N);
#pragma unroll
    for (int i = 0; i < kPer; ++i) ends[threadIdx.x * kPer + i] = min(before + e[i], N);
    __syncthreads();
    const int docs = min(kTokens, M - m0);
    int doc = -1;  // of the token before, in this turn
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int tok = t0 + threadIdx.x * kPer + i;
      if (tok < carry || tok >= total) continue;
      if (doc < 0 || ends[doc] <= tok) {
        int lo = doc + 1, hi = docs - 1;  // ends[docs - 1] = total > tok
        while (lo < hi) {
          const int mid = (lo + hi) / 2;
          if (ends[mid] > tok)
            hi = mid;
          else
            lo = mid + 1;
        }
        doc = lo;
      }
      const int s = doc > 0 ? ends[doc - 1] : carry, end = ends[doc];
      int vis = end;
      if (causal) {
        vis = tok + 1;
        if (prefix_lens) {
          const int pre = min(max(prefix_lens[static_cast<size_t>(b) * M + m0 + doc], 0), N);
          vis = max(vis, min(s + pre, end));
        }
      }
      out[i] = make_int2(s, vis);
    }
    carry = total;
  }
  // through shared memory, so that a warp writes consecutive tokens
#pragma unroll
  for (int i = 0; i < kPer; ++i) staged[threadIdx.x * kPer + i] = out[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int at = i * kThreads + threadIdx.x;
    if (t0 + at < N) ranges[static_cast<size_t>(b) * N + t0 + at] = staged[at];
  }
}

}  // namespace
}  // namespace attn

extern "C" int attn_row_ranges(const int* doc_lens, const int* prefix_lens, int* ranges, int B,
                               int N, int M, int causal, cudaStream_t stream) {
  using namespace attn;
  if (!doc_lens || !ranges) return ATTN_ERR_NULL;
  if (B < 1 || B > 65535 || N < 1 || N > (1 << 30) || M < 1 || M > (1 << 30))
    return ATTN_ERR_SHAPE;
  if (static_cast<long long>(B) * N >= (1ll << 40)) return ATTN_ERR_SHAPE;
  if ((reinterpret_cast<uintptr_t>(ranges) & 7u) || (reinterpret_cast<uintptr_t>(doc_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(prefix_lens) & 3u))
    return ATTN_ERR_ALIGN;
  if (int rc = check_device()) return rc;
  const dim3 grid(static_cast<unsigned>((N + kTokens - 1) / kTokens), static_cast<unsigned>(B));
  row_ranges_kernel<<<grid, kThreads, 0, stream>>>(doc_lens, prefix_lens,
                                                   reinterpret_cast<int2*>(ranges), N, M,
                                                   causal ? 1 : 0);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}
