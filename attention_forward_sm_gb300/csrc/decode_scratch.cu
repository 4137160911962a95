// Partial-state scratch of the split decodes (attn_decode_splitkv, _states,
// attn_decode_varlen, attn_decode_prefix): a small per-device cache of device
// buffers, one per recently used stream, so that a decode step allocates nothing
// once its stream has been seen.
//
// Why: a stream-ordered cudaMallocAsync + cudaFreeAsync pair around the two
// decode kernels costs about 6 us of GPU time per call on GB300 (measured:
// 342 us per call against 336 us with a fixed scratch on the B8 Hq32 Hkv8
// Nk65536 step), about 2 % of a bandwidth-bound step.
//
// Ordering.  A buffer belongs to one stream at a time.  Each use records the
// entry's event after the launches, and the first use on another stream waits on
// it, so a buffer is never used by two calls at once.  Streams are told apart
// by their ids: a destroyed stream's handle may come back for a new stream while
// the old one still has work queued, its id does not.  A
// buffer that grows, or whose entry is taken over by another stream, is freed
// stream-ordered after that event.  Calls during stream capture take the
// plain stream-ordered allocation path, so a captured graph owns its scratch.
#include <cuda_runtime.h>

#include <mutex>

#include "../../include/attn.h"
#include "internal.h"

namespace attn {
namespace {

constexpr int kMaxDevices = 64;
constexpr int kEntries = 8;  // streams remembered per device

struct Entry {
  unsigned long long stream = 0;  // its id: unlike a handle, never given out again
  void* ptr = nullptr;
  size_t bytes = 0;
  cudaEvent_t done = nullptr;  // recorded after the entry's last use
  unsigned long long last_use = 0;
  bool live = false;
};

struct Cache {
  std::mutex mu;
  Entry e[kEntries];
  unsigned long long tick = 0;
};
Cache g_cache[kMaxDevices];

}  // namespace

int with_own_scratch(size_t bytes, cudaStream_t stream, int (*launch)(void*, void*, cudaStream_t),
                     void* ctx) {
  void* ws = nullptr;
  if (cudaMallocAsync(&ws, bytes, stream) != cudaSuccess) {
    cudaGetLastError();
    return ATTN_ERR_ALLOC;
  }
  int rc = launch(ctx, ws, stream);
  if (cudaFreeAsync(ws, stream) != cudaSuccess && rc == ATTN_OK) rc = ATTN_ERR_CUDA;
  return rc;
}

int with_scratch(size_t bytes, int dev, cudaStream_t stream,
                 int (*launch)(void*, void*, cudaStream_t), void* ctx) {
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cap) != cudaSuccess) {
    cudaGetLastError();
    return ATTN_ERR_CUDA;
  }
  if (cap != cudaStreamCaptureStatusNone) return with_own_scratch(bytes, stream, launch, ctx);

  if (dev < 0 || dev >= kMaxDevices) return ATTN_ERR_DEVICE;
  Cache& c = g_cache[dev];
  // held until the launches and the event record are queued, so that no
  // other host thread frees or regrows this buffer in between
  std::lock_guard<std::mutex> lock(c.mu);
  Entry* en = nullptr;
  unsigned long long id = 0;
  if (cudaStreamGetId(stream, &id) != cudaSuccess) {
    cudaGetLastError();
    return ATTN_ERR_CUDA;
  }
  for (Entry& x : c.e)
    if (x.live && x.stream == id) en = &x;
  // is the buffer's previous use in front of us on our stream?  (The handle of
  // the per-thread stream stands for another stream in every thread.)
  const bool same = en != nullptr && stream != cudaStreamPerThread;
  if (!en) {
    // a free entry, else the least recently used one
    for (Entry& x : c.e)
      if (!x.live) {
        en = &x;
        break;
      }
    if (!en) {
      en = &c.e[0];
      for (Entry& x : c.e)
        if (x.last_use < en->last_use) en = &x;
    }
    en->live = true;
    en->stream = id;
    if (!en->done && cudaEventCreateWithFlags(&en->done, cudaEventDisableTiming) != cudaSuccess) {
      en->live = false;
      return ATTN_ERR_CUDA;
    }
  }
  // after the entry's previous use, if another stream made it
  if (!same && cudaStreamWaitEvent(stream, en->done, 0) != cudaSuccess) {
    en->live = false;  // nobody's: whoever takes it next waits
    return ATTN_ERR_CUDA;
  }
  if (en->bytes < bytes) {
    if (en->ptr && cudaFreeAsync(en->ptr, stream) != cudaSuccess) {
      en->live = false;
      return ATTN_ERR_CUDA;
    }
    en->ptr = nullptr;
    en->bytes = 0;
    if (cudaMallocAsync(&en->ptr, bytes, stream) != cudaSuccess) {
      cudaGetLastError();
      en->ptr = nullptr;
      en->live = false;
      return ATTN_ERR_ALLOC;
    }
    en->bytes = bytes;
  }
  en->last_use = ++c.tick;
  int rc = launch(ctx, en->ptr, stream);
  // recorded even after a failed launch: whatever did get queued is covered
  if (cudaEventRecord(en->done, stream) != cudaSuccess && rc == ATTN_OK) rc = ATTN_ERR_CUDA;
  return rc;
}

int decode_with_cached_scratch(DecodeParams& p, cudaStream_t stream) {
  if (int rc = decode_bind_device(&p)) return rc;
  struct Ctx {
    DecodeParams* p;
    size_t o_bytes;
  } ctx = {&p, 0};
  const size_t bytes = decode_scratch_bytes(p, &ctx.o_bytes);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
  return with_scratch(
      bytes, dev, stream,
      [](void* c, void* ws, cudaStream_t s) -> int {
        DecodeParams& p = *static_cast<Ctx*>(c)->p;
        p.ws_o = static_cast<float*>(ws);
        p.ws_lse = reinterpret_cast<float*>(static_cast<char*>(ws) + static_cast<Ctx*>(c)->o_bytes);
        return launch_decode_split(p, s) == cudaSuccess &&
                       launch_decode_combine(p, s) == cudaSuccess
                   ? ATTN_OK
                   : ATTN_ERR_LAUNCH;
      },
      &ctx);
}

}  // namespace attn
