// The scratch cache of the decodes (decode_scratch.cu) compiled for the host, over a fake
// of the CUDA calls that it makes: what waits for what, also when a call fails.
#include <stdio.h>
#include <string.h>

#include <cuda.h>
#include <cuda_runtime.h>

#include "decode_scratch.cu"

namespace {
int waits = 0, fail_waits = 0, fail_allocs = 0, mallocs = 0, launches = 0;
long long next_ptr = 0x1000;
}  // namespace

extern "C" {
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaGetDevice(int* d) { return *d = 0, cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* s) {
  return *s = cudaStreamCaptureStatusNone, cudaSuccess;
}
cudaError_t cudaStreamGetId(cudaStream_t s, unsigned long long* id) {
  return *id = reinterpret_cast<unsigned long long>(s), cudaSuccess;
}
cudaError_t cudaEventCreateWithFlags(cudaEvent_t* e, unsigned) {
  return *e = reinterpret_cast<cudaEvent_t>(next_ptr += 16), cudaSuccess;
}
cudaError_t cudaStreamWaitEvent(cudaStream_t, cudaEvent_t, unsigned) {
  if (fail_waits > 0) return --fail_waits, cudaErrorUnknown;
  return ++waits, cudaSuccess;
}
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMallocAsync(void** p, size_t, cudaStream_t) {
  if (fail_allocs > 0) return --fail_allocs, cudaErrorMemoryAllocation;
  return ++mallocs, *p = reinterpret_cast<void*>(next_ptr += 256), cudaSuccess;
}
cudaError_t cudaFreeAsync(void*, cudaStream_t) { return cudaSuccess; }
}

namespace attn {
int decode_bind_device(DecodeParams*) { return ATTN_OK; }
size_t decode_scratch_bytes(const DecodeParams&, size_t* o) { return *o = 0, 256; }
cudaError_t launch_decode_split(const DecodeParams&, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_decode_combine(const DecodeParams&, cudaStream_t) { return cudaSuccess; }
}  // namespace attn

int use(long long stream, size_t bytes = 256) {
  return attn::with_scratch(bytes, 0, reinterpret_cast<cudaStream_t>(stream),
                            [](void*, void*, cudaStream_t) -> int { return ++launches, ATTN_OK; }, nullptr);
}

#define CHECK(x) \
  if (!(x)) return printf("line %d: %s\n", __LINE__, #x), 1

int main() {
  // a stream's first use waits for the buffer's last one, the next ones are behind it
  for (long long s = 100; s < 108; ++s) {
    waits = 0;
    CHECK(use(s) == ATTN_OK && waits == 1);
    CHECK(use(s) == ATTN_OK && waits == 1);
  }
  CHECK(mallocs == 8);
  // a ninth stream takes over the least recently used buffer, behind its last use
  waits = 0;
  CHECK(use(108) == ATTN_OK && waits == 1 && mallocs == 8);
  // the per-thread stream's handle stands for many streams: every use waits
  const long long per_thread = reinterpret_cast<long long>(cudaStreamPerThread);
  waits = 0;
  for (int i = 0; i < 3; ++i) CHECK(use(per_thread) == ATTN_OK);
  CHECK(waits == 3);
  // a take-over whose wait failed: nothing is launched, and the next use waits
  launches = waits = 0;
  fail_waits = 1;
  CHECK(use(200) == ATTN_ERR_CUDA && launches == 0);
  CHECK(use(200) == ATTN_OK && waits == 1 && launches == 1);
  // a buffer that could not grow: the next use gets one
  launches = 0;
  fail_allocs = 1;
  CHECK(use(200, 4096) == ATTN_ERR_ALLOC && launches == 0);
  CHECK(use(200, 4096) == ATTN_OK && launches == 1);
  puts("ok");
  return 0;
}
