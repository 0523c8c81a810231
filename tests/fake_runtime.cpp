// A CUDA runtime and kernel launchers that do nothing but write down what was called, with the device
// that was current and the stream: the library's host side (csrc/pool.cpp) is linked against it and
// tested on the CPU.  Devices are numbers; every address of a buffer lies on `g_buffer_device`.
#include <cuda_runtime.h>
#include <stdint.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>

#include "mkv_internal.h"
#include "selftest.h"

namespace {

int g_device = 0, g_buffer_device = 0;
char g_log[1 << 16];
size_t g_len = 0;
long g_allocations_left = -1;  // -1: host allocations never fail

cudaError_t note(const char* what, const void* stream = nullptr) {
  if (g_len + 128 < sizeof g_log)
    g_len += snprintf(g_log + g_len, sizeof g_log - g_len, "%s %d %llu\n", what, g_device,
                      static_cast<unsigned long long>(reinterpret_cast<uintptr_t>(stream)));
  return cudaSuccess;
}

void* allocate(size_t n) {
  if (g_allocations_left == 0) throw std::bad_alloc();
  if (g_allocations_left > 0) --g_allocations_left;
  void* p = std::malloc(n ? n : 1);
  if (!p) throw std::bad_alloc();
  return p;
}

}  // namespace

void* operator new(size_t n) { return allocate(n); }
void* operator new[](size_t n) { return allocate(n); }
void operator delete(void* p) noexcept { std::free(p); }
void operator delete[](void* p) noexcept { std::free(p); }
void operator delete(void* p, size_t) noexcept { std::free(p); }
void operator delete[](void* p, size_t) noexcept { std::free(p); }

extern "C" {

__attribute__((visibility("default"))) void fake_devices(int current, int of_buffers) {
  g_device = current;
  g_buffer_device = of_buffers;
}
__attribute__((visibility("default"))) int fake_current_device() { return g_device; }
__attribute__((visibility("default"))) const char* fake_log() {
  g_log[g_len] = 0;
  g_len = 0;
  return g_log;
}
// The n-th host allocation from now on and all later ones fail (-1: none).
__attribute__((visibility("default"))) void fake_allocations(long n) { g_allocations_left = n; }
__attribute__((visibility("default"))) long fake_allocations_left() { return g_allocations_left; }

cudaError_t cudaGetDevice(int* d) {
  *d = g_device;
  return cudaSuccess;
}
cudaError_t cudaSetDevice(int d) {
  g_device = d;
  return cudaSuccess;
}
const char* cudaGetErrorString(cudaError_t) { return "fake"; }
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes* a, const void*) {
  a->type = cudaMemoryTypeDevice;
  a->device = g_buffer_device;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int device) {
  *v = 100 + device;
  return cudaSuccess;
}
cudaError_t cudaEventCreate(cudaEvent_t* e) {
  *e = reinterpret_cast<cudaEvent_t>(uintptr_t(16));
  return note("event_create");
}
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t s) { return note("event_record", s); }
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventSynchronize(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventElapsedTime(float* ms, cudaEvent_t, cudaEvent_t) {
  *ms = 1.f;
  return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t s) { return note("memset_async", s); }
cudaError_t cudaMemset(void*, int, size_t) { return note("memset"); }
cudaError_t cudaMemcpy(void* to, const void*, size_t n, cudaMemcpyKind) {
  std::memset(to, 0, n);
  return note("memcpy");
}
cudaError_t cudaMemcpyAsync(void* to, const void*, size_t n, cudaMemcpyKind, cudaStream_t s) {
  std::memset(to, 0, n);
  return note("memcpy_async", s);
}
cudaError_t cudaStreamSynchronize(cudaStream_t s) { return note("stream_synchronize", s); }

}  // extern "C"

namespace mkv {

cudaError_t launch_append(const AppendParams&, cudaStream_t s) { return note("append", s); }
cudaError_t launch_demote(const DemoteParams&, cudaStream_t s) { return note("demote", s); }
cudaError_t launch_retag(const RetagParams&, cudaStream_t s) { return note("retag", s); }
cudaError_t launch_page_ops(PageOpParams&, cudaStream_t s) { return note("page_ops", s); }
cudaError_t launch_materialise(const MaterialiseParams&, cudaStream_t s) { return note("materialise", s); }
cudaError_t launch_pack(const PackParams&, cudaStream_t s) { return note("pack", s); }
cudaError_t launch_prompt(const PromptParams&, const PromptInputs&, cudaStream_t s) { return note("prompt", s); }
cudaError_t launch_rope(RopeParams&, cudaStream_t s) { return note("rope", s); }
cudaError_t launch_partial(const DecodeParams&, cudaStream_t s) { return note("partial", s); }
cudaError_t launch_merge(const DecodeParams&, cudaStream_t s) { return note("merge", s); }
cudaError_t launch_wait_selftest(int32_t*, uint64_t, cudaStream_t s) { return note("wait_selftest", s); }
cudaError_t launch_tc_logits_selftest(const void*, const void*, float*, int32_t*, cudaStream_t s) {
  return note("tc_selftest", s);
}
int prompt_tiles_per_unit(int) { return 2; }
bool partial_supported(int, int NC) { return NC >= 1 && NC <= 32; }
int partial_ctas_per_sm(int, int, int) {  // (set up on the device that is current)
  note("occupancy");
  return 1;
}
cudaError_t static_decode_scratch(void** p, size_t* n) {
  *p = reinterpret_cast<void*>(uintptr_t(1 << 20));
  *n = size_t(32) << 20;
  return note("scratch");
}

}  // namespace mkv
