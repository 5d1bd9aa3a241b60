// A CUDA runtime and kernels for host-side tests of the attention-side entry points: several devices, memory known
// by its address (device d holds (d + 1) * 2^40 ..), and a log of what ran while which device was current.
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <string>

#include <cuda.h>
#include <cuda_runtime_api.h>

#include "moe_attn.h"

namespace moe {
struct KvView;
struct AttnArgs;
struct AttnWs;
struct KvMaps;
}  // namespace moe

namespace {

constexpr int kDevices = 4;
int g_current = 0, g_flags = 0;
uintptr_t g_next[kDevices];
std::string g_log, g_error;
uint64_t g_inc[128];  // the last rotary call's fractions of a turn per position

int device_of(const void* p) {
  const auto d = static_cast<long long>(reinterpret_cast<uintptr_t>(p) >> 40) - 1;
  return d >= 0 && d < kDevices ? static_cast<int>(d) : -1;
}
void note(const char* what) { g_log += std::string(what) + "@" + std::to_string(g_current) + " "; }

}  // namespace

extern "C" {

void fake_reset(int device) {
  g_current = device, g_flags = 0;
  g_log.clear();
  for (int d = 0; d < kDevices; ++d) g_next[d] = (static_cast<uintptr_t>(d + 1) << 40) + (1u << 30);
}
void fake_make_current(int device) { g_current = device; }
int fake_current() { return g_current; }
void fake_set_flags(int flags) { g_flags = flags; }
const char* fake_log() { return g_log.c_str(); }
void fake_clear_log() { g_log.clear(); }
uint64_t fake_rope_inc(int i) { return g_inc[i]; }

cudaError_t cudaGetDevice(int* d) {
  *d = g_current;
  return cudaSuccess;
}
cudaError_t cudaSetDevice(int d) {
  if (d < 0 || d >= kDevices) return cudaErrorInvalidDevice;
  g_current = d;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) {
  *v = 152;
  return cudaSuccess;
}
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes* a, const void* p) {
  memset(a, 0, sizeof(*a));
  const int d = device_of(p);
  if (d < 0) return cudaErrorInvalidValue;
  a->type = cudaMemoryTypeDevice;
  a->device = d;
  a->devicePointer = const_cast<void*>(p);
  return cudaSuccess;
}
cudaError_t cudaMalloc(void** p, size_t n) {
  *p = reinterpret_cast<void*>(g_next[g_current]);
  g_next[g_current] += (n + 255) / 256 * 256;
  note("malloc");
  return cudaSuccess;
}
cudaError_t cudaFree(void*) {
  note("free");
  return cudaSuccess;
}
cudaError_t cudaMemset(void*, int, size_t) {
  note("memset");
  return cudaSuccess;
}
cudaError_t cudaMemcpy(void* dst, const void*, size_t n, cudaMemcpyKind) {
  memcpy(dst, &g_flags, n < sizeof(g_flags) ? n : sizeof(g_flags));
  note("memcpy");
  return cudaSuccess;
}
cudaError_t cudaDeviceSynchronize() {
  note("sync");
  return cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "a fake error"; }

static CUresult encode_tiled(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** fn, unsigned int, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *fn = reinterpret_cast<void*>(&encode_tiled);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}

const char* moe_last_error(const moe_layer_t*) { return g_error.c_str(); }

}  // extern "C"

namespace moe {

void set_thread_error(const char* fmt, ...) {
  char text[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof(text), fmt, ap);
  va_end(ap);
  g_error = text;
}
const char* device_extent_error(const void* p, size_t, int device) {
  return device_of(p) == device ? nullptr : "lies elsewhere";
}
cudaError_t rope_launch(const uint64_t* inc, int rot_dim, float, bool, const moe_rope_tensor_t*, const moe_rope_tensor_t*, int,
                        moe_dtype_t, const int32_t*, int, cudaStream_t) {
  memcpy(g_inc, inc, sizeof(uint64_t) * (rot_dim / 2));
  note("rope");
  return cudaSuccess;
}
cudaError_t kv_write_launch(const KvView&, const void*, int64_t, const void*, int64_t, moe_dtype_t, cudaStream_t) {
  note("write");
  return cudaSuccess;
}
cudaError_t kv_read_launch(const KvView&, void*, void*, moe_dtype_t, cudaStream_t) {
  note("read");
  return cudaSuccess;
}
cudaError_t attn_few_launch(const KvView&, const AttnArgs&, const AttnWs&, const KvMaps&, int, cudaStream_t) {
  note("few");
  return cudaSuccess;
}
cudaError_t attn_tiles_launch(const KvView&, const AttnArgs&, const AttnWs&, const KvMaps&, int, cudaStream_t) {
  note("tiles");
  return cudaSuccess;
}

}  // namespace moe
