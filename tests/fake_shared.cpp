// The launches of attention over shared prefixes and of rotary positions with several axes for host-side tests (beside
// fake_cuda.cpp): a log of what ran while which device was current.
#include <cstdint>
#include <string>

#include <cuda_runtime_api.h>

#include "moe_attn.h"

extern "C" int fake_current();

namespace {
std::string g_log;
cudaError_t note(const char* what) {
  g_log += std::string(what) + "@" + std::to_string(fake_current()) + " ";
  return cudaSuccess;
}
}  // namespace

extern "C" const char* fake_shared_log() {
  static std::string last;
  last = g_log;
  g_log.clear();
  return last.c_str();
}

namespace moe {
struct KvView;
struct AttnArgs;
struct Share;
struct KvMaps;
struct AttnWs;
size_t attn_shared_workspace(const KvView&, const Share&, int, int) { return 4096; }
cudaError_t attn_shared_launch(const KvView&, const AttnArgs&, const Share&, const AttnWs&, void*, size_t have, size_t* need,
                               const KvMaps&, int, cudaStream_t) {
  *need = 4096;
  return have < *need ? cudaErrorInvalidValue : note("shared");
}
cudaError_t rope_axes_launch(const uint64_t*, const uint8_t*, int, float, bool, const moe_rope_tensor_t*,
                             const moe_rope_tensor_t*, int, moe_dtype_t, const int32_t*, int64_t, int, cudaStream_t) {
  return note("axes");
}
}  // namespace moe
