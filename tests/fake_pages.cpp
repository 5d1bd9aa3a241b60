// The launches of the page pool and of copying pages for host-side tests (beside fake_cuda.cpp): a log of what ran
// while which device was current.
#include <cstdint>
#include <string>

#include <cuda_runtime_api.h>

#include "moe_pages.h"

extern "C" {
int fake_current();
}

namespace {
std::string g_log;
cudaError_t note(const char* what) {
  g_log += std::string(what) + "@" + std::to_string(fake_current()) + " ";
  return cudaSuccess;
}
}  // namespace

extern "C" const char* fake_pages_log() {
  static std::string last;
  last = g_log;
  g_log.clear();
  return last.c_str();
}

namespace moe {
struct PagesView;
struct KvView;
cudaError_t pages_fork_launch(const PagesView&, const int32_t*, const int32_t*, const int32_t*, moe_page_move_t*, int,
                              cudaStream_t) {
  return note("fork");
}
cudaError_t pages_compact_launch(const PagesView&, moe_page_move_t*, int, cudaStream_t) { return note("compact"); }
cudaError_t kv_copy_launch(const KvView&, const moe_page_move_t*, int, int, cudaStream_t) { return note("copy"); }
}  // namespace moe
