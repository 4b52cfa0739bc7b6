// The wait limit, the per-kernel timing records and the launch status that all
// entry points share.
#include "launch.h"

#include <cstring>

namespace ssd {

std::atomic<unsigned long long> g_wait_limit_ns{sm100::kDefaultWaitLimitNs};

namespace {

constexpr int kProfMax = 65536;
bool g_prof_on = false;
cudaEvent_t *g_prof_ev = nullptr;  // 2 * kProfMax events, created on first begin
const char *g_prof_name[kProfMax];
int g_prof_n = 0;

}  // namespace

ProfScope::ProfScope(const char *name, cudaStream_t st) : s(st) {
  if (g_prof_on && g_prof_n < kProfMax) {
    idx = g_prof_n++;
    g_prof_name[idx] = name;
    cudaEventRecord(g_prof_ev[2 * idx], s);
  }
}
ProfScope::~ProfScope() {
  if (idx >= 0) cudaEventRecord(g_prof_ev[2 * idx + 1], s);
}

ssd_status launch_status() {
  const bool host_err = take_host_error();
  return (cudaPeekAtLastError() == cudaSuccess && !host_err) ? SSD_OK : SSD_ERR_CUDA;
}

void allow_smem(const void *kernel, int bytes, std::atomic<uint64_t> &done) {
  int dev = 0;
  // the attribute belongs to the current device; past the 64th it is set in every call
  const uint64_t bit = cudaGetDevice(&dev) == cudaSuccess && dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess)
    done.fetch_or(bit, std::memory_order_relaxed);
}

}  // namespace ssd

using namespace ssd;

extern "C" {

uint64_t ssd_set_wait_limit_ns(uint64_t limit_ns) { return g_wait_limit_ns.exchange(limit_ns); }

ssd_status ssd_profile_begin(void) {
  if (!g_prof_ev) {
    g_prof_ev = new cudaEvent_t[2 * kProfMax];
    for (int i = 0; i < 2 * kProfMax; ++i)
      if (cudaEventCreate(&g_prof_ev[i]) != cudaSuccess) return SSD_ERR_CUDA;
  }
  g_prof_n = 0;
  g_prof_on = true;
  return SSD_OK;
}

int32_t ssd_profile_end(ssd_kernel_time *out, int32_t max_entries) {
  g_prof_on = false;
  if (!g_prof_ev) return 0;
  int n = 0;
  for (int i = 0; i < g_prof_n; ++i) {
    if (cudaEventSynchronize(g_prof_ev[2 * i + 1]) != cudaSuccess) return SSD_ERR_CUDA;
    float ms = 0.f;
    if (cudaEventElapsedTime(&ms, g_prof_ev[2 * i], g_prof_ev[2 * i + 1]) != cudaSuccess) return SSD_ERR_CUDA;
    int j = 0;
    while (j < n && strcmp(out[j].name, g_prof_name[i]) != 0) ++j;
    if (j == n) {
      if (n >= max_entries) continue;
      out[n++] = {g_prof_name[i], 0, 0.f};
    }
    out[j].launches += 1;
    out[j].total_ms += ms;
  }
  g_prof_n = 0;
  return n;
}

}  // extern "C"
