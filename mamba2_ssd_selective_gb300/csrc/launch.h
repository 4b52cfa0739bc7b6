// What the entry points' sources share: the wait limit, pointer checks, the
// per-kernel timing scope and the status of a launch sequence (launch.cu).
#pragma once

#include <atomic>
#include <cstdint>
#include <initializer_list>

#include "kernels.h"
#include "ssd.h"

namespace ssd {

// limit of the kernels' bounded hand-off waits, for every later call
extern std::atomic<unsigned long long> g_wait_limit_ns;

inline int elem_bytes(int dtype) { return dtype == SSD_BF16 ? 2 : 4; }
inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// limits of the token-major operators' dimensions
constexpr long long kMaxRows = 1LL << 30, kMaxChannels = 1 << 16;
constexpr int kMaxSeqs = 1 << 20;

// an output that starts where one of these inputs does
inline bool on_input(const void *out, std::initializer_list<const void *> inputs) {
  for (const void *p : inputs)
    if (out && out == p) return true;
  return false;
}

// brackets a launch with a pair of events while ssd_profile_begin is in effect
struct ProfScope {
  int idx = -1;
  cudaStream_t s;
  ProfScope(const char *name, cudaStream_t st);
  ~ProfScope();
};
#define SSD_LAUNCH(name, call) \
  do {                         \
    ProfScope _ps(name, s);    \
    call;                      \
  } while (0)

ssd_status launch_status();

// Lets a kernel take that much dynamic shared memory; `done` (the kernel's own) keeps the devices where it may already.
void allow_smem(const void *kernel, int bytes, std::atomic<uint64_t> &done);

}  // namespace ssd
