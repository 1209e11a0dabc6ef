// abi.h -- host-side helpers shared by the files that implement C entry points
// (include/moe.h): argument checks, the device query and the optional
// per-kernel timing.  Not installed.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe.h"
#include "internal.h"

namespace moe {

constexpr size_t kHeader = 256;  // bytes ahead of every scratch layout; the status word is at offset 0

inline size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }
inline bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct DevInfo {
  int sms = 0;
  bool ok = false;
};
// The current device; MOE_ERR_UNSUPPORTED when it is no sm_103a part.
moe_status device_info(DevInfo *out);

// Per-kernel timing around one launch: a slot (or -1: not attached or full) and
// the event records before and after.
int timing_slot(const char *label);
bool timing_record(int slot, bool after, cudaStream_t s);

template <class F>
moe_status timed(const char *label, cudaStream_t s, F &&launch) {
  const int slot = timing_slot(label);
  if (slot >= 0 && !timing_record(slot, false, s)) return MOE_ERR_CUDA;
  const cudaError_t e = launch();
  if (slot >= 0 && e == cudaSuccess && !timing_record(slot, true, s)) return MOE_ERR_CUDA;
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

#define MOE_TRY(x)                      \
  do {                                  \
    moe_status _st = (x);               \
    if (_st != MOE_OK) return _st;      \
  } while (0)

}  // namespace moe
