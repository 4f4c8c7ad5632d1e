// Host-side helpers shared by the library's translation units: launch
// accounting, argument checks, the device check and the workspace pool.
// Defined in infini_attn.cu; nothing here is exported from the library.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace infini {

constexpr size_t kAlign = 256;  // workspace buffers start on multiples of this
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
constexpr int kSms = 148;  // B200 SM count: grid sizing (device independent, so plans are too)

enum Phase { kPhaseUpdate = 0, kPhaseState = 1, kPhaseAttn = 2, kPhasePre = 3, kPhaseProj = 4, kPhaseBwd = 5, kPhaseBwdTc = 6,
             kPhaseBwdMemTc = 7, kPhases = 8 };

// Counts one kernel launch and, when its phase is being timed, brackets it
// with events on `stream`.  Construct right before the launch, destroy
// right after it.
struct LaunchScope {
  int phase;
  cudaStream_t stream;
  cudaEvent_t a = nullptr, b = nullptr;
  unsigned long long ctx = 0;
  LaunchScope(int ph, cudaStream_t st);
  ~LaunchScope();
};

unsigned long long current_context_id();
bool ranges_overlap(const void* a, size_t an, const void* b, size_t bn);
int check_device(bool need_tc);
int note_cuda_error(cudaError_t e);
int launch_status();
bool ws_alloc(void** ptr, size_t bytes, cudaStream_t stream);

}  // namespace infini
