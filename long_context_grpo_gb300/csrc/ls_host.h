// Host-side helpers shared by the entry points' translation units: alignment checks, the NVTX
// range of an API call, the launch timer behind ls_timing_*, tensor-map encoding.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cstddef>
#include <cstdint>

namespace ls {

// One NVTX range per API call (visible to profilers; no-op without one attached).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

inline bool aligned_n(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0u; }
inline bool aligned16(const void* p) { return aligned_n(p, 16); }
inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Brackets the launches made during its lifetime when timing is enabled.
class LaunchTimer {
 public:
  LaunchTimer(int kernel, cudaStream_t s);
  ~LaunchTimer();
  LaunchTimer(const LaunchTimer&) = delete;
  LaunchTimer& operator=(const LaunchTimer&) = delete;

 private:
  int kernel_;
  cudaStream_t s_;
  cudaEvent_t start_ = nullptr, stop_ = nullptr;
};

// Tiled bf16 tensor map with 128-byte swizzle (an ls_status; ls_last_error() on failure).
int encode_bf16_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims,
                    const cuuint64_t* strides, const cuuint32_t* box);

}  // namespace ls
