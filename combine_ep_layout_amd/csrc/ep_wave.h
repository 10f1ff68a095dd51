// The wave's width and its uniform values, for kernels.  Not installed; callers
// use include/ep_layout.h.
#pragma once

#include <hip/hip_runtime.h>

namespace epk {
namespace {

constexpr int kWave = 64;

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

}  // namespace
}  // namespace epk
