// Host helpers shared by the translation units of the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace projgb {

// Host-side fault injection (proj_api.cu): which kinds of calls fail.
constexpr int kFaultAlloc = 1, kFaultEncode = 2, kFaultLaunch = 4;
int fault_mask();
inline bool launch_faulted() { return (fault_mask() & kFaultLaunch) != 0; }

// Every device allocation of the library goes through here.
cudaError_t dev_malloc(void **p, size_t bytes);

inline cudaStream_t as_stream(void *s) { return static_cast<cudaStream_t>(s); }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace projgb
