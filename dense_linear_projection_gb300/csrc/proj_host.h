// Host helpers shared by the translation units of the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace projgb {

// Host-side fault injection (proj_api.cu): which kinds of calls fail.
constexpr int kFaultAlloc = 1, kFaultEncode = 2, kFaultLaunch = 4, kFaultDevice = 8;
int fault_mask();
inline bool launch_faulted() { return (fault_mask() & kFaultLaunch) != 0; }
int64_t fault_wait_place();  // of "wait<n>", −1 without

// Every device allocation of the library goes through here.
cudaError_t dev_malloc(void **p, size_t bytes);

// The current device's SM count, 0 if it is not a GB300 (compute capability
// 10.3), -1 if the runtime fails.  (Single attributes: the whole property
// structure takes over 100 us to fill.)
inline int gb300_sm_count() {
    int device = 0, major = 0, minor = 0, sms = 0;
    if (cudaGetDevice(&device) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
        cudaGetLastError();
        return -1;
    }
    return major == 10 && minor == 3 ? sms : 0;
}

// The device that a handle made now belongs to: the current one, -1 if the
// runtime fails.  Calls with the handle are refused while another is current:
// its scratch and its kernels' attributes are that device's.
inline int device_of_handle() {
    int device = -1;
    if (cudaGetDevice(&device) != cudaSuccess) {
        cudaGetLastError();
        return -1;
    }
    return (fault_mask() & kFaultDevice) ? device + 1 : device;
}
inline bool is_current(int device) {
    int now = -1;
    if (cudaGetDevice(&now) != cudaSuccess) cudaGetLastError();
    return now == device && now >= 0;
}

// A 4-D tensor map (a CUtensorMap at `map`) of 2- or 1-byte elements, boxes of b0 × b1 of the inner two
// dimensions; strides in bytes.  Two-byte rows are 128-byte swizzled.  False where the driver refuses it.
bool encode_4d(void *map, const void *ptr, int elem, const uint64_t (&dims)[4], const uint64_t (&strides)[3], uint32_t b0,
               uint32_t b1);

inline cudaStream_t as_stream(void *s) { return static_cast<cudaStream_t>(s); }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace projgb
