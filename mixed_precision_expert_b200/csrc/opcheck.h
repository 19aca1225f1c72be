// Host-side checks shared by the context-free operators (select.cu, linear.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace mpe {

// api.cu: keeps msg as the calling thread's last error and returns code.
int report_global_error(int code, const char* msg);
// The same with a printf-style message.
int report_global_errorf(int code, const char* fmt, ...);

inline bool aligned(const void* p, size_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

inline int type_bytes(int32_t type) { return type == 0 ? 4 : 2; }

// Multiprocessors of the current device (0: the query failed).
inline int current_sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return n;
}

}  // namespace mpe
