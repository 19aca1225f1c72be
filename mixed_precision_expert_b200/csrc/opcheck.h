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

// rows of `cols` values of sz bytes, ld values apart, as a set of bytes
struct Block {
    uintptr_t base;
    int64_t pitch, width, rows;
    Block(const void* p, int64_t r, int64_t cols, int64_t ld, int sz)
        : base(reinterpret_cast<uintptr_t>(p)), pitch(r > 1 ? ld * sz : cols * sz), width(cols * sz), rows(r) {}
    uintptr_t end() const {
        if (rows > 1 && pitch > (INT64_MAX / 4) / rows) return UINTPTR_MAX;  // more than any memory
        return base + (uintptr_t)((rows - 1) * pitch + width);
    }
};

// Whether two blocks share a byte. Blocks of one pitch (or one row and any block)
// whose spans interleave, columns of one buffer, share none when their columns do
// not meet; blocks of different pitches count as overlapping when their spans do.
inline bool overlap(const Block& p, const Block& q) {
    if (p.end() <= q.base || q.end() <= p.base) return false;
    if (p.rows == 1 && q.rows > 1) return overlap(q, p);
    if (p.rows > 1 && (q.rows == 1 || p.pitch == q.pitch)) {
        // where q's rows start in p's
        const int64_t at = q.base >= p.base ? (int64_t)(q.base - p.base) % p.pitch
                                            : (p.pitch - (int64_t)(p.base - q.base) % p.pitch) % p.pitch;
        return at < p.width || at + q.width > p.pitch;
    }
    return true;
}

}  // namespace mpe
