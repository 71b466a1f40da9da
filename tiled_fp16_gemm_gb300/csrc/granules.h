// Rows of a matrix that need not begin on 16 bytes, read as the aligned 16-byte granules
// around them.  Pure integer arithmetic, compiled for both host and device.
#pragma once

#include <cstdint>

#ifndef TG_HD
#if defined(__CUDACC__)
#define TG_HD __host__ __device__ __forceinline__
#else
#define TG_HD inline
#endif
#endif

namespace tg {

struct Granules {
    int32_t skip;   // bytes of the first granule before the row
    int32_t end;    // of the row, counted from the first granule's beginning on
    bool outside;   // the first granule begins before the matrix does: its other bytes are
                    // not the caller's.  (Not only in the first row: rows may lie less
                    // than 16 bytes apart.)
};

// The row of `bytes` bytes that begins `offset` bytes into the matrix at address `base`.
TG_HD Granules granules(uint64_t base, uint64_t offset, int32_t bytes) {
    const uint64_t at = base + offset;
    Granules g;
    g.skip = static_cast<int32_t>(at & 15);
    g.end = g.skip + bytes;
    g.outside = offset < static_cast<uint64_t>(g.skip);
    return g;
}

}  // namespace tg
