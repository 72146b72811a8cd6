// row_chunks.h -- which aligned 16-byte chunks of a row lie inside its matrix (host and device).
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MOE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MOE_HOST_DEVICE inline
#endif

namespace moe {

// A row of `bytes` bytes at address `row` in a matrix whose bytes are [first, last), as chunks of 16
// bytes from the aligned address at or below the row's start on: the row lies in [off, end) of them.
// A chunk may hold bytes in front of and behind the row, of other rows or between them, but it moves
// whole only where it lies inside the matrix.
struct RowChunks {
    int off, end;
    int from;      // first and number of the chunk addresses that may move whole
    unsigned many;
    MOE_HOST_DEVICE RowChunks(uintptr_t row, uintptr_t first, uintptr_t last, int bytes) {
        off = (int)(row & 15);
        end = off + bytes;
        const uintptr_t base = row - off, left = last - base;
        from = base < first ? (int)(first - base) : 0;
        const int to = left < (1u << 30) ? (int)left : 1 << 30;
        many = to - 15 > from ? (unsigned)(to - 15 - from) : 0u;
    }
    MOE_HOST_DEVICE bool whole(int c) const { return (unsigned)(c - from) < many; }
};

}  // namespace moe
