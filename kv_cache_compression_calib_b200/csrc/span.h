// Slot ranges of key tiles, in arithmetic that fits for rows of up to 2^31 - 256 slots.
// Plain C++: compiled for the device, and by the tests for the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define TRI_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define TRI_HOST_DEVICE inline
#endif

namespace tri {

// Slots start .. start + count - 1.
struct Span {
    int start, count;
};

// Of `tiles` key tiles of `bn` slots from tile `beg` on, the slots from `seen` on (the
// first that some row does not see) that lie before slot `there`.  An item's rows are at most
// 256 tokens, so these are a few hundred slots, however long the row is.
TRI_HOST_DEVICE Span unseen_span(int beg, int tiles, int bn, int seen, int64_t there) {
    const int begin = beg * bn, start = seen > begin ? seen : begin;
    const int64_t end = (int64_t)(beg + tiles) * bn, stop = there < end ? there : end;
    return Span{start, stop > start ? (int)(stop - start) : 0};
}

}  // namespace tri
