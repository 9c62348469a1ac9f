// Counter-based random words for dropout: Philox4x32-10 (J. K. Salmon, M. A.
// Moraes, R. O. Dror, D. E. Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// SC 2011).  A call maps (counter, key) to four 32-bit words with no state, so
// the forward pass and the backward pass draw the same mask and neither stores it.
#pragma once

#include <stdint.h>

namespace gdn2 {

__device__ __forceinline__ uint4 philox4x32(uint4 c, uint2 k) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p0 = (uint64_t)0xD2511F53u * c.x, p1 = (uint64_t)0xCD9E8D57u * c.z;
        c = make_uint4((uint32_t)(p1 >> 32) ^ c.y ^ k.x, (uint32_t)p1, (uint32_t)(p0 >> 32) ^ c.w ^ k.y, (uint32_t)p0);
        k.x += 0x9E3779B9u;
        k.y += 0xBB67AE85u;
    }
    return c;
}

// The dropout of one call: element (row, column) is kept where its word -- word
// column % 4 of the counter (column / 4, row, offset), key = seed -- is at least
// `threshold` = floor(p 2^32), and is then scaled by 1 / (1 - p).
struct Dropout {
    const unsigned long long *rng;   // device: seed, offset; null: nothing is dropped
    uint32_t threshold;
    float inv_keep;
};

}  // namespace gdn2
