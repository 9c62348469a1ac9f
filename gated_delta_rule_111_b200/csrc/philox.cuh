// Counter-based random words for dropout: Philox4x32-10 (J. K. Salmon, M. A.
// Moraes, R. O. Dror, D. E. Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// SC 2011).  It maps (counter, key) to four 32-bit words with no state, so the
// forward pass and the backward pass draw the same mask and neither stores it.
//
// A round takes (x, y, z, w) to (hi(M1 z) ^ y ^ k0, lo(M1 z), hi(M0 x) ^ w ^ k1, lo(M0 x))
// and adds (W0, W1) to the key.  Here x is a thread's column group, which stays the
// same from row to row, y the row, and (z, w) the offset of the call.  The row enters
// the first round only through its x, the same in all threads, so of the first three
// rounds a thread keeps what does not depend on the row (Lane) and does one
// multiplication per row, and 14 in the other seven: 15 of 20.
#pragma once

#include <stdint.h>

namespace gdn2 {
namespace philox {

constexpr uint32_t M0 = 0xD2511F53u, M1 = 0xCD9E8D57u, W0 = 0x9E3779B9u, W1 = 0xBB67AE85u;

__device__ __forceinline__ uint32_t hi(uint32_t a, uint32_t b) { return (uint32_t)((uint64_t)a * b >> 32); }

// What a column group's first three rounds need besides the row.
struct Lane { uint32_t z1, x2, z2, w2; };
__device__ __forceinline__ Lane lane_for(uint32_t group, uint2 key, uint2 offset) {
    const uint32_t z0 = hi(M0, group) ^ offset.y ^ key.y;                       // after round 1
    const uint32_t x1 = hi(M1, z0) ^ M1 * offset.x ^ (key.x + W0);              // after round 2
    return {M0 * group ^ (key.y + W1), M1 * z0 ^ (key.x + 2 * W0), hi(M0, x1) ^ (key.y + 2 * W1), M0 * x1};
}

// A row's share: M0 times the x that round 1 gives it.
struct Row { uint32_t high, low; };
__device__ __forceinline__ Row row_for(uint32_t row, uint2 key, uint2 offset) {
    const uint64_t p = (uint64_t)M0 * (hi(M1, offset.x) ^ row ^ key.x);
    return {(uint32_t)(p >> 32), (uint32_t)p};
}

__device__ __forceinline__ uint4 words(const Lane &l, const Row &r, uint2 key) {
    const uint64_t p = (uint64_t)M1 * (r.high ^ l.z1);
    uint4 c = make_uint4((uint32_t)(p >> 32) ^ l.x2, (uint32_t)p, r.low ^ l.z2, l.w2);
#pragma unroll
    for (uint32_t i = 3; i < 10; ++i) {
        const uint64_t a = (uint64_t)M0 * c.x, b = (uint64_t)M1 * c.z;
        c = make_uint4((uint32_t)(b >> 32) ^ c.y ^ (key.x + i * W0), (uint32_t)b,
                       (uint32_t)(a >> 32) ^ c.w ^ (key.y + i * W1), (uint32_t)a);
    }
    return c;
}

}  // namespace philox

// The dropout of one call: element (row, column) is kept where its word -- word
// column % 4 of the counter (column / 4, row, offset), key = seed -- is at least
// `threshold` = floor(p 2^32), and is then scaled by 1 / (1 - p).
struct Dropout {
    const unsigned long long *rng;   // device: seed, offset; null: nothing is dropped
    uint32_t threshold;
    float inv_keep;
};

}  // namespace gdn2
