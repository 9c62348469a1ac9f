// Copying, forking, compacting and freeing the states of a cache: for every pair
// (src[i], dst[i]) and every layer, state dst[i] becomes what state src[i] was
// before the call (src[i] = -1: zeros).
//
// Memory-bound: every destination is written once and every source read once, however
// many destinations it has.
//
// The pairs may form any permutation of one cache (swaps, chains, cycles), so a
// destination must not be written before every pair that reads it has done so.
// No pair depends on another's bytes at a different offset inside the state, so the
// work is split by offset, not by pair: a CTA takes a slice of w 16-byte words at the
// same offset in every pair's state, reads all pairs' slices into shared memory, passes a
// barrier, and writes them.  Slices are independent, so nothing is ordered between
// CTAs, no copy of the data is made, and the next slice arrives (asynchronous copies)
// while one is written.
//
// Of two pairs with the same destination the later one counts, and pairs with the same
// source share what the first of them read: each CTA finds both with a hash table in
// shared memory before it starts.
//
// Measured on a B200: 96 pairs of 1 MiB states in four layers, half of them a permutation,
// 123 us = 6.14 TB/s (95 % of a copy's rate; 154 us with the slices held in registers
// and nothing read ahead).
#include "async_copy.cuh"
#include "layer.cuh"

namespace gdn2 {
namespace {

constexpr int kThreads = 512;
constexpr int kRing = 8192;                     // 16-byte words of shared memory for slices
constexpr int kMaxPairs = 4096;                 // two words of every pair fit
constexpr int kSkip = -2;

__device__ __forceinline__ unsigned hash_of(int d, int mask) { return ((unsigned)d * 2654435761u >> 7) & mask; }

// Enters `key` for pair i into the table and lets `better` decide which pair it keeps;
// at most n of the table's 2 n or more entries are taken, so every search ends.
template <typename F> __device__ __forceinline__ int find(int *keys, int table, int key, F at_entry) {
    unsigned at = hash_of(key, table - 1);
    while (true) {
        const int was = atomicCAS(keys + at, -1, key);
        if (was == -1 || was == key) return at_entry((int)at);
        at = (at + 1) & (table - 1);
    }
}

// AHEAD slices of kRing / AHEAD words each.
template <int AHEAD>
__global__ void __launch_bounds__(kThreads, 1)
state_copy_kernel(const uint4 *src_pool, uint4 *dst_pool, const int *__restrict__ src, const int *__restrict__ dst,
                  int n, int layers, int n_src, int n_dst, unsigned words, int log_w, int table, int ring_at) {
    constexpr int kSlice = kRing / AHEAD, kWords = kSlice / kThreads;
    extern __shared__ __align__(16) int sm[];
    int *s_src = sm, *s_dst = sm + n, *s_lead = sm + 2 * n, *s_key = sm + ring_at, *s_val = s_key + table;
    bool follows = false;
    if (n <= 32) {
        // One warp, a pair a lane: the last pair of each destination, then the first pair left
        // of each source, which reads for the others.
        const int i = threadIdx.x;
        if (i < 32) {
            int s = kSkip, d = -1;
            if (i < n) {
                s = __ldg(src + i);
                d = __ldg(dst + i);
            }
            if (!(d >= 0 && d < n_dst && s >= -1 && s < n_src)) s = kSkip;
            const unsigned same = __match_any_sync(0xffffffffu, s == kSkip ? -1 - i : d);
            if (31 - __clz(same) != i || (src_pool == dst_pool && s == d)) s = kSkip;
            const int lead = __ffs(__match_any_sync(0xffffffffu, s >= 0 ? s : -1 - i)) - 1;
            follows = lead != i;
            if (i < n) {
                s_src[i] = s;
                s_dst[i] = d;
                s_lead[i] = lead;
            }
        }
    } else {
        // The same with a hash table in shared memory.
        for (int i = threadIdx.x; i < table; i += kThreads) s_key[i] = s_val[i] = -1;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const int s = __ldg(src + i), d = __ldg(dst + i);
            const bool ok = d >= 0 && d < n_dst && s >= -1 && s < n_src;
            s_src[i] = ok ? s : kSkip;
            s_dst[i] = d;
            if (ok) find(s_key, table, d, [&](int at) { return atomicMax(s_val + at, i); });
        }
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const int s = s_src[i], d = s_dst[i];
            if (s == kSkip) continue;
            const int last = find(s_key, table, d, [&](int at) { return s_val[at]; });
            if (last != i || (src_pool == dst_pool && s == d)) s_src[i] = kSkip;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < table; i += kThreads) {
            s_key[i] = -1;
            s_val[i] = n;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kThreads)
            if (s_src[i] >= 0) find(s_key, table, s_src[i], [&](int at) { return atomicMin(s_val + at, i); });
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kThreads) {
            s_lead[i] = s_src[i] >= 0 ? find(s_key, table, s_src[i], [&](int at) { return s_val[at]; }) : i;
            follows |= s_lead[i] != i;
        }
    }
    const bool shared = __syncthreads_or(follows);

    const unsigned per_layer = words >> log_w, w = 1u << log_w;
    const int total = n << log_w;
    const long long items = (long long)layers * per_layer;
    uint4 *ring = reinterpret_cast<uint4 *>(sm + ring_at);
    auto base_of = [&](long long item, size_t states) {
        return (size_t)(item / per_layer) * states * words + ((size_t)(item % per_layer) << log_w);
    };
    auto fetch = [&](long long item, int stage) {
        if (item < items) {
            const uint4 *from = src_pool + base_of(item, n_src);
#pragma unroll
            for (int u = 0; u < kWords; ++u) {
                const int idx = threadIdx.x + u * kThreads, i = idx >> log_w;
                if (idx < total && s_src[i] >= 0 && s_lead[i] == i)
                    copy_async<16>(smem_address(ring + stage * kSlice + idx),
                                   from + (size_t)s_src[i] * words + (idx & (w - 1)));
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fetch(blockIdx.x + (long long)i * gridDim.x, i);
    int stage = 0;
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
        copy_wait<AHEAD - 1>();
        __syncthreads();                        // the whole slice has been read: it may be written
        uint4 *to = dst_pool + base_of(item, n_dst);
#pragma unroll
        for (int u = 0; u < kWords; ++u) {
            const int idx = threadIdx.x + u * kThreads, i = idx >> log_w;
            if (idx < total && s_src[i] != kSkip)
                __stcs(to + (size_t)s_dst[i] * words + (idx & (w - 1)),
                       s_src[i] >= 0 ? ring[stage * kSlice + (s_lead[i] << log_w) + (idx & (w - 1))]
                                     : make_uint4(0, 0, 0, 0));
        }
        if (shared) __syncthreads();            // other threads' words have been read, too
        fetch(item + (long long)AHEAD * gridDim.x, stage);
        stage = stage + 1 == AHEAD ? 0 : stage + 1;
    }
}

}  // namespace

int state_copy_max_pairs() { return kMaxPairs; }

cudaError_t launch_state_copy(const float *src_pool, float *dst_pool, const int *src, const int *dst, int n,
                              int layers, int n_src, int n_dst, size_t state_floats, cudaStream_t st) {
    int dev = 0, sms = 148;
    cudaError_t e = device_sms(&dev, &sms);
    if (e != cudaSuccess) return e;
    // One slice read ahead of the one that is written, unless the pairs are so many that half
    // the ring holds only 32 bytes (a sector) of each: then the whole ring is one slice.
    const bool ahead = n <= kRing / 8;
    const int slice = ahead ? kRing / 2 : kRing;
    int log_w = 10;                             // words of a state are a multiple of 1,024
    while (log_w > 1 && ((long long)n << log_w) > slice) --log_w;
    int table = 32;
    while (table < 2 * n) table *= 2;
    // the pairs, then the ring; the hash table, done with before the first copy, lies under the ring
    const int ring_at = (3 * n + 3) / 4 * 4;
    static_assert(3 * kMaxPairs * sizeof(int) + kRing * 16 <= 227 * 1024 && 4 * kMaxPairs * sizeof(int) <= kRing * 16,
                  "shared memory of a CTA");
    const size_t smem = ring_at * sizeof(int) + kRing * 16;
    auto kernel = ahead ? state_copy_kernel<2> : state_copy_kernel<1>;
    static std::atomic<unsigned long long> allowed[2];
    e = allow_shared(kernel, 3 * kMaxPairs * (int)sizeof(int) + kRing * 16, dev, allowed[ahead]);
    if (e != cudaSuccess) return e;
    const long long items = (long long)layers * (long long)((state_floats / 4) >> log_w);
    kernel<<<(unsigned)(items < sms ? items : sms), kThreads, smem, st>>>(
        reinterpret_cast<const uint4 *>(src_pool), reinterpret_cast<uint4 *>(dst_pool), src, dst, n, layers, n_src,
        n_dst, (unsigned)(state_floats / 4), log_w, table, ring_at);
    return cudaGetLastError();
}

}  // namespace gdn2
