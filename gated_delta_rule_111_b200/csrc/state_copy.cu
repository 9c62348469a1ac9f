// Copying, forking, compacting and freeing the states of a cache: for every pair
// (src[i], dst[i]) and every layer, state dst[i] becomes what state src[i] was
// before the call (src[i] = -1: zeros).
//
// Memory-bound: every destination is written once and every source read once
// (a source with several destinations comes from L2 after its first read).
//
// The pairs may form any permutation of one cache (swaps, chains, cycles), so a
// destination must not be written before every pair that reads it has done so.
// No pair depends on another's bytes at a different offset inside the state, so the
// work is split by offset, not by pair: a CTA takes a slice of w 16-byte words at the
// same offset in every pair's state, holds all pairs' slices in registers, passes a
// barrier, and stores them.  Slices are independent, so nothing is ordered between
// CTAs and no copy of the data is made.
//
// Of two pairs with the same destination the later one counts: each CTA enters
// the destinations into a hash table in shared memory that keeps the largest pair.
#include "common.cuh"

namespace gdn2 {
namespace {

constexpr int kThreads = 512;
constexpr int kWords = 8;                       // 16-byte words per thread and slice
constexpr int kMaxPairs = kThreads * kWords;    // a slice is at least one word of every pair
constexpr int kSkip = -2;

__device__ __forceinline__ unsigned hash_of(int d, int mask) { return ((unsigned)d * 2654435761u >> 7) & mask; }

__global__ void __launch_bounds__(kThreads, 2)
state_copy_kernel(const uint4 *src_pool, uint4 *dst_pool, const int *__restrict__ src, const int *__restrict__ dst,
                  int n, int layers, int n_src, int n_dst, unsigned words, int log_w, int table) {
    extern __shared__ int sm[];
    int *s_src = sm, *s_dst = sm + n, *s_key = sm + 2 * n, *s_val = s_key + table;
    for (int i = threadIdx.x; i < table; i += kThreads) {
        s_key[i] = -1;
        s_val[i] = -1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int s = __ldg(src + i), d = __ldg(dst + i);
        const bool ok = d >= 0 && d < n_dst && s >= -1 && s < n_src;
        s_src[i] = ok ? s : kSkip;
        s_dst[i] = d;
        if (ok) {
            unsigned at = hash_of(d, table - 1);                    // at most n of >= 2 n entries are taken
            while (true) {
                const int was = atomicCAS(s_key + at, -1, d);
                if (was == -1 || was == d) break;
                at = (at + 1) & (table - 1);
            }
            atomicMax(s_val + at, i);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int d = s_dst[i];
        if (s_src[i] == kSkip) continue;
        unsigned at = hash_of(d, table - 1);
        while (s_key[at] != d) at = (at + 1) & (table - 1);
        if (s_val[at] != i || (src_pool == dst_pool && s_src[i] == d)) s_src[i] = kSkip;
    }
    __syncthreads();

    const unsigned per_layer = words >> log_w, w = 1u << log_w;
    const int total = n << log_w;
    for (long long item = blockIdx.x; item < (long long)layers * per_layer; item += gridDim.x) {
        const unsigned layer = (unsigned)(item / per_layer);
        const size_t base = (size_t)(item % per_layer) << log_w;
        const uint4 *from = src_pool + (size_t)layer * n_src * words + base;
        uint4 *to = dst_pool + (size_t)layer * n_dst * words + base;
        uint4 buf[kWords];
#pragma unroll
        for (int u = 0; u < kWords; ++u) {
            const int idx = threadIdx.x + u * kThreads;
            buf[u] = make_uint4(0, 0, 0, 0);
            if (idx < total) {
                const int s = s_src[idx >> log_w];
                if (s >= 0) buf[u] = __ldcs(from + (size_t)s * words + (idx & (w - 1)));
            }
        }
        __syncthreads();                        // every slice is read before any is written
#pragma unroll
        for (int u = 0; u < kWords; ++u) {
            const int idx = threadIdx.x + u * kThreads;
            if (idx < total && s_src[idx >> log_w] != kSkip)
                __stcs(to + (size_t)s_dst[idx >> log_w] * words + (idx & (w - 1)), buf[u]);
        }
    }
}

}  // namespace

int state_copy_max_pairs() { return kMaxPairs; }

cudaError_t launch_state_copy(const float *src_pool, float *dst_pool, const int *src, const int *dst, int n,
                              int layers, int n_src, int n_dst, size_t state_floats, cudaStream_t st) {
    int dev = 0, sms = 148;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    int log_w = 9;                              // words of a state are a multiple of 1,024
    while (log_w > 0 && ((long long)n << log_w) > kMaxPairs) --log_w;
    int table = 32;
    while (table < 2 * n) table *= 2;
    const size_t smem = (2 * (size_t)n + 2 * (size_t)table) * sizeof(int);
    static_assert((2 * kMaxPairs + 4 * kMaxPairs) * sizeof(int) <= 100 * 1024, "two CTAs per SM");
    if (smem > 48 * 1024) {
        e = cudaFuncSetAttribute(state_copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    const long long items = (long long)layers * (long long)((state_floats / 4) >> log_w), cap = 2ll * sms;
    state_copy_kernel<<<(unsigned)(items < cap ? items : cap), kThreads, smem, st>>>(
        reinterpret_cast<const uint4 *>(src_pool), reinterpret_cast<uint4 *>(dst_pool), src, dst, n, layers, n_src,
        n_dst, (unsigned)(state_floats / 4), log_w, table);
    return cudaGetLastError();
}

}  // namespace gdn2
