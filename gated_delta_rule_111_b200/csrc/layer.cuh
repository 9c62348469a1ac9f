// Declarations of the operators around the recurrence (not part of the public ABI).
#pragma once

#include <atomic>

#include "common.cuh"

namespace gdn2 {

// The device's number of SMs, and a kernel's opt-in to more than 48 KB of shared memory,
// asked for once per device (`done`: one bit a device, a static of the call's own).
inline cudaError_t device_sms(int *dev, int *sms) {
    cudaError_t e = cudaGetDevice(dev);
    return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
}
template <typename K>
cudaError_t allow_shared(K kernel, int bytes, int dev, std::atomic<unsigned long long> &done) {
    const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
    if (bit && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// The norm in front of a block with the residual addition before it, rows of D
// channels; r null: no addition (h null too).  rng: device (seed, offset), read where p > 0.
cudaError_t launch_residual_norm(const void *x, const void *r, const float *weight, const float *scale, double p,
                                 const unsigned long long *rng, float eps, void *h, void *y, float *rstd, int rows,
                                 int D, gdn2_dtype stream_dt, gdn2_dtype dt, cudaStream_t stream);
// Its gradient; dh, dr and dscale (with r and scale) may be null.
size_t residual_norm_bwd_workspace_bytes(int rows, int D);
cudaError_t launch_residual_norm_bwd(const void *dy, const void *h, const float *rstd, const float *weight,
                                     const void *dh, const void *r, const float *scale, double p,
                                     const unsigned long long *rng, void *dx, void *dr, float *dweight, float *dscale,
                                     float *workspace, int rows, int D, gdn2_dtype stream_dt, gdn2_dtype dt,
                                     cudaStream_t stream);

// The output epilogue's gradient: rows = B*T*H rows of dv channels.
size_t output_gate_bwd_workspace_bytes(int dv);
cudaError_t launch_output_gate_bwd(const void *dy, const void *o, const void *g, const float *weight, float eps,
                                   void *d_o, void *d_g, float *dweight, float *workspace, long long rows, int dv,
                                   gdn2_dtype dt, cudaStream_t stream);

// Column sums of G rows of W partial sums: the first D0 columns to out0, the others to out1.
cudaError_t launch_reduce_parts(const float *part, int G, int W, int D0, float *out0, float *out1,
                                cudaStream_t stream);

// Tokens of N sequences against the states of a cache; logits: q .. w are BF16 logits.
cudaError_t launch_slot_steps(const void *q, const void *k, const void *v, const void *alpha, const void *b,
                              const void *w, bool logits, float *pool, const int *slots, const int *cu,
                              const int *keep, const void *gate, const float *weight, float eps, void *o, int N,
                              int T, int H, int n_slots, int dk, int dv, gdn2_dtype dt, cudaStream_t stream);

// Copies of whole states between slots of one cache or of two.
int state_copy_max_pairs();
cudaError_t launch_state_copy(const float *src_pool, float *dst_pool, const int *src, const int *dst, int n,
                              int layers, int n_src, int n_dst, size_t state_floats, cudaStream_t stream);

}  // namespace gdn2
