// Internal helpers shared by the libgdn2 kernels (not part of the public ABI).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "gdn2.h"

namespace gdn2 {

// Element type of q, k, v, o.
template <typename T> struct Elem;
template <> struct Elem<float> {
    static __device__ __forceinline__ float load(const float *p) { return __ldg(p); }
    static __device__ __forceinline__ void store(float *p, float x) { *p = x; }
};
template <> struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ float load(const __nv_bfloat16 *p) { return __bfloat162float(__ldg(p)); }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
};

// alpha below FLT_MIN is treated as FLT_MIN (documented precondition: alpha > 0).
__device__ __forceinline__ float clamp_alpha(float a) { return fmaxf(a, 1.17549435e-38f); }

// Streaming (read-once / write-once) 16-byte accesses for the decode state.
__device__ __forceinline__ float4 ld_stream(const float4 *p) { return __ldcs(p); }
__device__ __forceinline__ void st_stream(float4 *p, float4 v) { __stcs(p, v); }

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

// Host-side launchers (one per kernel family); each returns cudaGetLastError().
cudaError_t launch_recurrent_step(const void *q, const void *k, const void *v, const float *alpha,
                                  const float *b, const float *w, float *S, void *o, int B, int H,
                                  int dk, int dv, gdn2_dtype dt, cudaStream_t stream);

// B sequences of T tokens (cu_seqlens == nullptr), or B packed sequences with device
// offsets cu_seqlens[0..B] into T tokens in all.
cudaError_t launch_chunk_simt(const void *q, const void *k, const void *v, const float *alpha,
                              const float *b, const float *w, const float *S0, void *o, float *S_T,
                              int B, int T, int H, int dk, int dv, gdn2_dtype dt, const int *cu_seqlens,
                              cudaStream_t stream);

// Chunkwise prefill on the tensor cores (BF16 q/k/v, d_k = d_v = 128): nseq
// sequences of T tokens each; or packed, with device offsets cu_seqlens[0..nseq]
// or device token ranges ranges[0..nseq) (x, y: tokens [x, y) of the flat axis;
// z != 0: written values taken as zero) into T tokens in all.  o may be null;
// only sequences below nst (all when nst < 0) write S_T.
bool chunk_tc_supported(int dk, int dv, gdn2_dtype dt);
cudaError_t launch_chunk_tc(const void *q, const void *k, const void *v, const void *alpha, const void *b,
                            const void *w, const float *S0, void *o, float *S_T, int nseq, int T, int H,
                            const int *cu_seqlens, bool logits, cudaStream_t stream, const int4 *ranges = nullptr,
                            int nst = -1);

// Segment-parallel prefill of B sequences of T tokens cut into P segments of L
// tokens (the last shorter): workspace of segmented_workspace_bytes(B, H, P).
size_t segmented_workspace_bytes(int B, int H, int P);
cudaError_t launch_chunk_segmented(const void *q, const void *k, const void *v, const float *alpha, const float *b,
                                   const float *w, const float *S0, void *o, float *S_T, int B, int T, int H,
                                   int P, int L, void *workspace, cudaStream_t stream);

// Chunkwise backward: prep, state and gradient launches.  workspace holds
// chunk_bwd_workspace_floats(B, T, H, dk, dv) floats.
size_t chunk_bwd_workspace_floats(int B, int T, int H, int dk, int dv);
cudaError_t launch_chunk_bwd(const void *q, const void *k, const void *v, const float *alpha, const float *b,
                             const float *w, const float *S0, const void *dO, const float *dST, void *dq, void *dk,
                             void *dv, float *dalpha, float *db, float *dw, float *dS0, float *workspace, int B,
                             int T, int H, int d_k, int d_v, gdn2_dtype dt, cudaStream_t stream);

// Output epilogue: rows = B*T*H rows of dv channels (dv 64 or 128).
cudaError_t launch_output_gate(const void *o, const void *g, const float *weight, float eps, void *y,
                               long long rows, int dv, gdn2_dtype dt, cudaStream_t stream);

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
