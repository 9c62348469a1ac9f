// Gradient of the output epilogue y = o / sqrt(mean(o^2) + eps) * weight * sigmoid(g)
// (output_gate.cu), per (token, head) row of d_v channels.  With
// rstd = 1 / sqrt(mean(o^2) + eps), n = o rstd, s = sigmoid(g), t = dy weight s:
//   do = rstd (t - n mean(t n)),   dg = dy n weight s (1 - s),   dweight = sum_rows dy n s.
//
// Memory-bound: o, g and dy are read once, do and dg written once.  A lane holds 16
// bytes of a row (8 BF16 or 4 FP32 channels), so a row takes 8 to 32 lanes and its
// two sums are shuffles among them; rstd is formed again from o rather than kept by
// the forward.  A warp issues the loads of UNROLL row groups before it reduces any.
// dweight adds up in registers over the rows of a lane, then over the CTA in shared
// memory; each CTA writes one row of partial sums, and a second launch adds those in
// a fixed order, so the result does not change from call to call.
// With x = exp(-g): s = 1 / (1 + x) and 1 - s = x s, which keeps its digits where the gate
// is open, as a subtraction would not.  Where x is infinite, s = 0, and so is dg.
//
// Measured on a B200, 4 x 4,096 tokens x 16 heads of 128: BF16 57.8 us = 5.81 TB/s (90 % of a
// copy's rate), FP32 106.8 us = 6.28 TB/s (97 %).
// A lane of 8 BF16 channels keeps n, dy s and 1 - s over the sums' shuffles, which
// takes more than the 80 registers of three CTAs an SM (61 us with two row groups); with two
// CTAs of 128 registers it is four row groups that hide the memory (60.5 us with two).
// Where two already cover all rows in one round, they are taken: 4.0 us against 4.5 at 64
// tokens x 16 heads.  FP32 has 4 channels a lane and needs no more than two: 107 us, 111
// with four, 111 with three CTAs.
#include "layer.cuh"

namespace gdn2 {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kThreads = 256;
constexpr int kPerSm = 2;
constexpr int kMaxGrid = 148 * kPerSm;

template <typename T> struct Lane;
template <> struct Lane<bf16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(uint4 r, float (&v)[8]) {
        const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(u[e] << 16);
            v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
            u[e] = *reinterpret_cast<const uint32_t *>(&p);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <> struct Lane<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(uint4 r, float (&v)[4]) {
        v[0] = __uint_as_float(r.x); v[1] = __uint_as_float(r.y);
        v[2] = __uint_as_float(r.z); v[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};

template <typename T, int DV, int UNROLL>
__global__ void __launch_bounds__(kThreads, kPerSm)
output_gate_bwd_kernel(const T *__restrict__ dy, const T *__restrict__ o, const T *__restrict__ g,
                       const float *__restrict__ weight, float eps, T *__restrict__ d_o, T *__restrict__ d_g,
                       float *__restrict__ part, long long rows) {
    using L = Lane<T>;
    constexpr int N = L::N, LPR = DV / N, RPW = 32 / LPR, WARPS = kThreads / 32;
    __shared__ float acc[WARPS][DV];
    cudaTriggerProgrammaticLaunchCompletion();       // the sums' launch may be set up; it waits for this grid's end
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / LPR, at = lane % LPR;
    const long long groups = (rows + RPW - 1) / RPW, step = (long long)gridDim.x * WARPS * UNROLL;
    float wt[N], aw[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
        wt[e] = __ldg(weight + at * N + e);
        aw[e] = 0.f;
    }
    for (long long g0 = ((long long)blockIdx.x * WARPS + warp) * UNROLL; g0 < groups; g0 += step) {
        uint4 ro[UNROLL], rg[UNROLL], rd[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const long long row = (g0 + u) * RPW + sub;
            const size_t off = (size_t)row * LPR + at;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            const bool in = row < rows;
            ro[u] = in ? __ldcs(reinterpret_cast<const uint4 *>(o) + off) : zero;
            rd[u] = in ? __ldcs(reinterpret_cast<const uint4 *>(dy) + off) : zero;
            rg[u] = in ? __ldcs(reinterpret_cast<const uint4 *>(g) + off) : zero;
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const long long row = (g0 + u) * RPW + sub;
            float n[N], c[N], t[N];                 // o, then n; g, then 1 - s; dy, then dy s
            L::unpack(ro[u], n);
            L::unpack(rg[u], c);
            L::unpack(rd[u], t);
            // both sums in one pass over the row: mean(t n) = rstd * mean(t o)
            float ss = 0.f, dot = 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float x = __expf(-c[e]), s = __fdividef(1.f, 1.f + x);
                c[e] = __saturatef(x * s);
                t[e] *= s;
                ss = fmaf(n[e], n[e], ss);
                dot = fmaf(t[e] * wt[e], n[e], dot);
            }
#pragma unroll
            for (int m = LPR / 2; m > 0; m >>= 1) {
                ss += __shfl_xor_sync(0xffffffffu, ss, m);
                dot += __shfl_xor_sync(0xffffffffu, dot, m);
            }
            // behind the last row 0, so that without an eps its zeros add no 0 * inf to dweight
            const float rstd = row < rows ? rsqrtf(ss * (1.f / DV) + eps) : 0.f, mean = dot * rstd * (1.f / DV);
            float x[N], y[N];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                n[e] *= rstd;
                aw[e] = fmaf(t[e], n[e], aw[e]);
                const float dn = t[e] * wt[e];
                x[e] = rstd * (dn - n[e] * mean);
                y[e] = dn * n[e] * c[e];
            }
            if (row < rows) {
                const size_t off = (size_t)row * LPR + at;
                reinterpret_cast<uint4 *>(d_o)[off] = L::pack(x);
                reinterpret_cast<uint4 *>(d_g)[off] = L::pack(y);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
#pragma unroll
        for (int m = LPR; m < 32; m <<= 1) aw[e] += __shfl_xor_sync(0xffffffffu, aw[e], m);
        if (sub == 0) acc[warp][at * N + e] = aw[e];
    }
    __syncthreads();
    if (threadIdx.x < DV) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) s += acc[i][threadIdx.x];
        part[(size_t)blockIdx.x * DV + threadIdx.x] = s;
    }
}

// CTAs that rows of dv channels take, `unroll` row groups of a warp at a time.
template <typename T> long long ctas_for(long long rows, int dv, int unroll) {
    const int per = 32 / (dv / Lane<T>::N) * (kThreads / 32) * unroll;
    return (rows + per - 1) / per;
}

struct Args {
    const void *dy, *o, *g;
    const float *weight;
    float eps;
    void *d_o, *d_g;
    float *dweight, *workspace;
    long long rows;
};

template <typename T, int DV, int UNROLL> cudaError_t launch_typed(const Args &a, cudaStream_t st) {
    const long long need = ctas_for<T>(a.rows, DV, UNROLL);
    const int grid = (int)(need < kMaxGrid ? need : kMaxGrid);
    output_gate_bwd_kernel<T, DV, UNROLL><<<grid, kThreads, 0, st>>>(
        static_cast<const T *>(a.dy), static_cast<const T *>(a.o), static_cast<const T *>(a.g), a.weight, a.eps,
        static_cast<T *>(a.d_o), static_cast<T *>(a.d_g), grid == 1 ? a.dweight : a.workspace, a.rows);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || grid == 1) return e;                // one CTA's sums are the result
    return launch_reduce_parts(a.workspace, grid, DV, DV, a.dweight, nullptr, st);
}
template <int DV> cudaError_t launch_bf16(const Args &a, cudaStream_t st) {
    return ctas_for<bf16>(a.rows, DV, 2) > kMaxGrid ? launch_typed<bf16, DV, 4>(a, st) : launch_typed<bf16, DV, 2>(a, st);
}

}  // namespace

size_t output_gate_bwd_workspace_bytes(int dv) { return (size_t)kMaxGrid * dv * sizeof(float); }

cudaError_t launch_output_gate_bwd(const void *dy, const void *o, const void *g, const float *weight, float eps,
                                   void *d_o, void *d_g, float *dweight, float *workspace, long long rows, int dv,
                                   gdn2_dtype dt, cudaStream_t st) {
    const Args a{dy, o, g, weight, eps, d_o, d_g, dweight, workspace, rows};
    if (dt == GDN2_BF16) return dv == 128 ? launch_bf16<128>(a, st) : launch_bf16<64>(a, st);
    return dv == 128 ? launch_typed<float, 128, 2>(a, st) : launch_typed<float, 64, 2>(a, st);
}

}  // namespace gdn2
