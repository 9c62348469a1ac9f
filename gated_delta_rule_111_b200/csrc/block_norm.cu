// The norm in front of a block, with the residual addition that ends the block
// before it.  Per token row of D channels,
//   h = x + scale * dropout(r),   rstd = 1 / sqrt(mean(h^2) + eps),   y = h * rstd * weight,
// and the gradient of both outputs.  dropout() draws its mask from a counter
// (philox.cuh), so the backward regenerates it.
//
// Memory-bound: the forward reads x and r once and writes h and y once, the
// backward reads dy, h, dh (and r for the scale's gradient) and writes dx and dr.
// One CTA holds one row at a time in registers, one 8-channel vector per thread
// (two above 8,192 channels), and walks the rows with a stride of the grid, so
// that weight and scale are read once per CTA and, in the backward, their
// gradients accumulate in registers over the CTA's rows.  The next row's loads
// are issued before the current row's reduction.  Rows whose width is no
// multiple of 8 are not 16-byte aligned; they go by 4-channel groups of single
// elements.
#include "common.cuh"
#include "philox.cuh"

namespace gdn2 {
namespace {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(bf16 x) { return __bfloat162float(x); }

// One thread's V consecutive channels of a row, as loaded.
template <typename T, bool ALIGNED> struct Frag;
template <> struct Frag<bf16, true> {
    static constexpr int V = 8;
    uint4 raw;
    __device__ __forceinline__ void load(const bf16 *row, int c, int D) {
        raw = c < D ? __ldcs(reinterpret_cast<const uint4 *>(row + c)) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(u[e] << 16);
            v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ void store(bf16 *row, int c, int D, const float (&v)[8]) {
        if (c >= D) return;
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
            u[e] = *reinterpret_cast<const uint32_t *>(&p);
        }
        *reinterpret_cast<uint4 *>(row + c) = make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <> struct Frag<float, true> {
    static constexpr int V = 8;
    float4 raw[2];
    __device__ __forceinline__ void load(const float *row, int c, int D) {
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        raw[0] = c < D ? __ldcs(reinterpret_cast<const float4 *>(row + c)) : zero;
        raw[1] = c < D ? __ldcs(reinterpret_cast<const float4 *>(row + c) + 1) : zero;
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = raw[0].x; v[1] = raw[0].y; v[2] = raw[0].z; v[3] = raw[0].w;
        v[4] = raw[1].x; v[5] = raw[1].y; v[6] = raw[1].z; v[7] = raw[1].w;
    }
    static __device__ __forceinline__ void store(float *row, int c, int D, const float (&v)[8]) {
        if (c >= D) return;
        reinterpret_cast<float4 *>(row + c)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(row + c)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
};
template <typename T> struct Frag<T, false> {
    static constexpr int V = 4;
    float raw[4];
    __device__ __forceinline__ void load(const T *row, int c, int D) {
#pragma unroll
        for (int e = 0; e < 4; ++e) raw[e] = c + e < D ? to_float(__ldcs(row + c + e)) : 0.f;
    }
    __device__ __forceinline__ void get(float (&v)[4]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = raw[e];
    }
    static __device__ __forceinline__ void store(T *row, int c, int D, const float (&v)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < D) Elem<T>::store(row + c + e, v[e]);
    }
};

template <int V> __device__ __forceinline__ void load_channels(const float *p, int c, int D, float fill, float (&v)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = p && c + e < D ? __ldg(p + c + e) : fill;
}

// Sum over the CTA, the same bits in every thread.  `buf` alternates between two
// halves from one call to the next, so one barrier per call is enough.
__device__ __forceinline__ float cta_sum(float x, float *buf) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return x;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < warps; ++i) s += buf[i];
    return s;
}

// dropout of V channels starting at column c (a multiple of 4)
template <int V>
__device__ __forceinline__ void drop(float (&v)[V], const Dropout &dp, uint2 key, uint2 offset, int row, int c) {
#pragma unroll
    for (int q = 0; q < V; q += 4) {
        const uint4 w = philox4x32(make_uint4((uint32_t)(c + q) >> 2, (uint32_t)row, offset.x, offset.y), key);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[q + e] = u[e] >= dp.threshold ? v[q + e] * dp.inv_keep : 0.f;
    }
}

__device__ __forceinline__ void rng_words(const Dropout &dp, uint2 &key, uint2 &offset) {
    key = offset = make_uint2(0u, 0u);
    if (!dp.rng) return;
    const unsigned long long s = __ldg(dp.rng), o = __ldg(dp.rng + 1);
    key = make_uint2((uint32_t)s, (uint32_t)(s >> 32));
    offset = make_uint2((uint32_t)o, (uint32_t)(o >> 32));
}

template <typename TS, typename TB, bool ALIGNED, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT)
residual_norm_kernel(const TS *x, const TB *r, const float *__restrict__ weight, const float *__restrict__ scale,
                     Dropout dp, float eps, TS *h, TB *y, float *__restrict__ rstd, int rows, int D) {
    using FS = Frag<TS, ALIGNED>;
    using FB = Frag<TB, ALIGNED>;
    constexpr int V = FS::V;
    __shared__ float red[2][32];
    uint2 key, offset;
    rng_words(dp, key, offset);
    float wt[VPT][V], sc[VPT][V];
    FS fx[VPT];
    FB fr[VPT];
    const float inv_d = 1.f / (float)D;
    int row = blockIdx.x;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = (j * blockDim.x + threadIdx.x) * V;
        load_channels<V>(weight, c, D, 0.f, wt[j]);
        load_channels<V>(scale, c, D, 1.f, sc[j]);
        fx[j].load(x + (size_t)row * D, c, D);
        if (r) fr[j].load(r + (size_t)row * D, c, D);
    }
    for (int it = 0; row < rows; row += gridDim.x, ++it) {
        float hv[VPT][V], ss = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = (j * blockDim.x + threadIdx.x) * V;
            fx[j].get(hv[j]);
            if (r) {
                float b[V];
                fr[j].get(b);
                if (dp.rng) drop<V>(b, dp, key, offset, row, c);
#pragma unroll
                for (int e = 0; e < V; ++e) hv[j][e] = fmaf(b[e], sc[j][e], hv[j][e]);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) ss = fmaf(hv[j][e], hv[j][e], ss);
        }
        if (row + (long long)gridDim.x < rows) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int c = (j * blockDim.x + threadIdx.x) * V;
                fx[j].load(x + (size_t)(row + gridDim.x) * D, c, D);
                if (r) fr[j].load(r + (size_t)(row + gridDim.x) * D, c, D);
            }
        }
        const float rs = rsqrtf(cta_sum(ss, red[it & 1]) * inv_d + eps);
        if (threadIdx.x == 0) rstd[row] = rs;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = (j * blockDim.x + threadIdx.x) * V;
            if (h) FS::store(h + (size_t)row * D, c, D, hv[j]);
#pragma unroll
            for (int e = 0; e < V; ++e) hv[j][e] = hv[j][e] * rs * wt[j][e];
            FB::store(y + (size_t)row * D, c, D, hv[j]);
        }
        if (row > rows - (int)gridDim.x) break;      // keeps row + gridDim.x below 2^31
    }
}

// The gradient.  With n = h rstd, t = weight dy:
//   dx = rstd (t - n mean(t n)) + dh,   dr = dropout'(scale dx),
//   dweight = sum_rows dy n,   dscale = sum_rows dx dropout(r).
// A CTA adds its rows' shares of the two sums in registers and writes them to its
// row of `part` ([gridDim][1 or 2][D]); reduce_parts_kernel adds those in a fixed
// order, so the result does not change from call to call.
template <typename TS, typename TB, bool ALIGNED, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT)
residual_norm_bwd_kernel(const TB *__restrict__ dy, const TS *__restrict__ h, const float *__restrict__ rstd,
                         const float *__restrict__ weight, const TS *dh, const TB *__restrict__ r,
                         const float *__restrict__ scale, Dropout dp, TS *dx, TB *__restrict__ dr,
                         float *__restrict__ part, int rows, int D) {
    using FS = Frag<TS, ALIGNED>;
    using FB = Frag<TB, ALIGNED>;
    constexpr int V = FS::V;
    __shared__ float red[2][32];
    uint2 key, offset;
    rng_words(dp, key, offset);
    float wt[VPT][V], sc[VPT][V], aw[VPT][V], as[VPT][V];
    FB fdy[VPT], fr[VPT];
    FS fh[VPT], fdh[VPT];
    const float inv_d = 1.f / (float)D;
    auto load_row = [&](int row) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = (j * blockDim.x + threadIdx.x) * V;
            fdy[j].load(dy + (size_t)row * D, c, D);
            fh[j].load(h + (size_t)row * D, c, D);
            if (dh) fdh[j].load(dh + (size_t)row * D, c, D);
            if (r) fr[j].load(r + (size_t)row * D, c, D);
        }
    };
    int row = blockIdx.x;
    load_row(row);
    float rs_next = __ldg(rstd + row);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = (j * blockDim.x + threadIdx.x) * V;
        load_channels<V>(weight, c, D, 0.f, wt[j]);
        load_channels<V>(scale, c, D, 1.f, sc[j]);
#pragma unroll
        for (int e = 0; e < V; ++e) aw[j][e] = as[j][e] = 0.f;
    }
    for (int it = 0; row < rows; row += gridDim.x, ++it) {
        const float rs = rs_next;
        float n[VPT][V], t[VPT][V], gx[VPT][V], b[VPT][V], dot = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            fdy[j].get(t[j]);
            fh[j].get(n[j]);
            if (dh) fdh[j].get(gx[j]);
            if (r) fr[j].get(b[j]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (!dh) gx[j][e] = 0.f;
                n[j][e] *= rs;
                aw[j][e] = fmaf(t[j][e], n[j][e], aw[j][e]);
                t[j][e] *= wt[j][e];
                dot = fmaf(t[j][e], n[j][e], dot);
            }
        }
        if (row + (long long)gridDim.x < rows) {
            load_row(row + gridDim.x);
            rs_next = __ldg(rstd + row + gridDim.x);
        }
        const float mean = cta_sum(dot, red[it & 1]) * inv_d;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = (j * blockDim.x + threadIdx.x) * V;
            float g[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                gx[j][e] = fmaf(rs, t[j][e] - n[j][e] * mean, gx[j][e]);
                g[e] = gx[j][e];
            }
            FS::store(dx + (size_t)row * D, c, D, gx[j]);
            if (dr || r) {
                float keep[V];
#pragma unroll
                for (int e = 0; e < V; ++e) keep[e] = 1.f;
                if (dp.rng) drop<V>(keep, dp, key, offset, row, c);      // 1 / (1 - p) or 0
                if (r) {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        as[j][e] = keep[e] != 0.f ? fmaf(g[e] * keep[e], b[j][e], as[j][e]) : as[j][e];
                }
                if (dr) {
#pragma unroll
                    for (int e = 0; e < V; ++e) g[e] = keep[e] != 0.f ? g[e] * sc[j][e] * keep[e] : 0.f;
                    FB::store(dr + (size_t)row * D, c, D, g);
                }
            }
        }
        if (row > rows - (int)gridDim.x) break;
    }
    float *pw = part + (size_t)blockIdx.x * (r ? 2 : 1) * D;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = (j * blockDim.x + threadIdx.x) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (c + e < D) {
                pw[c + e] = aw[j][e];
                if (r) pw[D + c + e] = as[j][e];
            }
        }
    }
}

// out0[c] = sum_g part[g][c] and out1[c] = sum_g part[g][D0 + c]: column sums of a
// [G][W] array of partial sums, W = D0 (+ D0 when out1 is given).  A CTA owns 32
// columns; its 32 warps take every 32nd row and are added in a fixed order.
__global__ void __launch_bounds__(1024)
reduce_parts_kernel(const float *__restrict__ part, int G, int W, int D0, float *__restrict__ out0,
                    float *__restrict__ out1) {
    __shared__ float acc[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < W)
        for (int g = warp; g < G; g += 32) s += part[(size_t)g * W + c];
    acc[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < W) {
        s = 0.f;
#pragma unroll
        for (int g = 0; g < 32; ++g) s += acc[g][lane];
        if (c < D0)
            out0[c] = s;
        else
            out1[c - D0] = s;
    }
}

int device_sms() {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

int threads_for(int D, bool aligned, int vpt) {
    const int per = (aligned ? 8 : 4) * vpt;
    return ((D + per - 1) / per + 31) / 32 * 32;
}

template <typename TS, typename TB, bool AL, int VPT>
cudaError_t fwd_typed(const void *x, const void *r, const float *weight, const float *scale, const Dropout &dp,
                      float eps, void *h, void *y, float *rstd, int rows, int D, cudaStream_t st) {
    const int threads = threads_for(D, AL, VPT);
    const int per_sm = threads >= 1024 ? 1 : 1024 / threads;
    const long long cap = (long long)device_sms() * (per_sm > 32 ? 32 : per_sm);
    const int grid = (int)(rows < cap ? rows : cap);
    auto kernel = threads <= 256   ? residual_norm_kernel<TS, TB, AL, VPT, 256>
                  : threads <= 512 ? residual_norm_kernel<TS, TB, AL, VPT, 512>
                                   : residual_norm_kernel<TS, TB, AL, VPT, 1024>;
    kernel<<<grid, threads, 0, st>>>(static_cast<const TS *>(x), static_cast<const TB *>(r), weight, scale, dp, eps,
                                     static_cast<TS *>(h), static_cast<TB *>(y), rstd, rows, D);
    return cudaGetLastError();
}

template <typename TS, typename TB>
cudaError_t fwd_sized(const void *x, const void *r, const float *weight, const float *scale, const Dropout &dp,
                      float eps, void *h, void *y, float *rstd, int rows, int D, cudaStream_t st) {
    if (D % 8 == 0) {
        if (D <= 8192) return fwd_typed<TS, TB, true, 1>(x, r, weight, scale, dp, eps, h, y, rstd, rows, D, st);
        return fwd_typed<TS, TB, true, 2>(x, r, weight, scale, dp, eps, h, y, rstd, rows, D, st);
    }
    if (D <= 4096) return fwd_typed<TS, TB, false, 1>(x, r, weight, scale, dp, eps, h, y, rstd, rows, D, st);
    return fwd_typed<TS, TB, false, 4>(x, r, weight, scale, dp, eps, h, y, rstd, rows, D, st);
}

struct BwdArgs {
    const void *dy, *h;
    const float *rstd, *weight;
    const void *dh, *r;
    const float *scale;
    Dropout dp;
    void *dx, *dr;
    float *dweight, *dscale, *part;
    int rows, D;
};

template <typename TS, typename TB, bool AL, int VPT>
cudaError_t bwd_typed(const BwdArgs &a, int grid, cudaStream_t st) {
    float *part = grid == 1 && !a.dscale ? a.dweight : a.part;       // one CTA's sums are the result
    const int threads = threads_for(a.D, AL, VPT);
    auto kernel = threads <= 256   ? residual_norm_bwd_kernel<TS, TB, AL, VPT, 256>
                  : threads <= 512 ? residual_norm_bwd_kernel<TS, TB, AL, VPT, 512>
                                   : residual_norm_bwd_kernel<TS, TB, AL, VPT, 1024>;
    kernel<<<grid, threads, 0, st>>>(
        static_cast<const TB *>(a.dy), static_cast<const TS *>(a.h), a.rstd, a.weight, static_cast<const TS *>(a.dh),
        static_cast<const TB *>(a.dscale ? a.r : nullptr), a.scale, a.dp, static_cast<TS *>(a.dx),
        static_cast<TB *>(a.dr), part, a.rows, a.D);
    return cudaGetLastError();
}

template <typename TS, typename TB> cudaError_t bwd_sized(const BwdArgs &a, int grid, cudaStream_t st) {
    if (a.D % 8 == 0) return a.D <= 8192 ? bwd_typed<TS, TB, true, 1>(a, grid, st) : bwd_typed<TS, TB, true, 2>(a, grid, st);
    return a.D <= 4096 ? bwd_typed<TS, TB, false, 1>(a, grid, st) : bwd_typed<TS, TB, false, 4>(a, grid, st);
}

// CTAs of the backward: the workspace holds one row of partial sums for each, so
// the count goes by the sizes alone.
int bwd_grid(int rows, int D) {
    const int threads = threads_for(D, D % 8 == 0, D % 8 == 0 ? (D <= 8192 ? 1 : 2) : (D <= 4096 ? 1 : 4));
    const int per_sm = threads >= 512 ? 1 : 512 / threads;
    const long long cap = 148ll * (per_sm > 16 ? 16 : per_sm);
    return (int)(rows < cap ? rows : cap);
}

}  // namespace

cudaError_t launch_reduce_parts(const float *part, int G, int W, int D0, float *out0, float *out1, cudaStream_t st) {
    reduce_parts_kernel<<<(W + 31) / 32, 1024, 0, st>>>(part, G, W, D0, out0, out1);
    return cudaGetLastError();
}

cudaError_t launch_residual_norm(const void *x, const void *r, const float *weight, const float *scale, double p,
                                 const unsigned long long *rng, float eps, void *h, void *y, float *rstd, int rows,
                                 int D, gdn2_dtype stream_dt, gdn2_dtype dt, cudaStream_t st) {
    const Dropout dp{p > 0.0 && r ? rng : nullptr, (uint32_t)(p * 4294967296.0), (float)(1.0 / (1.0 - p))};
    if (stream_dt == GDN2_BF16) return fwd_sized<bf16, bf16>(x, r, weight, scale, dp, eps, h, y, rstd, rows, D, st);
    if (dt == GDN2_BF16) return fwd_sized<float, bf16>(x, r, weight, scale, dp, eps, h, y, rstd, rows, D, st);
    return fwd_sized<float, float>(x, r, weight, scale, dp, eps, h, y, rstd, rows, D, st);
}

size_t residual_norm_bwd_workspace_bytes(int rows, int D) {
    return (size_t)bwd_grid(rows, D) * 2 * D * sizeof(float);
}

cudaError_t launch_residual_norm_bwd(const void *dy, const void *h, const float *rstd, const float *weight,
                                     const void *dh, const void *r, const float *scale, double p,
                                     const unsigned long long *rng, void *dx, void *dr, float *dweight, float *dscale,
                                     float *workspace, int rows, int D, gdn2_dtype stream_dt, gdn2_dtype dt,
                                     cudaStream_t st) {
    const Dropout dp{p > 0.0 ? rng : nullptr, (uint32_t)(p * 4294967296.0), (float)(1.0 / (1.0 - p))};
    const BwdArgs a{dy, h, rstd, weight, dh, r, scale, dp, dx, dr, dweight, dscale, workspace, rows, D};
    const int grid = bwd_grid(rows, D);
    cudaError_t e = stream_dt == GDN2_BF16 ? bwd_sized<bf16, bf16>(a, grid, st)
                    : dt == GDN2_BF16      ? bwd_sized<float, bf16>(a, grid, st)
                                           : bwd_sized<float, float>(a, grid, st);
    if (e != cudaSuccess || (grid == 1 && !dscale)) return e;
    return launch_reduce_parts(workspace, grid, dscale ? 2 * D : D, D, dweight, dscale, st);
}

}  // namespace gdn2
