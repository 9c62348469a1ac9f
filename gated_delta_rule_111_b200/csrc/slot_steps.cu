// The recurrent form over a cache of states: sequence n owns state slots[n] and
// brings its next tokens (one while decoding, several while drafts are verified).
// Per token and head, as in the decode step:
//   Sbar = diag(alpha) S;  u = w v - Sbar^T (b k);  S' = Sbar + k u^T;  o = S'^T q = Sbar^T q + (k . q) u,
// optionally from BF16 pre-activation logits (q = silu(xq)/||silu(xq)||, k alike,
// v = silu(xv), alpha = 1/(1 + e^xa), b = sigmoid(xb), w = sigmoid(xw)) and optionally
// through the output epilogue (RMS norm over the head, weight, sigmoid gate).  The
// state after the first keep[n] tokens goes back to the slot.
//
// HBM-bound for a few tokens: a head's state (64 KiB at 128 x 128) is read once into
// registers and written once, whatever the number of tokens; a token costs 4 d_k d_v
// fused multiply-adds in between.
//
// One CTA per (sequence, head); the columns of a state evolve independently, so a
// warp owns 16 of them with all rows: lane = (row group of 8, column quad of 4), a
// lane holds d_k / 8 rows x 4 columns, and a 16-byte load takes 64 contiguous bytes
// of each of eight rows.  A token then needs no barrier: its two column sums
// (Sbar^T (b k) and Sbar^T q) are added over the eight row groups by seven shuffles
// that halve the number of sums at each step.  Rows are paired in 64-bit registers
// for the packed FP32 multiply-adds of sm_100, which halves their issue slots.
// Token vectors are staged in shared memory eight tokens at a time, one warp per
// token.
#include "common.cuh"
#include "f32x2.cuh"

namespace gdn2 {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kTile = 8;                  // tokens staged at a time

__device__ unsigned int g_slot_conflict = 0;   // nonzero: a slot was named by two sequences, one of them writing it

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// N (2 or 4) consecutive channels of a token's vector
template <int N> __device__ __forceinline__ void load_n(const float *p, float (&v)[N]) {
    if (N == 4) {
        const float4 r = __ldg(reinterpret_cast<const float4 *>(p));
        v[0] = r.x; v[1] = r.y; v[N - 2] = r.z; v[N - 1] = r.w;
    } else {
        const float2 r = __ldg(reinterpret_cast<const float2 *>(p));
        v[0] = r.x; v[1] = r.y;
    }
}
template <int N> __device__ __forceinline__ void load_n(const bf16 *p, float (&v)[N]) {
    if (N == 4) {
        const uint2 r = __ldg(reinterpret_cast<const uint2 *>(p));
        v[0] = __uint_as_float(r.x << 16); v[1] = __uint_as_float(r.x & 0xFFFF0000u);
        v[N - 2] = __uint_as_float(r.y << 16); v[N - 1] = __uint_as_float(r.y & 0xFFFF0000u);
    } else {
        const uint32_t r = __ldg(reinterpret_cast<const uint32_t *>(p));
        v[0] = __uint_as_float(r << 16); v[1] = __uint_as_float(r & 0xFFFF0000u);
    }
}
template <int N> __device__ __forceinline__ void store_n(float *p, const float (&v)[N]) {
    if (N == 4)
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[N - 2], v[N - 1]);
    else
        *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
}
template <int N> __device__ __forceinline__ void store_n(bf16 *p, const float (&v)[N]) {
#pragma unroll
    for (int e = 0; e < N; e += 2) *reinterpret_cast<__nv_bfloat162 *>(p + e) = __floats2bfloat162_rn(v[e], v[e + 1]);
}

struct StepArgs {
    const void *q, *k, *v, *alpha, *b, *w;     // alpha, b, w: FP32 values, or BF16 logits
    float *pool;
    const int *slots, *cu, *keep;
    const void *gate;                          // null: no epilogue
    const float *weight;
    float eps;
    void *o;
    int N, T, H, n_slots;
};

template <typename TIn, int DK, int DV, bool LOGITS>
__global__ void __launch_bounds__(DV * 2, DV == 128 ? 2 : 4)
slot_steps_kernel(const StepArgs a) {
    using TG = typename std::conditional<LOGITS, bf16, float>::type;
    constexpr int WARPS = DV / 16, PAIRS = DK / 16, CK = DK / 32, CV = DV / 32;
    __shared__ float4 s_ae[kTile][DK / 2], s_qk[kTile][DK / 2];       // (alpha, alpha', e, e'), (q, q', k, k') per row pair
    __shared__ __align__(16) float s_z[kTile][DV], s_o[kTile][DV];
    __shared__ float s_kq[kTile];

    const int seq = blockIdx.x / a.H, head = blockIdx.x - seq * a.H;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rg = lane >> 2, col = warp * 16 + (lane & 3) * 4;

    int t0 = seq, t1 = seq + 1;
    if (a.cu) {
        t0 = min(max(__ldg(a.cu + seq), 0), a.T);
        t1 = min(max(__ldg(a.cu + seq + 1), t0), a.T);
    }
    if (t0 >= t1) return;
    const int slot = __ldg(a.slots + seq);
    int keep = t1 - t0;
    if (a.keep) keep = min(max(__ldg(a.keep + seq), 0), keep);
    bool refused = slot < 0 || slot >= a.n_slots;

    // the state: rows 2m and 2m + 1 for m = rg + 8 j, four columns each
    float *Sh = a.pool + ((size_t)(refused ? 0 : slot) * a.H + head) * (DK * DV);
    Pair S[PAIRS][4];
    if (!refused) {
        float4 r0[PAIRS], r1[PAIRS];
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) {
            const float *p = Sh + (size_t)(2 * (rg + 8 * j)) * DV + col;
            r0[j] = __ldcs(reinterpret_cast<const float4 *>(p));
            r1[j] = __ldcs(reinterpret_cast<const float4 *>(p + DV));
        }
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) {
            S[j][0] = pack2(r0[j].x, r1[j].x); S[j][1] = pack2(r0[j].y, r1[j].y);
            S[j][2] = pack2(r0[j].z, r1[j].z); S[j][3] = pack2(r0[j].w, r1[j].w);
        }
    }

    // Two sequences that name one slot would race if either writes it: both are refused.
    bool clash = false;
    for (int m = tid; m < a.N; m += DV * 2) {
        if (m == seq || refused || __ldg(a.slots + m) != slot) continue;
        int len = 1;
        if (a.cu) {
            const int u0 = min(max(__ldg(a.cu + m), 0), a.T);
            len = min(max(__ldg(a.cu + m + 1), u0), a.T) - u0;
        }
        const int other = a.keep ? min(max(__ldg(a.keep + m), 0), len) : len;
        clash |= len > 0 && (keep > 0 || other > 0);
    }

    for (int base = t0; base < t1; base += kTile) {
        const int count = min(kTile, t1 - base);
        for (int i = warp; i < count; i += WARPS) {
            const size_t row = (size_t)(base + i) * a.H + head, ok = row * DK + lane * CK, ov = row * DV + lane * CV;
            float q[CK], k[CK], al[CK], b[CK], v[CV], w[CV];
            load_n<CK>(static_cast<const TIn *>(a.q) + ok, q);
            load_n<CK>(static_cast<const TIn *>(a.k) + ok, k);
            load_n<CK>(static_cast<const TG *>(a.alpha) + ok, al);
            load_n<CK>(static_cast<const TG *>(a.b) + ok, b);
            load_n<CV>(static_cast<const TIn *>(a.v) + ov, v);
            load_n<CV>(static_cast<const TG *>(a.w) + ov, w);
            if (LOGITS) {
                float sq = 0.f, sk = 0.f;
#pragma unroll
                for (int e = 0; e < CK; ++e) {
                    q[e] *= sigmoid(q[e]);
                    k[e] *= sigmoid(k[e]);
                    sq = fmaf(q[e], q[e], sq);
                    sk = fmaf(k[e], k[e], sk);
                    al[e] = sigmoid(-al[e]);
                    b[e] = sigmoid(b[e]);
                }
                sq = warp_sum(sq);
                sk = warp_sum(sk);
                const float iq = sq > 0.f ? rsqrtf(sq) : 0.f, ik = sk > 0.f ? rsqrtf(sk) : 0.f;   // a zero row stays zero
#pragma unroll
                for (int e = 0; e < CK; ++e) {
                    q[e] *= iq;
                    k[e] *= ik;
                }
#pragma unroll
                for (int e = 0; e < CV; ++e) {
                    v[e] *= sigmoid(v[e]);
                    w[e] = sigmoid(w[e]);
                }
            }
            float kq = 0.f;
#pragma unroll
            for (int e = 0; e < CK; ++e) kq = fmaf(k[e], q[e], kq);
            kq = warp_sum(kq);
            if (lane == 0) s_kq[i] = kq;
#pragma unroll
            for (int e = 0; e < CK; e += 2) {
                s_ae[i][(lane * CK + e) / 2] = make_float4(al[e], al[e + 1], b[e] * k[e], b[e + 1] * k[e + 1]);
                s_qk[i][(lane * CK + e) / 2] = make_float4(q[e], q[e + 1], k[e], k[e + 1]);
            }
#pragma unroll
            for (int e = 0; e < CV; ++e) s_z[i][lane * CV + e] = w[e] * v[e];
        }
        if (base == t0) {
            if (__syncthreads_or(clash)) {
                if (tid == 0) atomicOr(&g_slot_conflict, 1u);
                refused = true;
            }
        } else {
            __syncthreads();
        }
        if (refused) {                     // no state: this sequence's outputs are zero
            for (int i = tid; i < (t1 - t0) * DV; i += DV * 2)
                Elem<TIn>::store(static_cast<TIn *>(a.o) + ((size_t)(t0 + i / DV) * a.H + head) * DV + i % DV, 0.f);
            return;
        }

        for (int i = 0; i < count; ++i) {
            Pair r[4], p[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) r[c].v = p[c].v = 0ull;
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
                const float4 ae = s_ae[i][rg + 8 * j], qk = s_qk[i][rg + 8 * j];
                const Pair al = pack2(ae.x, ae.y), e = pack2(ae.z, ae.w), q = pack2(qk.x, qk.y);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    S[j][c] = mul2(S[j][c], al);
                    r[c] = fma2(S[j][c], e, r[c]);
                    p[c] = fma2(S[j][c], q, p[c]);
                }
            }
            // Add over the row groups: lane bit 4 keeps one of the two sums, bits 3 and 2 one column.
            float x[4];
            const bool up = lane & 16;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float r0, r1, p0, p1;
                unpack2(r[c], r0, r1);
                unpack2(p[c], p0, p1);
                r0 += r1;
                p0 += p1;
                x[c] = (up ? p0 : r0) + __shfl_xor_sync(0xffffffffu, up ? r0 : p0, 16);
            }
            const bool b3 = lane & 8, b2 = lane & 4;
            const float y0 = (b3 ? x[2] : x[0]) + __shfl_xor_sync(0xffffffffu, b3 ? x[0] : x[2], 8);
            const float y1 = (b3 ? x[3] : x[1]) + __shfl_xor_sync(0xffffffffu, b3 ? x[1] : x[3], 8);
            const float mine = (b2 ? y1 : y0) + __shfl_xor_sync(0xffffffffu, b2 ? y0 : y1, 4);
            const float other = __shfl_xor_sync(0xffffffffu, mine, 16);
            const int c_own = col + (b3 ? 2 : 0) + (b2 ? 1 : 0);
            const float u = s_z[i][c_own] - (up ? other : mine);
            if (up) s_o[i][c_own] = fmaf(s_kq[i], u, mine);
            Pair u2[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float uc = __shfl_sync(0xffffffffu, u, (lane & 3) | (c & 1) << 2 | (c & 2) << 2);
                u2[c] = pack2(uc, uc);
            }
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
                const float4 qk = s_qk[i][rg + 8 * j];
                const Pair k = pack2(qk.z, qk.w);
#pragma unroll
                for (int c = 0; c < 4; ++c) S[j][c] = fma2(k, u2[c], S[j][c]);
            }
            if (base + i - t0 + 1 == keep) {
#pragma unroll
                for (int j = 0; j < PAIRS; ++j) {
                    float4 r0, r1;
                    unpack2(S[j][0], r0.x, r1.x); unpack2(S[j][1], r0.y, r1.y);
                    unpack2(S[j][2], r0.z, r1.z); unpack2(S[j][3], r0.w, r1.w);
                    float *p2 = Sh + (size_t)(2 * (rg + 8 * j)) * DV + col;
                    __stcs(reinterpret_cast<float4 *>(p2), r0);
                    __stcs(reinterpret_cast<float4 *>(p2 + DV), r1);
                }
            }
        }
        __syncthreads();
        for (int i = warp; i < count; i += WARPS) {
            const size_t ov = ((size_t)(base + i) * a.H + head) * DV + lane * CV;
            float x[CV];
#pragma unroll
            for (int e = 0; e < CV; ++e) x[e] = s_o[i][lane * CV + e];
            if (a.gate) {
                float gv[CV], ss = 0.f;
                load_n<CV>(static_cast<const TIn *>(a.gate) + ov, gv);
#pragma unroll
                for (int e = 0; e < CV; ++e) ss = fmaf(x[e], x[e], ss);
                const float rs = rsqrtf(warp_sum(ss) * (1.f / DV) + a.eps);
#pragma unroll
                for (int e = 0; e < CV; ++e) x[e] = x[e] * rs * __ldg(a.weight + lane * CV + e) * sigmoid(gv[e]);
            }
            store_n<CV>(static_cast<TIn *>(a.o) + ov, x);
        }
    }
}

template <typename TIn, bool LOGITS>
cudaError_t launch_dims(const StepArgs &a, int dk, int dv, cudaStream_t st) {
    const unsigned grid = (unsigned)a.N * (unsigned)a.H;
    if (dk == 128 && dv == 128)
        slot_steps_kernel<TIn, 128, 128, LOGITS><<<grid, 256, 0, st>>>(a);
    else if (dk == 64 && dv == 64)
        slot_steps_kernel<TIn, 64, 64, LOGITS><<<grid, 128, 0, st>>>(a);
    else if (dk == 128)
        slot_steps_kernel<TIn, 128, 64, LOGITS><<<grid, 128, 0, st>>>(a);
    else
        slot_steps_kernel<TIn, 64, 128, LOGITS><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_slot_steps(const void *q, const void *k, const void *v, const void *alpha, const void *b,
                              const void *w, bool logits, float *pool, const int *slots, const int *cu,
                              const int *keep, const void *gate, const float *weight, float eps, void *o, int N,
                              int T, int H, int n_slots, int dk, int dv, gdn2_dtype dt, cudaStream_t st) {
    const StepArgs a{q, k, v, alpha, b, w, pool, slots, cu, keep, gate, weight, eps, o, N, T, H, n_slots};
    if (logits) return launch_dims<bf16, true>(a, dk, dv, st);
    if (dt == GDN2_BF16) return launch_dims<bf16, false>(a, dk, dv, st);
    return launch_dims<float, false>(a, dk, dv, st);
}

cudaError_t read_slot_conflict(unsigned int *value, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_slot_conflict, sizeof(unsigned int));
    if (e == cudaSuccess && clear && *value) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_slot_conflict, &zero, sizeof(unsigned int));
    }
    return e;
}

}  // namespace gdn2
