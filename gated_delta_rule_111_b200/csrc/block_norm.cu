// The norm in front of a block, with the residual addition that ends the block
// before it.  Per token row of D channels,
//   h = x + scale * dropout(r),   rstd = 1 / sqrt(mean(h^2) + eps),   y = h * rstd * weight,
// and the gradient of both outputs.  dropout() draws its mask from a counter
// (philox.cuh), so the backward regenerates it.
//
// Memory-bound: the forward reads x and r once and writes h and y once, the
// backward reads dy, h, dh (and r for the scale's gradient) and writes dx and dr.
// One CTA holds one row at a time, 8 channels a thread (16 in the backward above
// 6,144), and walks the rows with a stride of the grid, so that weight and scale are
// read once per CTA and, in the backward, their gradients accumulate in registers over
// the CTA's rows. The next rows arrive by asynchronous copies into shared memory. What
// the layout has to keep: a lane's access covers whole 32-byte sectors together with
// its neighbours' (8 consecutive FP32 channels a lane cost 125 us where 4 cost 95,
// 16,384 x 2,048 backward with an FP32 stream), and not too much is in flight, 32 to
// 96 KB an SM in the forward and 60 to 136 in the backward (deeper rings were 5 to 15
// % slower). The dropout's integer work (about 80 instructions per 8 channels) comes
// before the wait for a row's data.
//
// Where D is no multiple of a vector, rows start inside one.  A CTA's rows all start at
// the same place of a vector, because they are a multiple of 8 rows apart, so its threads
// take aligned vectors that begin up to 7 channels before the row (SHIFT): a thread's
// channels stay the same from row to row, and only the vectors at a row's two ends are
// masked when read and written element by element.
//
// Measured on a B200, 16,384 x 2,048, residual scale and p = 0.1 (1 to 3 % between sessions):
// forward, BF16, 50 us = 5.37 TB/s (45 us without dropout); FP32 stream and BF16 branch 67 us =
// 6.0 TB/s, both FP32 94; backward, FP32 stream, 95.9 us = 6.30 TB/s (97 % of a copy's rate),
// BF16 75 us = 5.4 TB/s, bound there by the mask's and the conversions' instructions, both FP32
// 120.  Forward with a BF16 and an FP32 stream, backward with an FP32 and a BF16 one: 6,553 x
// 5,120 55, 63, 100 and 80 us; 4,096 x 8,192 53, 68, 116 and 99 us.  Shifted rows: 32,768 x 1,001
// forward without dropout 49.5 us = 5.30 TB/s; 16,384 x 2,047 with it, BF16, 87 us and
// backward 125 us, bound by putting the mask together and by the rows' ends.
#include "async_copy.cuh"
#include "f32x2.cuh"
#include "layer.cuh"
#include "philox.cuh"

namespace gdn2 {
namespace {

using bf16 = __nv_bfloat16;

// A vector: V consecutive channels of a row in one thread, as pairs, 8 or 16 bytes of
// every tensor, so that the lanes of a warp touch whole sectors (8 FP32 channels a lane
// would leave each access half of a sector).
template <typename TS, typename TB> constexpr int vector_channels() { return sizeof(TS) + sizeof(TB) == 4 ? 8 : 4; }

template <int BYTES> struct Raw;
template <> struct Raw<16> { uint4 u; };
template <> struct Raw<8> { uint2 u; };
template <typename T, int V> using RawOf = Raw<V * (int)sizeof(T)>;

__device__ __forceinline__ void widen(uint32_t u, Pair &v) {
    v = pack2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
__device__ __forceinline__ void unpack(const Raw<16> &r, Pair (&v)[4]) {       // 8 BF16
    widen(r.u.x, v[0]); widen(r.u.y, v[1]); widen(r.u.z, v[2]); widen(r.u.w, v[3]);
}
__device__ __forceinline__ void unpack(const Raw<8> &r, Pair (&v)[2]) {        // 4 BF16
    widen(r.u.x, v[0]); widen(r.u.y, v[1]);
}
__device__ __forceinline__ void unpack(const Raw<16> &r, Pair (&v)[2]) {       // 4 FP32
    v[0] = pack2(__uint_as_float(r.u.x), __uint_as_float(r.u.y));
    v[1] = pack2(__uint_as_float(r.u.z), __uint_as_float(r.u.w));
}
__device__ __forceinline__ uint32_t narrow(Pair v) {
    float a, b;
    unpack2(v, a, b);
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ void pack(const Pair (&v)[4], Raw<16> &r) {
    r.u = make_uint4(narrow(v[0]), narrow(v[1]), narrow(v[2]), narrow(v[3]));
}
__device__ __forceinline__ void pack(const Pair (&v)[2], Raw<8> &r) { r.u = make_uint2(narrow(v[0]), narrow(v[1])); }
__device__ __forceinline__ void pack(const Pair (&v)[2], Raw<16> &r) {
    float a, b, c, d;
    unpack2(v[0], a, b);
    unpack2(v[1], c, d);
    r.u = make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
}

// Masks V values of type T (one word of m per pair).
__device__ __forceinline__ void mask(Raw<16> &r, const uint32_t (&m)[4]) { r.u.x &= m[0]; r.u.y &= m[1]; r.u.z &= m[2]; r.u.w &= m[3]; }
__device__ __forceinline__ void mask(Raw<8> &r, const uint32_t (&m)[2]) { r.u.x &= m[0]; r.u.y &= m[1]; }
__device__ __forceinline__ void mask(Raw<16> &r, const uint32_t (&m)[2]) {
    r.u.x &= __byte_perm(m[0], 0, 0x1010); r.u.y &= __byte_perm(m[0], 0, 0x3232);
    r.u.z &= __byte_perm(m[1], 0, 0x1010); r.u.w &= __byte_perm(m[1], 0, 0x3232);
}

// The mask words of a vector whose first `skip` channels are the row before's.
template <int V> __device__ __forceinline__ void inside(int skip, uint32_t (&m)[V / 2]) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) m[i] = 2 * i >= skip ? 0xffffffffu : 2 * i + 1 >= skip ? 0xffff0000u : 0u;
}

// Writes the elements [from, to) of a vector, one of its ends being whole: single halves
// (BF16), words and pairs of words where they lie.
__device__ __forceinline__ void store_part(bf16 *p, const Raw<8> &r, int from, int to) {
    const uint32_t w[2] = {r.u.x, r.u.y};
    if (from & 1) reinterpret_cast<uint16_t *>(p)[from] = (uint16_t)((from & 2 ? w[1] : w[0]) >> 16);
    if (to & 1) reinterpret_cast<uint16_t *>(p)[to - 1] = (uint16_t)(to & 2 ? w[1] : w[0]);
    if (from <= 0 && to >= 2) reinterpret_cast<uint32_t *>(p)[0] = w[0];
    if (from <= 2 && to >= 4) reinterpret_cast<uint32_t *>(p)[1] = w[1];
}
__device__ __forceinline__ void store_part(bf16 *p, const Raw<16> &r, int from, int to) {
    const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
    if (from & 1) reinterpret_cast<uint16_t *>(p)[from] = (uint16_t)((from & 4 ? from & 2 ? w[3] : w[2] : from & 2 ? w[1] : w[0]) >> 16);
    if (to & 1) reinterpret_cast<uint16_t *>(p)[to - 1] = (uint16_t)(to & 4 ? to & 2 ? w[3] : w[2] : to & 2 ? w[1] : w[0]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (from <= 2 * i && to >= 2 * i + 2) reinterpret_cast<uint32_t *>(p)[i] = w[i];
}
__device__ __forceinline__ void store_part(float *p, const Raw<16> &r, int from, int to) {
    const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (from <= i && to >= i + 1) reinterpret_cast<uint32_t *>(p)[i] = w[i];
}

// Writes a vector to p, channels c and on of its row; where it reaches beyond the row (SHIFT),
// the channels of the row alone.
template <typename T, int V, bool SHIFT>
__device__ __forceinline__ void store(T *p, int c, int D, const Pair (&v)[V / 2], const uint32_t (*m)[V / 2] = nullptr) {
    RawOf<T, V> r;
    pack(v, r);
    if (m) mask(r, *m);
    if (c >= D) return;
    if (SHIFT && (c < 0 || c + V > D))
        store_part(p, r, c < 0 ? -c : 0, min(V, D - c));
    else
        *reinterpret_cast<decltype(r.u) *>(p) = r.u;
}

// Rows of one tensor on their way to a thread, VPT vectors of each row, by asynchronous
// copies into shared memory, S rows ahead.  A thread reads only what it copied itself, so
// waiting for its own copies is all the synchronisation there is.  A thread's vector j of
// a stage lies `at` + j vectors of MAXT threads into the stage; its first channel is
// c0 + j blockDim V.
template <typename T, int V, int VPT, int MAXT, int S, bool SHIFT> struct Rows {
    static constexpr int B = V * (int)sizeof(T), BYTES = VPT * MAXT * B;       // of a stage
    const T *base;
    int c0, D;
    // Vectors past the row's end are zero: set here once, never copied over.
    __device__ __forceinline__ void init(const T *p, int c, int d, uint32_t at, uint32_t stage_bytes) {
        base = p;
        c0 = c;
        D = d;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (c0 + j * (int)blockDim.x * V >= D)
                for (int i = 0; i < S; ++i) zero_shared<B>(at + i * stage_bytes + threadIdx.x * B + j * MAXT * B);
    }
    // `e`: the element offset of the thread's first vector.  Past a row's end nothing is read (the last
    // row's may be the tensor's).
    __device__ __forceinline__ void fetch(int j, size_t e, uint32_t at) {
        if (!base) return;
        const int c = c0 + j * (int)blockDim.x * V;
        const uint32_t to = at + threadIdx.x * B + j * MAXT * B;
        if (c >= D) return;
        if (SHIFT && c + V > D)
            copy_async_part<B>(to, base + e + j * (int)blockDim.x * V, (D - c) * (int)sizeof(T));
        else
            copy_async<B>(to, base + e + j * (int)blockDim.x * V);
    }
    __device__ __forceinline__ void fetch(size_t e, uint32_t at) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) fetch(j, e, at);
    }
    __device__ __forceinline__ void read(int j, uint32_t at, Pair (&v)[V / 2], const uint32_t (*m)[V / 2] = nullptr) {
        RawOf<T, V> r;
        load_shared(at + threadIdx.x * B + j * MAXT * B, r.u);
        if (m) mask(r, *m);
        if (SHIFT && c0 < 0 && j == 0) {           // the row before, in the first thread's vector
            uint32_t in[V / 2];
            inside<V>(-c0, in);
            mask(r, in);
        }
        unpack(r, v);
    }
};

// A [D] vector's channels of one thread, times `factor`; `fill` where p is null.  In
// registers, or (SHARED: instances of the backward that are short of them, bwd_shared) in
// the thread's own part of shared memory.
template <int V, int VPT, int MAXT, bool SHARED> struct Channels {
    Pair reg[SHARED ? 1 : VPT][V / 2];
    uint32_t at;
    __device__ __forceinline__ void init(const float *p, uint32_t smem, int c0, int D, float fill, float factor) {
        at = smem + threadIdx.x * 16;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = c0 + j * (int)blockDim.x * V;
            auto channel = [&](int at) { return (p && at >= 0 && at < D ? __ldg(p + at) : fill) * factor; };
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const Pair x = pack2(channel(c + 2 * i), channel(c + 2 * i + 1));
                if constexpr (SHARED)
                    store_shared(at + (j * V / 4 + i / 2) * MAXT * 16 + i % 2 * 8, x.v);
                else
                    reg[j][i] = x;
            }
        }
    }
    __device__ __forceinline__ void get(int j, Pair (&v)[V / 2]) const {
#pragma unroll
        for (int i = 0; i < V / 2; i += 2) {
            if constexpr (SHARED) {
                load_shared(at + (j * V / 4 + i / 2) * MAXT * 16, v[i].v, v[i + 1].v);
            } else {
                v[i] = reg[j][i];
                v[i + 1] = reg[j][i + 1];
            }
        }
    }
};

// Sum over the CTA, the same bits in every thread.  `buf` alternates between two
// halves from one call to the next, so one barrier per call is enough.
template <int MAXT> __device__ __forceinline__ float cta_sum(float x, float *buf) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (warps == 1) {
        __syncwarp();                       // as the barrier for what lanes leave to one another
        return x;
    }
    if (lane == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    constexpr int W = MAXT <= 64 ? 2 : MAXT <= 128 ? 4 : MAXT <= 256 ? 8 : MAXT <= 512 ? 16 : 32;
    x = (lane & (W - 1)) < warps ? buf[lane & (W - 1)] : 0.f;
#pragma unroll
    for (int m = W / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// Which channels of a thread's vectors a row keeps: one word per pair, its low half ones
// for the first channel and its high half for the second.  Two BF16 values are masked
// by one operation, and a dropped value leaves nothing, whatever it was.
//
// Vector j of a thread is vector n = j blockDim + threadIdx of the row.  The thread draws
// channels n V to n V + V - 1.  Where rows are not shifted, those are the vector's.  Where
// they are, its first `skip` channels are the last ones that vector n - 1 drew: a lane gets
// them from the lane before, and the first lane of a warp from shared memory, where the
// last lane of the warp before left them.  So a shifted row's channels are drawn
// (start) before the barrier of the row before it, and put together (finish) after it.
template <int V, int VPT, bool SHIFT> struct Keep {
    static constexpr int GROUPS = V / 4;               // groups of four channels
    philox::Lane lane[VPT][GROUPS];
    uint32_t m[VPT][V / 2], drawn[SHIFT ? VPT : 1];
    __device__ __forceinline__ void init(const Dropout &dp, uint2 key, uint2 offset) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int first = (j * (int)blockDim.x + (int)threadIdx.x) * GROUPS;
            if (dp.rng)
#pragma unroll
                for (int q = 0; q < GROUPS; ++q) lane[j][q] = philox::lane_for((uint32_t)(first + q), key, offset);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) m[j][i] = 0xffffffffu;
        }
    }
    __device__ __forceinline__ void draw(const Dropout &dp, uint2 key, uint2 offset, int row) {
        const philox::Row r = philox::row_for((uint32_t)row, key, offset);
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int q = 0; q < GROUPS; ++q) {
                const uint4 w = philox::words(lane[j][q], r, key);
                m[j][2 * q] = (w.x >= dp.threshold ? 0xffffu : 0u) | (w.y >= dp.threshold ? 0xffff0000u : 0u);
                m[j][2 * q + 1] = (w.z >= dp.threshold ? 0xffffu : 0u) | (w.w >= dp.threshold ? 0xffff0000u : 0u);
            }
    }
    // `left`: a word per vector and warp of shared memory, another one from row to row
    __device__ __forceinline__ void start(const Dropout &dp, uint2 key, uint2 offset, int row, uint32_t (*left)[32]) {
        const philox::Row r = philox::row_for((uint32_t)row, key, offset);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            uint32_t bits = 0;
#pragma unroll
            for (int q = 0; q < GROUPS; ++q) {
                const uint4 w = philox::words(lane[j][q], r, key);
                bits |= (w.x >= dp.threshold ? 1u << 4 * q : 0u) | (w.y >= dp.threshold ? 2u << 4 * q : 0u) |
                        (w.z >= dp.threshold ? 4u << 4 * q : 0u) | (w.w >= dp.threshold ? 8u << 4 * q : 0u);
            }
            drawn[j] = bits;
            if ((threadIdx.x & 31) == 31) left[j][threadIdx.x >> 5] = bits;
        }
    }
    __device__ __forceinline__ void finish(int skip, const uint32_t (*left)[32]) {
        const int warp = threadIdx.x >> 5;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            uint32_t before = __shfl_up_sync(0xffffffffu, drawn[j], 1);
            if ((threadIdx.x & 31) == 0)
                before = warp > 0 ? left[j][warp - 1] : j > 0 ? left[j - 1][(blockDim.x >> 5) - 1] : 0u;
            const uint32_t bits = (drawn[j] << V | before) >> (V - skip);
#pragma unroll
            for (int i = 0; i < V / 2; ++i)
                m[j][i] = (bits >> 2 * i & 1 ? 0xffffu : 0u) | (bits >> 2 * i & 2 ? 0xffff0000u : 0u);
        }
    }
};

__device__ __forceinline__ void rng_words(const Dropout &dp, uint2 &key, uint2 &offset) {
    key = offset = make_uint2(0u, 0u);
    if (!dp.rng) return;
    const unsigned long long s = __ldg(dp.rng), o = __ldg(dp.rng + 1);
    key = make_uint2((uint32_t)s, (uint32_t)(s >> 32));
    offset = make_uint2((uint32_t)o, (uint32_t)(o >> 32));
}

template <typename TS, typename TB, bool SHIFT, int VPT, int MAXT, int S>
__global__ void __launch_bounds__(MAXT, 1024 / MAXT)
residual_norm_kernel(const TS *x, const TB *r, const float *__restrict__ weight, const float *__restrict__ scale,
                     Dropout dp, float eps, TS *h, TB *y, float *__restrict__ rstd, int rows, int D) {
    constexpr int V = vector_channels<TS, TB>(), P = V / 2;
    using RS = Rows<TS, V, VPT, MAXT, S, SHIFT>;
    using RB = Rows<TB, V, VPT, MAXT, S, SHIFT>;
    constexpr uint32_t kStage = RS::BYTES + RB::BYTES;
    extern __shared__ uint4 ring[];
    __shared__ float red[2][32];
    __shared__ uint32_t left[2][SHIFT ? VPT : 1][32];
    const uint32_t ring0 = smem_address(ring);
    uint2 key, offset;
    rng_words(dp, key, offset);
    const int grid = gridDim.x;
    // the CTA's rows start `skip` channels into a vector
    const int skip = SHIFT ? (int)((size_t)blockIdx.x * D % V) : 0, c0 = threadIdx.x * V - skip;
    RS rx;
    RB rr;
    rx.init(x, c0, D, ring0, kStage);
    rr.init(r, c0, D, ring0 + RS::BYTES, kStage);
    const size_t step = (size_t)grid * D;
    int row = blockIdx.x, ahead = row;                  // the row in hand and the next one to fetch
    size_t e = (size_t)row * D + c0, e_ahead = e;
    auto fetch = [&](uint32_t at) {
        if (ahead < rows) {
            rx.fetch(e_ahead, at);
            rr.fetch(e_ahead, at + RS::BYTES);
        }
        ahead = ahead < rows - grid ? ahead + grid : rows;      // row + grid may pass 2^31
        e_ahead += step;
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < S; ++i) fetch(ring0 + i * kStage);
    Channels<V, VPT, MAXT, false> wt, sc;
    wt.init(weight, 0, c0, D, 0.f, 1.f);
    sc.init(scale, 0, c0, D, 1.f, dp.inv_keep);
    Keep<V, VPT, SHIFT> keep;
    keep.init(dp, key, offset);
    if (SHIFT && dp.rng) {
        keep.start(dp, key, offset, row, left[0]);
        __syncthreads();
    }
    const float inv_d = 1.f / (float)D;
    uint32_t at = ring0;
    for (int it = 0; row < rows; row += grid, it ^= 1) {
        if (dp.rng) {                               // before the wait: needs no data
            if constexpr (SHIFT)
                keep.finish(skip, left[it]);
            else
                keep.draw(dp, key, offset, row);
        }
        copy_wait<S - 1>();
        Pair hv[VPT][P], ss2 = pack2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            rx.read(j, at, hv[j]);
            if (r) {
                Pair b[P], s[P];
                rr.read(j, at + RS::BYTES, b, &keep.m[j]);
                sc.get(j, s);
#pragma unroll
                for (int i = 0; i < P; ++i) hv[j][i] = fma2(b[i], s[i], hv[j][i]);
            }
#pragma unroll
            for (int i = 0; i < P; ++i) ss2 = fma2(hv[j][i], hv[j][i], ss2);
        }
        fetch(at);                                  // this thread's part of the stage has been read
        at = at == ring0 + (S - 1) * kStage ? ring0 : at + kStage;
        if (SHIFT && dp.rng && row < rows - grid) keep.start(dp, key, offset, row + grid, left[it ^ 1]);
        float s0, s1;
        unpack2(ss2, s0, s1);
        const float rs = rsqrtf(cta_sum<MAXT>(s0 + s1, red[it]) * inv_d + eps);
        if (threadIdx.x == 0) rstd[row] = rs;
        const Pair rs2 = pack2(rs, rs);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = c0 + j * (int)blockDim.x * V;
            if (h) store<TS, V, SHIFT>(h + e + (c - c0), c, D, hv[j]);
            Pair w[P];
            wt.get(j, w);
#pragma unroll
            for (int i = 0; i < P; ++i) hv[j][i] = mul2(mul2(hv[j][i], rs2), w[i]);
            store<TB, V, SHIFT>(y + e + (c - c0), c, D, hv[j]);
        }
        e += step;
        if (row >= rows - grid) break;
    }
}

// The gradient.  With n = h rstd, t = weight dy:
//   dx = rstd (t - n mean(t n)) + dh,   dr = dropout'(scale dx),
//   dweight = sum_rows dy n,   dscale = sum_rows dx dropout(r).
// A CTA adds its rows' shares of the two sums in registers and writes them to its
// row of `part` ([gridDim][1 or 2][D]); reduce_parts_kernel adds those in a fixed
// order, so the result does not change from call to call.
// CTAs of the backward on an SM: 512 threads of 128 registers, or, where that would leave much
// of the SM idle, three CTAs of 192 or two of 320 (96 registers each): 13,107 x 2,560 BF16 74
// us, 96 with one CTA.  One CTA of more than 512 threads has 96 registers at 640, 80 at 768.
constexpr int bwd_ctas(int maxt) { return maxt == 192 ? 3 : maxt == 320 ? 2 : maxt <= 512 ? 512 / maxt : 1; }
// Those with fewer than 128 registers, and 16 channels a thread, keep weight and scale in shared memory.
constexpr bool bwd_shared(int maxt, int channels) { return channels == 16 || maxt > 512 || maxt == 192 || maxt == 320; }

template <typename TS, typename TB, bool SHIFT, int VPT, int MAXT, int S>
__global__ void __launch_bounds__(MAXT, bwd_ctas(MAXT))
residual_norm_bwd_kernel(const TB *__restrict__ dy, const TS *__restrict__ h, const float *__restrict__ rstd,
                         const float *__restrict__ weight, const TS *dh, const TB *__restrict__ r,
                         const float *__restrict__ scale, Dropout dp, TS *dx, TB *__restrict__ dr,
                         float *__restrict__ part, int rows, int D) {
    constexpr int V = vector_channels<TS, TB>(), P = V / 2;
    using RS = Rows<TS, V, VPT, MAXT, S, SHIFT>;
    using RB = Rows<TB, V, VPT, MAXT, S, SHIFT>;
    using C = Channels<V, VPT, MAXT, bwd_shared(MAXT, VPT * V)>;
    constexpr bool SPLIT = S == 1, DEEP = VPT * V == 16;       // DEEP: part of a row by part, to save registers
    static_assert(SPLIT || !DEEP, "one stage");
    constexpr uint32_t kDh = RS::BYTES, kDy = 2 * RS::BYTES, kR = kDy + RB::BYTES, kStage = kR + RB::BYTES;
    extern __shared__ uint4 ring[];
    __shared__ float red[2][32];
    __shared__ uint32_t left[2][SHIFT ? VPT : 1][32];
    cudaTriggerProgrammaticLaunchCompletion();       // the sums' launch may be set up; it waits for this grid's end
    const uint32_t ring0 = smem_address(ring);
    uint2 key, offset;
    rng_words(dp, key, offset);
    RB rdy, rr;
    RS rh, rdh;
    const int grid = gridDim.x;
    // the CTA's rows start `skip` channels into a vector
    const int skip = SHIFT ? (int)((size_t)blockIdx.x * D % V) : 0, c0 = threadIdx.x * V - skip;
    rdy.init(dy, c0, D, ring0 + kDy, kStage);
    rr.init(r, c0, D, ring0 + kR, kStage);
    rh.init(h, c0, D, ring0, kStage);
    rdh.init(dh, c0, D, ring0 + kDh, kStage);
    const size_t step = (size_t)grid * D;
    int row = blockIdx.x, ahead = row;                  // the row in hand and the next one to fetch
    size_t e = (size_t)row * D + c0, e_ahead = e;
    // A row comes in two parts: what its sum is made of, and what is wanted after the sum.  With one
    // row ahead (SPLIT) each part of the next row is sent for when this row's has been read (16,384 x
    // 2,048 FP32 120 us against 128); with two, both after the sum (BF16 74 us against 96).
    auto fetch_first = [&](int j, uint32_t at) {
        if (ahead >= rows) return;
        rdy.fetch(j, e_ahead, at + kDy);
        rh.fetch(j, e_ahead, at);
    };
    auto fetch_rest = [&](int j, uint32_t at) {
        if (ahead >= rows) return;
        rdh.fetch(j, e_ahead, at + kDh);
        rr.fetch(j, e_ahead, at + kR);
    };
    auto next_row = [&]() {
        ahead = ahead < rows - grid ? ahead + grid : rows;      // row + grid may pass 2^31
        e_ahead += step;
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) fetch_first(j, ring0 + i * kStage);
        if (SPLIT) copy_commit();
#pragma unroll
        for (int j = 0; j < VPT; ++j) fetch_rest(j, ring0 + i * kStage);
        next_row();
    }
    float rs_next = __ldg(rstd + row);
    C wt, sc;
    wt.init(weight, ring0 + S * kStage, c0, D, 0.f, 1.f);
    sc.init(scale, ring0 + S * kStage + VPT * MAXT * V * 4, c0, D, 1.f, dp.inv_keep);
    Pair aw[VPT][P], as[VPT][P];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
#pragma unroll
        for (int i = 0; i < P; ++i) aw[j][i] = as[j][i] = pack2(0.f, 0.f);
    }
    Keep<V, VPT, SHIFT> keep;
    keep.init(dp, key, offset);
    if (SHIFT && dp.rng) {
        keep.start(dp, key, offset, row, left[0]);
        __syncthreads();
    }
    const float inv_d = 1.f / (float)D;
    uint32_t at = ring0;
    for (int it = 0; row < rows; row += grid, it ^= 1) {
        if (dp.rng) {                               // before the wait: needs no data
            if constexpr (SHIFT)
                keep.finish(skip, left[it]);
            else
                keep.draw(dp, key, offset, row);
        }
        const float rs = rs_next;
        const Pair rs2 = pack2(rs, rs);
        copy_wait<SPLIT ? 2 * S - 1 : S - 1>();
        Pair n[VPT][P], t[VPT][P], dot2 = pack2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            rdy.read(j, at + kDy, t[j]);
            rh.read(j, at, n[j]);
            if (DEEP) fetch_first(j, at);
            Pair w[P];
            wt.get(j, w);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                n[j][i] = mul2(n[j][i], rs2);
                aw[j][i] = fma2(t[j][i], n[j][i], aw[j][i]);
                t[j][i] = mul2(t[j][i], w[i]);
                dot2 = fma2(t[j][i], n[j][i], dot2);
            }
        }
        if (SPLIT && !DEEP)
#pragma unroll
            for (int j = 0; j < VPT; ++j) fetch_first(j, at);
        if (SPLIT) copy_commit();
        const bool last = row >= rows - grid;
        if (!last) rs_next = __ldg(rstd + row + grid);
        if (SHIFT && dp.rng && !last) keep.start(dp, key, offset, row + grid, left[it ^ 1]);
        float d0, d1;
        unpack2(dot2, d0, d1);
        const float mean = -cta_sum<MAXT>(d0 + d1, red[it]) * inv_d;
        const Pair mean2 = pack2(mean, mean);
        if (SPLIT) copy_wait<2 * S - 1>();
        constexpr int STEP = DEEP ? 1 : VPT;        // vectors whose part behind the sum is in registers at once
#pragma unroll
        for (int j0 = 0; j0 < VPT; j0 += STEP) {
            Pair gx[STEP][P], b[STEP][P];
#pragma unroll
            for (int j = j0; j < j0 + STEP; ++j) {
                if (dh) rdh.read(j, at + kDh, gx[j - j0]);
                if (r) rr.read(j, at + kR, b[j - j0], &keep.m[j]);
#pragma unroll
                for (int i = 0; i < P; ++i)
                    if (!dh) gx[j - j0][i] = pack2(0.f, 0.f);
            }
#pragma unroll
            for (int j = j0; j < j0 + STEP; ++j) {
                if (!SPLIT) fetch_first(j, at);
                fetch_rest(j, at);
            }
            if (!DEEP) next_row();
#pragma unroll
            for (int j = j0; j < j0 + STEP; ++j) {
                const int c = c0 + j * (int)blockDim.x * V;
                Pair (&d)[P] = gx[j - j0];
#pragma unroll
                for (int i = 0; i < P; ++i) d[i] = fma2(rs2, fma2(n[j][i], mean2, t[j][i]), d[i]);
                store<TS, V, SHIFT>(dx + e + (c - c0), c, D, d);
                if (r) {                            // as is scaled by 1 / (1 - p) at the end
#pragma unroll
                    for (int i = 0; i < P; ++i) as[j][i] = fma2(d[i], b[j - j0][i], as[j][i]);
                }
                if (dr) {
                    Pair s[P];
                    sc.get(j, s);
#pragma unroll
                    for (int i = 0; i < P; ++i) d[i] = mul2(d[i], s[i]);
                    store<TB, V, SHIFT>(dr + e + (c - c0), c, D, d, &keep.m[j]);
                }
            }
        }
        if (DEEP) next_row();
        at = at == ring0 + (S - 1) * kStage ? ring0 : at + kStage;
        e += step;
        if (last) break;
    }
    float *pw = part + (size_t)blockIdx.x * (r ? 2 : 1) * D;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = c0 + j * (int)blockDim.x * V;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float a0, a1, s0, s1;
            unpack2(aw[j][i], a0, a1);
            unpack2(as[j][i], s0, s1);
            if (c + 2 * i >= 0 && c + 2 * i < D) {
                pw[c + 2 * i] = a0;
                if (r) pw[D + c + 2 * i] = s0 * dp.inv_keep;
            }
            if (c + 2 * i + 1 >= 0 && c + 2 * i + 1 < D) {
                pw[c + 2 * i + 1] = a1;
                if (r) pw[D + c + 2 * i + 1] = s1 * dp.inv_keep;
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
    cudaGridDependencySynchronize();
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

// How a width is split over a CTA: 8 channels a thread up to 8,192; a few shifted widths
// below that need one vector more.  The backward gives a thread 16 channels above 6,144
// (`deep`), where 8 would leave its threads 64 registers (4,096 x 8,192, FP32 stream: 115 us
// against 125; at 5,120 the other way round, 100 against 144).
struct Split {
    int threads;
    bool shift, more, deep;
};
Split split_for(int D, int V, bool bwd) {
    Split s{0, D % V != 0, false, false};
    const int vectors = s.shift ? (D + 2 * V - 2) / V : D / V, k = 8 / V;
    s.deep = bwd && vectors > 768 * k;
    s.more = !s.deep && vectors > 1024 * k;
    const int each = s.deep ? 2 * k : s.more ? k + 1 : k;
    s.threads = s.more ? 1024 : ((vectors + each - 1) / each + 31) / 32 * 32;
    return s;
}

// CTAs: as many as an SM holds (`per_sm` threads: 1,024 of the forward, 64 registers each; of the
// backward, whose two sums' accumulators take more, see bwd_ctas).  Shifted rows want a multiple of
// 8 where a CTA gets several, so that they all start at the same place of a vector.
int grid_for(int rows, const Split &s, int per_sm, int sms) {
    const int ctas = s.threads >= per_sm ? 1 : per_sm / s.threads;
    long long cap = (long long)sms * ctas;
    if (s.shift) cap = cap > 8 ? cap / 8 * 8 : 8;
    return (int)(rows < cap ? rows : cap);
}

struct FwdArgs {
    const void *x, *r;
    const float *weight, *scale;
    Dropout dp;
    float eps;
    void *h, *y;
    float *rstd;
    int rows, D;
};

template <typename TS, typename TB, bool SHIFT, int VPT, int MAXT>
cudaError_t fwd_launch(const FwdArgs &a, const Split &s, cudaStream_t st) {
    constexpr int bytes = VPT * vector_channels<TS, TB>() * (int)(sizeof(TS) + sizeof(TB));
    // One row ahead where CTAs of 1,024 threads in all share an SM, 32 to 64 KB (96 with a vector
    // more; two rows measured slower), two where one CTA of 513 to 768 has it alone and they are at
    // most 72 KB (6,553 x 5,120, FP32 stream and BF16 branch: 63 us against 74; both FP32: 96 against 86).
    constexpr int S = MAXT > 512 && MAXT <= 768 && 2 * bytes * MAXT <= 73728 ? 2 : 1;
    auto kernel = residual_norm_kernel<TS, TB, SHIFT, VPT, MAXT, S>;
    const size_t smem = (size_t)MAXT * bytes * S;
    static std::atomic<unsigned long long> allowed{0};
    int dev = 0, sms = 148;
    cudaError_t e = device_sms(&dev, &sms);
    if (e == cudaSuccess) e = allow_shared(kernel, (int)smem, dev, allowed);
    if (e != cudaSuccess) return e;
    kernel<<<grid_for(a.rows, s, 1024, sms), s.threads, smem, st>>>(
        static_cast<const TS *>(a.x), static_cast<const TB *>(a.r), a.weight, a.scale, a.dp, a.eps,
        static_cast<TS *>(a.h), static_cast<TB *>(a.y), a.rstd, a.rows, a.D);
    return cudaGetLastError();
}

struct BwdArgs {
    const void *dy, *h;
    const float *rstd, *weight;
    const void *dh, *r;
    const float *scale;
    Dropout dp;
    void *dx, *dr;
    float *part;
    int rows, D, grid;
};

template <typename TS, typename TB, bool SHIFT, int VPT, int MAXT>
cudaError_t bwd_launch(const BwdArgs &a, const Split &s, cudaStream_t st) {
    constexpr int bytes = VPT * vector_channels<TS, TB>() * 2 * (int)(sizeof(TS) + sizeof(TB));
    // Two rows in flight where 512 threads, or the CTA's if more, have at most 96 KB of them, else one.
    // The three CTAs of 192 and the two of 320 then have 108 and 120 KB an SM with an FP32 stream and a
    // BF16 branch, where one row is slower (23,172 x 1,448 100.4 us against 97.4, 13,107 x 2,560 97.1
    // against 94.7).
    constexpr int S = 2 * bytes * (MAXT > 512 ? MAXT : 512) <= 98304 ? 2 : 1;
    auto kernel = residual_norm_bwd_kernel<TS, TB, SHIFT, VPT, MAXT, S>;
    constexpr bool shared_channels = bwd_shared(MAXT, VPT * vector_channels<TS, TB>());     // weight and scale, see Channels
    const size_t smem = (size_t)MAXT * (bytes * S + (shared_channels ? 2 * VPT * vector_channels<TS, TB>() * 4 : 0));
    static std::atomic<unsigned long long> allowed{0};
    int dev = 0, sms = 148;
    cudaError_t e = device_sms(&dev, &sms);
    if (e == cudaSuccess) e = allow_shared(kernel, (int)smem, dev, allowed);
    if (e != cudaSuccess) return e;
    kernel<<<a.grid, s.threads, smem, st>>>(
        static_cast<const TB *>(a.dy), static_cast<const TS *>(a.h), a.rstd, a.weight, static_cast<const TS *>(a.dh),
        static_cast<const TB *>(a.r), a.scale, a.dp, static_cast<TS *>(a.dx), static_cast<TB *>(a.dr), a.part, a.rows,
        a.D);
    return cudaGetLastError();
}

// The instance that a width needs; k vectors make 8 channels.  The forward's have 64 registers a thread
// up to 512 threads and differ there in a stage's stride and the length of the last sum.  That matters
// for CTAs of 32 threads, of which an SM holds 32 if their stages are short (131,072 x 256 BF16 49 us, 61
// with the instance of 256); instances of 128, 192 and 320 measured like those of 256 and 512.  One of 640
// may use more registers than one of 768 (6,553 x 5,120, FP32 stream, BF16 branch: 63 us against 67).  For
// the backward's see bwd_ctas.
#define GDN2_UP_TO(THREADS, LAUNCH, SHIFT) \
    if (s.threads <= THREADS) return LAUNCH<TS, TB, SHIFT, k, THREADS>(a, s, st)
#define GDN2_FWD(SHIFT)                                         \
    {                                                           \
        GDN2_UP_TO(64, fwd_launch, SHIFT);                      \
        GDN2_UP_TO(256, fwd_launch, SHIFT);                     \
        GDN2_UP_TO(512, fwd_launch, SHIFT);                     \
        GDN2_UP_TO(640, fwd_launch, SHIFT);                     \
        return fwd_launch<TS, TB, SHIFT, k, 768>(a, s, st);     \
    }
#define GDN2_BWD(SHIFT)                                         \
    {                                                           \
        GDN2_UP_TO(64, bwd_launch, SHIFT);                      \
        GDN2_UP_TO(128, bwd_launch, SHIFT);                     \
        GDN2_UP_TO(192, bwd_launch, SHIFT);                     \
        GDN2_UP_TO(256, bwd_launch, SHIFT);                     \
        GDN2_UP_TO(320, bwd_launch, SHIFT);                     \
        GDN2_UP_TO(512, bwd_launch, SHIFT);                     \
        GDN2_UP_TO(640, bwd_launch, SHIFT);                     \
        return bwd_launch<TS, TB, SHIFT, k, 768>(a, s, st);     \
    }

template <typename TS, typename TB> cudaError_t fwd_sized(const FwdArgs &a, cudaStream_t st) {
    constexpr int V = vector_channels<TS, TB>(), k = 8 / V;
    const Split s = split_for(a.D, V, false);
    if (s.more) return fwd_launch<TS, TB, true, k + 1, 1024>(a, s, st);
    if (s.threads > 768)
        return s.shift ? fwd_launch<TS, TB, true, k, 1024>(a, s, st) : fwd_launch<TS, TB, false, k, 1024>(a, s, st);
    if (s.shift) GDN2_FWD(true)
    GDN2_FWD(false)
}
template <typename TS, typename TB> cudaError_t bwd_sized(const BwdArgs &a, cudaStream_t st) {
    constexpr int V = vector_channels<TS, TB>(), k = 8 / V;
    const Split s = split_for(a.D, V, true);
    if (s.deep) {
        if (s.threads > 512) return bwd_launch<TS, TB, true, 2 * k, 544>(a, s, st);
        return s.shift ? bwd_launch<TS, TB, true, 2 * k, 512>(a, s, st) : bwd_launch<TS, TB, false, 2 * k, 512>(a, s, st);
    }
    if (s.shift) GDN2_BWD(true)
    GDN2_BWD(false)
}
#undef GDN2_FWD
#undef GDN2_BWD
#undef GDN2_UP_TO

// CTAs of the backward: the workspace holds one row of partial sums for each, so
// the count goes by the sizes alone (148 SMs).
int bwd_grid(int rows, int D, int V) {
    const Split s = split_for(D, V, true);
    const int tier = s.threads > 256 && s.threads <= 320 ? 320 : s.threads > 128 && s.threads <= 192 ? 192 : 512;
    return grid_for(rows, s, tier * bwd_ctas(tier), 148);
}
int vector_of(gdn2_dtype stream_dt, gdn2_dtype dt) {
    return stream_dt == GDN2_BF16 ? vector_channels<bf16, bf16>()
           : dt == GDN2_BF16      ? vector_channels<float, bf16>()
                                  : vector_channels<float, float>();
}

}  // namespace

// Launched while the grid that writes `part` still runs (programmatic dependent launch):
// its CTAs wait for that grid's end before they read.
cudaError_t launch_reduce_parts(const float *part, int G, int W, int D0, float *out0, float *out1, cudaStream_t st) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((W + 31) / 32);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, reduce_parts_kernel, part, G, W, D0, out0, out1);
}

cudaError_t launch_residual_norm(const void *x, const void *r, const float *weight, const float *scale, double p,
                                 const unsigned long long *rng, float eps, void *h, void *y, float *rstd, int rows,
                                 int D, gdn2_dtype stream_dt, gdn2_dtype dt, cudaStream_t st) {
    const Dropout dp{p > 0.0 && r ? rng : nullptr, (uint32_t)(p * 4294967296.0), (float)(1.0 / (1.0 - p))};
    const FwdArgs a{x, r, weight, scale, dp, eps, h, y, rstd, rows, D};
    if (stream_dt == GDN2_BF16) return fwd_sized<bf16, bf16>(a, st);
    return dt == GDN2_BF16 ? fwd_sized<float, bf16>(a, st) : fwd_sized<float, float>(a, st);
}

size_t residual_norm_bwd_workspace_bytes(int rows, int D) {       // whatever the types
    const int a = bwd_grid(rows, D, 4), b = bwd_grid(rows, D, 8);
    return (size_t)(a > b ? a : b) * 2 * D * sizeof(float);
}

cudaError_t launch_residual_norm_bwd(const void *dy, const void *h, const float *rstd, const float *weight,
                                     const void *dh, const void *r, const float *scale, double p,
                                     const unsigned long long *rng, void *dx, void *dr, float *dweight, float *dscale,
                                     float *workspace, int rows, int D, gdn2_dtype stream_dt, gdn2_dtype dt,
                                     cudaStream_t st) {
    const Dropout dp{p > 0.0 ? rng : nullptr, (uint32_t)(p * 4294967296.0), (float)(1.0 / (1.0 - p))};
    const int grid = bwd_grid(rows, D, vector_of(stream_dt, dt));
    const bool direct = grid == 1 && !dscale;          // one CTA's sums are the result
    const BwdArgs a{dy, h, rstd, weight, dh, dscale ? r : nullptr, scale, dp, dx, dr, direct ? dweight : workspace, rows, D, grid};
    const cudaError_t e = stream_dt == GDN2_BF16 ? bwd_sized<bf16, bf16>(a, st)
                          : dt == GDN2_BF16      ? bwd_sized<float, bf16>(a, st)
                                                 : bwd_sized<float, float>(a, st);
    if (e != cudaSuccess || direct) return e;
    return launch_reduce_parts(workspace, grid, dscale ? 2 * D : D, D, dweight, dscale, st);
}

}  // namespace gdn2
