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
// Work: an item is one (sequence, head), a unit up to four tokens of it.  A CTA takes
// items a grid apart and works through their units as a pipeline, with one barrier a
// unit, so that no latency but the state's arrival is left between two of them:
//   A  the unit's state, copied to shared memory asynchronously while the item before
//      ran, goes to registers, and the next item's copies start;
//   B  the unit's tokens, one after the other (below); the state after the last kept
//      token is stored;
//   C  the next unit's tokens are prepared (activations, norms, gates, products) by four
//      warps, one token each, from copies that started two units ago;
//   D  barrier;  E  the unit's outputs go through the epilogue, by the other warps.
// One thread plans three units ahead; what it needs of a sequence comes by asynchronous
// copies as well.
//
// Mapping: the columns of a state evolve independently, so a warp owns 16 of them with
// all rows: lane = (row group of 8, column quad of 4), a lane holds d_k / 8 rows x 4
// columns, and a 16-byte access takes 64 contiguous bytes of each of eight rows.  A
// token then needs no barrier: its two column sums (Sbar^T (b k) and Sbar^T q) are added
// over the eight row groups by seven shuffles that halve the number of sums at each step.
// Rows are paired in 64-bit registers for the packed FP32 multiply-adds of sm_100, which
// halves their issue slots.
//
// Measured on a B200, 16 heads of 128 x 128, BF16: one token of 256 sequences 98 us = 5.57
// TB/s (86 % of a copy's rate; 1,024 sequences 370 us = 5.92 TB/s), the same from logits with
// the epilogue 97 us; a CTA per item, each load waiting for the one before, took 104 and
// 125 us.  1 to 8 tokens of 48 sequences 28.5 us, 1 to 16 of 64 51 us: bound there by the
// tokens' vectors from shared memory and the chain of shuffles, 16 warps an SM.
#include <type_traits>

#include "async_copy.cuh"
#include "f32x2.cuh"
#include "layer.cuh"

namespace gdn2 {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kTile = 4;                  // tokens of a unit
constexpr int kPlan = 8;                  // units in the plan's ring

__device__ unsigned int g_slot_conflict = 0;   // nonzero: a slot was named by two sequences, one of them writing it

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// N (2 or 4) consecutive channels of a token's vector, from shared memory
template <int N> __device__ __forceinline__ void load_n(const float *p, float (&v)[N]) {
    if (N == 4) {
        const float4 r = *reinterpret_cast<const float4 *>(p);
        v[0] = r.x; v[1] = r.y; v[N - 2] = r.z; v[N - 1] = r.w;
    } else {
        const float2 r = *reinterpret_cast<const float2 *>(p);
        v[0] = r.x; v[1] = r.y;
    }
}
template <int N> __device__ __forceinline__ void load_n(const bf16 *p, float (&v)[N]) {
    if (N == 4) {
        const uint2 r = *reinterpret_cast<const uint2 *>(p);
        v[0] = __uint_as_float(r.x << 16); v[1] = __uint_as_float(r.x & 0xFFFF0000u);
        v[N - 2] = __uint_as_float(r.y << 16); v[N - 1] = __uint_as_float(r.y & 0xFFFF0000u);
    } else {
        const uint32_t r = *reinterpret_cast<const uint32_t *>(p);
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

// A sequence's entries as they stand in memory, and what they mean.
struct Entry { int slot, t0, t1, keep; };

// A unit: tokens [row, row + count) of sequence `seq`, head `head`; `keep`: how many of them,
// and of those after them, the stored state takes in; count 0: no more units.
struct __align__(16) Unit { int row, count, head, slot, keep, first, seq, unused; };

// The planning thread's own words in shared memory: the item in hand; the next round of
// items, its sequence (-1: there is none) and head; the entries of the first rounds, and
// of a later one where it was `sent` for.
constexpr int kEarly = 4;
struct Plan { int seq, head, t1, slot, keep, base, round, next_seq, next_head, sent, unused[2]; Entry early[kEarly], entry; };

template <typename TIn, int DK, int DV, bool LOGITS> struct Shape {
    using TG = typename std::conditional<LOGITS, bf16, float>::type;
    static constexpr int THREADS = DV * 2, WARPS = THREADS / 32, PAIRS = DK / 16, CK = DK / 32, CV = DV / 32;
    static_assert(WARPS >= kTile, "a warp for each token of a unit");
    // a lane's bytes of one token, as they come: q, k, alpha, b, v, w
    static constexpr int BK = CK * (int)sizeof(TIn), GK = CK * (int)sizeof(TG), BV = CV * (int)sizeof(TIn),
                         GV = CV * (int)sizeof(TG), RAW = 2 * BK + 2 * GK + BV + GV;
    // shared memory; what units share comes twice, by the unit's parity
    static constexpr int VEC = kTile * DK * 8, ROW = kTile * DV * 4, GATES = kTile * 32 * BV;
    static constexpr int STATE = 0, AE = STATE + DK * DV * 4, QK = AE + 2 * VEC, Z = QK + 2 * VEC, O = Z + 2 * ROW,
                         GATE = O + 2 * ROW, RAWS = GATE + 2 * GATES, KQ = RAWS + kTile * 32 * RAW,
                         UNITS = KQ + 2 * kTile * 4, PLAN = UNITS + kPlan * (int)sizeof(Unit),
                         ORDER = PLAN + (int)sizeof(Plan), BYTES = ORDER + 2 * THREADS;
    static constexpr int CTAS = DV == 128 ? 2 : DK == 128 ? 3 : 4;      // an SM holds, by registers and shared memory
};

__device__ __forceinline__ Entry clamped(const StepArgs &a, int seq, Entry e) {
    if (a.cu) {
        e.t0 = min(max(e.t0, 0), a.T);
        e.t1 = min(max(e.t1, e.t0), a.T);
    } else {
        e.t0 = seq;
        e.t1 = seq + 1;
    }
    e.keep = a.keep ? min(max(e.keep, 0), e.t1 - e.t0) : e.t1 - e.t0;
    return e;
}
__device__ __forceinline__ Entry load_entry(const StepArgs &a, int seq) {
    Entry e{__ldg(a.slots + seq), 0, 0, 0};
    if (a.cu) {
        e.t0 = __ldg(a.cu + seq);
        e.t1 = __ldg(a.cu + seq + 1);
    }
    if (a.keep) e.keep = __ldg(a.keep + seq);
    return clamped(a, seq, e);
}

// The sequence of this CTA's item of a round (-1: none) and its head.  Items are sequences x
// heads, the sequences in the order of `order` where there is one; every other round then
// goes through the CTAs backwards.
__device__ __forceinline__ int item_of(const StepArgs &a, const unsigned short *order, int round, int &head) {
    const int grid = gridDim.x, b = blockIdx.x;
    const long long at = (long long)round * grid + (order && round & 1 ? grid - 1 - b : b);
    if (at >= (long long)a.N * a.H) return -1;
    const int seq = (int)at / a.H;
    head = (int)at - seq * a.H;
    return order ? order[seq] : seq;
}

// The next unit of this CTA, by one thread.  `ahead`: send for the entry after it.
__device__ __forceinline__ void plan_unit(const StepArgs &a, const unsigned short *order, Plan &p, Unit &u, bool ahead) {
    bool first = false;
    if (p.base + kTile < p.t1) {
        p.base += kTile;
        p.keep -= kTile;
    } else {
        Entry e{-1, 0, 0, 0};
        while (p.next_seq >= 0) {              // past items without tokens
            e = p.round < kEarly ? p.early[p.round] : p.sent ? clamped(a, p.next_seq, p.entry) : load_entry(a, p.next_seq);
            p.seq = p.next_seq;
            p.head = p.next_head;
            p.sent = 0;
            p.next_seq = item_of(a, order, ++p.round, p.next_head);
            if (e.t0 < e.t1) break;
        }
        p.base = e.t0;
        p.t1 = e.t1;
        p.slot = e.slot;
        p.keep = e.keep;
        first = true;
    }
    if (ahead && !p.sent && p.next_seq >= 0 && p.round >= kEarly) {
        copy_async<4>(smem_address(&p.entry.slot), a.slots + p.next_seq);
        if (a.cu) {
            copy_async<4>(smem_address(&p.entry.t0), a.cu + p.next_seq);
            copy_async<4>(smem_address(&p.entry.t1), a.cu + p.next_seq + 1);
        }
        if (a.keep) copy_async<4>(smem_address(&p.entry.keep), a.keep + p.next_seq);
        p.sent = 1;
    }
    u = Unit{p.base, min(kTile, p.t1 - p.base), p.head, p.slot, p.keep, first, p.seq, 0};
}

template <typename TIn, int DK, int DV, bool LOGITS>
__global__ void __launch_bounds__(DV * 2, Shape<TIn, DK, DV, LOGITS>::CTAS)
slot_steps_kernel(const __grid_constant__ StepArgs a) {
    using X = Shape<TIn, DK, DV, LOGITS>;
    using TG = typename X::TG;
    constexpr int THREADS = X::THREADS, WARPS = X::WARPS, PAIRS = X::PAIRS, CK = X::CK, CV = X::CV;
    extern __shared__ __align__(16) unsigned char sm[];
    Unit *units = reinterpret_cast<Unit *>(sm + X::UNITS);
    Plan &plan = *reinterpret_cast<Plan *>(sm + X::PLAN);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rg = lane >> 2, col = warp * 16 + (lane & 3) * 4;
    const int late = (warp + WARPS / 2) % WARPS;           // the token whose output this warp finishes
    const bool planner = tid == THREADS - 1;
    const uint32_t state_at = smem_address(sm + X::STATE) + tid * 16;

    // Asynchronous copies of what this thread itself reads later: its part of a state, its
    // lane's channels of the token that its warp prepares and of the gate that it applies.
    auto fetch_state = [&](const Unit &u) {
        if (!u.first || u.count <= 0 || u.slot < 0 || u.slot >= a.n_slots) return;
        const float *p = a.pool + ((size_t)u.slot * a.H + u.head) * (DK * DV) + (size_t)(2 * rg) * DV + col;
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) {
            copy_async<16>(state_at + (2 * j) * THREADS * 16, p + 16 * j * DV);
            copy_async<16>(state_at + (2 * j + 1) * THREADS * 16, p + (16 * j + 1) * DV);
        }
    };
    auto fetch_token = [&](const Unit &u) {
        if (warp >= u.count) return;
        const size_t row = (size_t)(u.row + warp) * a.H + u.head, ok = row * DK + lane * CK, ov = row * DV + lane * CV;
        uint32_t at = smem_address(sm + X::RAWS) + warp * 32 * X::RAW;
        copy_async<X::BK>(at + lane * X::BK, static_cast<const TIn *>(a.q) + ok);
        copy_async<X::BK>((at += 32 * X::BK) + lane * X::BK, static_cast<const TIn *>(a.k) + ok);
        copy_async<X::GK>((at += 32 * X::BK) + lane * X::GK, static_cast<const TG *>(a.alpha) + ok);
        copy_async<X::GK>((at += 32 * X::GK) + lane * X::GK, static_cast<const TG *>(a.b) + ok);
        copy_async<X::BV>((at += 32 * X::GK) + lane * X::BV, static_cast<const TIn *>(a.v) + ov);
        copy_async<X::GV>((at += 32 * X::BV) + lane * X::GV, static_cast<const TG *>(a.w) + ov);
    };
    auto fetch_gate = [&](const Unit &u, int parity) {
        if (!a.gate || late >= u.count) return;
        copy_async<X::BV>(smem_address(sm + X::GATE) + parity * X::GATES + (late * 32 + lane) * X::BV,
                          static_cast<const TIn *>(a.gate) + ((size_t)(u.row + late) * a.H + u.head) * DV + lane * CV);
    };
    // The token that this warp prepares, from its copies to the vectors that B reads.
    auto prepare = [&](const Unit &u, int parity) {
        if (warp >= u.count) return;
        const unsigned char *raw = sm + X::RAWS + warp * 32 * X::RAW;
        float q[CK], k[CK], al[CK], b[CK], v[CV], w[CV];
        load_n<CK>(reinterpret_cast<const TIn *>(raw + lane * X::BK), q);
        load_n<CK>(reinterpret_cast<const TIn *>((raw += 32 * X::BK) + lane * X::BK), k);
        load_n<CK>(reinterpret_cast<const TG *>((raw += 32 * X::BK) + lane * X::GK), al);
        load_n<CK>(reinterpret_cast<const TG *>((raw += 32 * X::GK) + lane * X::GK), b);
        load_n<CV>(reinterpret_cast<const TIn *>((raw += 32 * X::GK) + lane * X::BV), v);
        load_n<CV>(reinterpret_cast<const TG *>((raw += 32 * X::BV) + lane * X::GV), w);
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
        if (lane == 0) reinterpret_cast<float *>(sm + X::KQ)[parity * kTile + warp] = kq;
        // per row pair: (alpha, alpha', e, e') and (q, q', k, k')
        float4 *ae = reinterpret_cast<float4 *>(sm + X::AE + parity * X::VEC) + warp * (DK / 2);
        float4 *qk = reinterpret_cast<float4 *>(sm + X::QK + parity * X::VEC) + warp * (DK / 2);
#pragma unroll
        for (int e = 0; e < CK; e += 2) {
            ae[(lane * CK + e) / 2] = make_float4(al[e], al[e + 1], b[e] * k[e], b[e + 1] * k[e + 1]);
            qk[(lane * CK + e) / 2] = make_float4(q[e], q[e + 1], k[e], k[e + 1]);
        }
        float *z = reinterpret_cast<float *>(sm + X::Z + parity * X::ROW) + warp * DV;
#pragma unroll
        for (int e = 0; e < CV; ++e) z[lane * CV + e] = w[e] * v[e];
    };
    // Two sequences that name one slot would race if either writes it: both are refused.  Every
    // item's slot is compared with all others', the first of them kept in a register, the rest
    // read four at a time.
    const int near = tid < a.N ? __ldg(a.slots + tid) : -1;
    const bool by_four = (reinterpret_cast<uintptr_t>(a.slots) & 15) == 0;
    auto clashes = [&](const Unit &u) {
        if (!u.first || u.count <= 0 || u.slot < 0 || u.slot >= a.n_slots) return false;
        bool clash = false;
        auto compare = [&](int m, int slot) {
            if (slot != u.slot || m == u.seq) return;
            const Entry other = load_entry(a, m);
            clash |= other.t0 < other.t1 && (u.keep > 0 || other.keep > 0);
        };
        compare(tid, near);
        int done = THREADS;
        if (by_four && a.N > THREADS) {
            const int4 *four = reinterpret_cast<const int4 *>(a.slots);
#pragma unroll 4
            for (int m = THREADS / 4 + tid; m < a.N / 4; m += THREADS) {
                const int4 v = __ldg(four + m);
                if (v.x == u.slot || v.y == u.slot || v.z == u.slot || v.w == u.slot) {
                    compare(4 * m, v.x);
                    compare(4 * m + 1, v.y);
                    compare(4 * m + 2, v.z);
                    compare(4 * m + 3, v.w);
                }
            }
            done = a.N / 4 * 4;
        }
        for (int m = done + tid; m < a.N; m += THREADS) compare(m, __ldg(a.slots + m));
        return clash;
    };

    // Where sequences have different lengths and a CTA gets few of them, they are taken from the
    // longest to the shortest, there and back, so that the CTAs' sums of tokens are alike.
    const unsigned short *order = nullptr;
    if (a.cu && a.N <= THREADS && a.N * a.H > (int)gridDim.x) {
        unsigned short *by_length = reinterpret_cast<unsigned short *>(sm + X::ORDER);
        int *lengths = reinterpret_cast<int *>(sm + X::AE);         // free until the first token is prepared
        int mine = 0;
        if (tid < a.N) {
            const Entry e = load_entry(a, tid);
            lengths[tid] = mine = e.t1 - e.t0;
        }
        __syncthreads();
        if (tid < a.N) {
            int rank = 0;
            for (int m = 0; m < a.N; ++m) rank += lengths[m] > mine || (lengths[m] == mine && m < tid);
            by_length[rank] = (unsigned short)tid;
        }
        __syncthreads();
        order = by_length;
    }
    if (warp == WARPS - 1) {
        if (lane < kEarly) {
            int head;
            const int seq = item_of(a, order, lane, head);
            plan.early[lane] = seq >= 0 ? load_entry(a, seq) : Entry{-1, 0, 0, 0};
        }
        __syncwarp();
        if (planner) {
            plan.base = plan.t1 = plan.round = plan.sent = 0;
            plan.next_seq = item_of(a, order, 0, plan.next_head);
            plan_unit(a, order, plan, units[0], false);
        }
    }
    __syncthreads();
    bool dead;                                 // the item has no state: its outputs are zero
    {
        const Unit u = units[0];
        fetch_token(u);
        fetch_gate(u, 0);
        copy_commit();
        fetch_state(u);
        copy_commit();
        if (planner) {
            plan_unit(a, order, plan, units[1], false);
            plan_unit(a, order, plan, units[2], false);
        }
        const bool clash = clashes(u);
        copy_wait<1>();
        prepare(u, 0);
        dead = __syncthreads_or(clash);
        fetch_token(units[1]);
        copy_commit();
        if (dead && planner) atomicOr(&g_slot_conflict, 1u);
    }

    Pair S[PAIRS][4];                          // rows 2m and 2m + 1 for m = rg + 8 j, four columns each
    for (int n = 0;; ++n) {
        const int parity = n & 1;
        const int count = units[n % kPlan].count;
        if (count <= 0) break;

        // A
        copy_wait<1>();                        // all but the next unit's tokens
        if (units[n % kPlan].first) {
            const int slot = units[n % kPlan].slot;
            dead |= slot < 0 || slot >= a.n_slots;
            if (!dead) {
#pragma unroll
                for (int j = 0; j < PAIRS; ++j) {
                    uint4 x, y;
                    load_shared(state_at + (2 * j) * THREADS * 16, x);
                    load_shared(state_at + (2 * j + 1) * THREADS * 16, y);
                    S[j][0] = pack2(__uint_as_float(x.x), __uint_as_float(y.x));
                    S[j][1] = pack2(__uint_as_float(x.y), __uint_as_float(y.y));
                    S[j][2] = pack2(__uint_as_float(x.z), __uint_as_float(y.z));
                    S[j][3] = pack2(__uint_as_float(x.w), __uint_as_float(y.w));
                }
            }
        }
        if (planner) plan_unit(a, order, plan, units[(n + 3) % kPlan], true);
        fetch_state(units[(n + 1) % kPlan]);
        copy_commit();

        // B
        if (!dead) {
            const float4 *s_ae = reinterpret_cast<const float4 *>(sm + X::AE + parity * X::VEC) + rg;
            const float4 *s_qk = reinterpret_cast<const float4 *>(sm + X::QK + parity * X::VEC) + rg;
            const float *s_z = reinterpret_cast<const float *>(sm + X::Z + parity * X::ROW);
            const float *s_kq = reinterpret_cast<const float *>(sm + X::KQ) + parity * kTile;
            float *s_o = reinterpret_cast<float *>(sm + X::O + parity * X::ROW);
            const bool up = lane & 16, b3 = lane & 8, b2 = lane & 4;
            const int c_own = col + (b3 ? 2 : 0) + (b2 ? 1 : 0);
            const int last = units[n % kPlan].keep - 1;
#pragma unroll 1                               // unrolled, or two tokens to a pass over the state: spills, a tenth slower
            for (int i = 0; i < count; ++i) {
                Pair r[4], p[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) r[c].v = p[c].v = 0ull;
#pragma unroll
                for (int j = 0; j < PAIRS; ++j) {
                    const float4 ae = s_ae[i * (DK / 2) + 8 * j], qk = s_qk[i * (DK / 2) + 8 * j];
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
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float r0, r1, p0, p1;
                    unpack2(r[c], r0, r1);
                    unpack2(p[c], p0, p1);
                    r0 += r1;
                    p0 += p1;
                    x[c] = (up ? p0 : r0) + __shfl_xor_sync(0xffffffffu, up ? r0 : p0, 16);
                }
                const float y0 = (b3 ? x[2] : x[0]) + __shfl_xor_sync(0xffffffffu, b3 ? x[0] : x[2], 8);
                const float y1 = (b3 ? x[3] : x[1]) + __shfl_xor_sync(0xffffffffu, b3 ? x[1] : x[3], 8);
                const float mine = (b2 ? y1 : y0) + __shfl_xor_sync(0xffffffffu, b2 ? y0 : y1, 4);
                const float other = __shfl_xor_sync(0xffffffffu, mine, 16);
                const float u = s_z[i * DV + c_own] - (up ? other : mine);
                const float out = fmaf(s_kq[i], u, mine);
                Pair u2[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float uc = __shfl_sync(0xffffffffu, u, (lane & 3) | (c & 1) << 2 | (c & 2) << 2);
                    u2[c] = pack2(uc, uc);
                }
#pragma unroll
                for (int j = 0; j < PAIRS; ++j) {
                    const float2 kk = reinterpret_cast<const float2 *>(s_qk + i * (DK / 2) + 8 * j)[1];
                    const Pair k = pack2(kk.x, kk.y);
#pragma unroll
                    for (int c = 0; c < 4; ++c) S[j][c] = fma2(k, u2[c], S[j][c]);
                }
                if (up) s_o[i * DV + c_own] = out;
                if (i == last) {
                    float *to = a.pool + ((size_t)units[n % kPlan].slot * a.H + units[n % kPlan].head) * (DK * DV) +
                                (size_t)(2 * rg) * DV + col;
#pragma unroll
                    for (int j = 0; j < PAIRS; ++j) {
                        float4 r0, r1;
                        unpack2(S[j][0], r0.x, r1.x); unpack2(S[j][1], r0.y, r1.y);
                        unpack2(S[j][2], r0.z, r1.z); unpack2(S[j][3], r0.w, r1.w);
                        __stcs(reinterpret_cast<float4 *>(to + 16 * j * DV), r0);
                        __stcs(reinterpret_cast<float4 *>(to + (16 * j + 1) * DV), r1);
                    }
                }
            }
        }

        // C
        copy_wait<1>();                        // all but the next item's state
        prepare(units[(n + 1) % kPlan], parity ^ 1);
        fetch_token(units[(n + 2) % kPlan]);
        fetch_gate(units[(n + 1) % kPlan], parity ^ 1);
        copy_commit();
        const bool clash = clashes(units[(n + 1) % kPlan]);

        // D
        const bool next_dead = __syncthreads_or(clash);

        // E
        if (late < count) {
            const Unit &u = units[n % kPlan];
            const size_t ov = ((size_t)(u.row + late) * a.H + u.head) * DV + lane * CV;
            float x[CV];
            load_n<CV>(reinterpret_cast<const float *>(sm + X::O + parity * X::ROW) + late * DV + lane * CV, x);
            if (a.gate) {
                float gv[CV], ss = 0.f;
                load_n<CV>(reinterpret_cast<const TIn *>(sm + X::GATE + parity * X::GATES + (late * 32 + lane) * X::BV), gv);
#pragma unroll
                for (int e = 0; e < CV; ++e) ss = fmaf(x[e], x[e], ss);
                const float rs = rsqrtf(warp_sum(ss) * (1.f / DV) + a.eps);
#pragma unroll
                for (int e = 0; e < CV; ++e) x[e] = x[e] * rs * __ldg(a.weight + lane * CV + e) * sigmoid(gv[e]);
            }
            if (dead) {
#pragma unroll
                for (int e = 0; e < CV; ++e) x[e] = 0.f;
            }
            store_n<CV>(static_cast<TIn *>(a.o) + ov, x);
        }
        if (units[(n + 1) % kPlan].first) {
            dead = next_dead;
            if (dead && planner) atomicOr(&g_slot_conflict, 1u);
        }
    }
}

template <typename TIn, int DK, int DV, bool LOGITS> cudaError_t launch_typed(const StepArgs &a, cudaStream_t st) {
    using X = Shape<TIn, DK, DV, LOGITS>;
    int dev = 0, sms = 148;
    static std::atomic<unsigned long long> allowed{0};
    cudaError_t e = device_sms(&dev, &sms);
    if (e == cudaSuccess) e = allow_shared(slot_steps_kernel<TIn, DK, DV, LOGITS>, X::BYTES, dev, allowed);
    if (e != cudaSuccess) return e;
    const int items = a.N * a.H, cap = sms * X::CTAS;
    slot_steps_kernel<TIn, DK, DV, LOGITS><<<items < cap ? items : cap, X::THREADS, X::BYTES, st>>>(a);
    return cudaGetLastError();
}

template <typename TIn, bool LOGITS> cudaError_t launch_dims(const StepArgs &a, int dk, int dv, cudaStream_t st) {
    if (dk == 128) return dv == 128 ? launch_typed<TIn, 128, 128, LOGITS>(a, st) : launch_typed<TIn, 128, 64, LOGITS>(a, st);
    return dv == 128 ? launch_typed<TIn, 64, 128, LOGITS>(a, st) : launch_typed<TIn, 64, 64, LOGITS>(a, st);
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
