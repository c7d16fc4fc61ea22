// gated_scan.cuh -- the gated linear recurrence over whole sequences.
//
//   u_t = rate * sigmoid(g_t + bias),  h_t = h_{t-1} + u_t (x_t - h_{t-1}),
//   out_t = h_t silu(z_t)
#pragma once

#include "device_utils.cuh"
#include "jamba_ssm_gated.h"
#include "s6_math.cuh"

namespace jssm {

constexpr int kGatedCkpt = JAMBA_SSM_GATED_CKPT_STEPS;

struct GatedArgs {
    const void *x, *g, *z;
    int64_t xs, gs, zs;  // row strides in elements
    const float *rate, *bias, *h0;
    void *out;
    float *h_final;
    const int32_t *cu;
    int64_t total;  // token rows
    const int32_t *state_indices, *initial_indices;
    int64_t num_slots;
    float *ckpt;
    int *status;
    int64_t seqlen;
    int d, batch;
    // backward
    const void *dout;
    const float *dh_final;
    void *dx, *dg, *dz;
    float *drate, *dbias, *dh0;
    float *partial;  // [batch][2][d]
};

// Rows of sequence b.
__device__ __forceinline__ void gated_rows(const GatedArgs &a, int b, int64_t &row0, int64_t &len) {
    if (a.cu) {
        const int64_t lo = min(max(int64_t(a.cu[b]), int64_t(0)), a.total);
        const int64_t hi = min(max(int64_t(a.cu[b + 1]), int64_t(0)), a.total);
        row0 = lo;
        len = max(hi - lo, int64_t(0));
    } else {
        row0 = int64_t(b) * a.seqlen;
        len = a.seqlen;
    }
}

__device__ __forceinline__ float sigmoid_f32(float v) {
    return rcp_mufu(1.0f + ex2_mufu(-v * kLog2e));
}

// Cache row of an index (-1: none); one past the cache is recorded by `report`.
__device__ __forceinline__ int64_t gated_slot(const GatedArgs &a, int idx, bool report) {
    if (idx < 0) return -1;
    if (idx >= a.num_slots) {
        if (report) record_status(a.status, kStInvalidArg);
        return -1;
    }
    return idx;
}

// ------------------------------------------------------------ lanes and pairs
// A lane holds 4 bytes of a row: two neighbouring bf16 channels or one fp32
// channel (one bf16 channel where the width, a stride or a pointer is odd), so
// a warp reads 128 (64) contiguous bytes of one row with one instruction.  Two
// channels are computed with one packed fp32 instruction each.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
    return bits_f2(r);
}
template <int VEC> struct Lane;
template <> struct Lane<1> {
    float v;
    __device__ __forceinline__ static Lane of(float a) { return {a}; }
    __device__ __forceinline__ float get(int) const { return v; }
    __device__ __forceinline__ void set(int, float a) { v = a; }
};
template <> struct Lane<2> {
    float2 v;
    __device__ __forceinline__ static Lane of(float a) { return {make_float2(a, a)}; }
    __device__ __forceinline__ float get(int i) const { return i ? v.y : v.x; }
    __device__ __forceinline__ void set(int i, float a) { (i ? v.y : v.x) = a; }
};
using Lane1 = Lane<1>;
using Lane2 = Lane<2>;
__device__ __forceinline__ Lane1 lfma(Lane1 a, Lane1 b, Lane1 c) { return {fmaf(a.v, b.v, c.v)}; }
__device__ __forceinline__ Lane1 lmul(Lane1 a, Lane1 b) { return {a.v * b.v}; }
__device__ __forceinline__ Lane1 ladd(Lane1 a, Lane1 b) { return {a.v + b.v}; }
__device__ __forceinline__ Lane1 lsub(Lane1 a, Lane1 b) { return {a.v - b.v}; }
__device__ __forceinline__ Lane1 lex2(Lane1 a) { return {ex2_mufu(a.v)}; }
__device__ __forceinline__ Lane1 lrcp(Lane1 a) { return {rcp_mufu(a.v)}; }
__device__ __forceinline__ Lane2 lfma(Lane2 a, Lane2 b, Lane2 c) { return {fma2(a.v, b.v, c.v)}; }
__device__ __forceinline__ Lane2 lmul(Lane2 a, Lane2 b) { return {mul2(a.v, b.v)}; }
__device__ __forceinline__ Lane2 ladd(Lane2 a, Lane2 b) { return {add2(a.v, b.v)}; }
// a - b as one packed instruction: b * -1 is exact
__device__ __forceinline__ Lane2 lsub(Lane2 a, Lane2 b) {
    return {fma2(b.v, make_float2(-1.0f, -1.0f), a.v)};
}
__device__ __forceinline__ Lane2 lex2(Lane2 a) { return {make_float2(ex2_mufu(a.v.x), ex2_mufu(a.v.y))}; }
__device__ __forceinline__ Lane2 lrcp(Lane2 a) { return {make_float2(rcp_mufu(a.v.x), rcp_mufu(a.v.y))}; }
template <int VEC> __device__ __forceinline__ Lane<VEC> lsigmoid(Lane<VEC> v) {
    return lrcp(ladd(lex2(lmul(v, Lane<VEC>::of(-kLog2e))), Lane<VEC>::of(1.0f)));
}

// Two sigmoids with one reciprocal: with p = 1 + e^-v0 and q = 1 + e^-v1,
// r = 1 / (p q) gives r q and r p.  The special-function pipe, at 4 lanes a
// cycle and scheduler, is the scan's narrowest: this takes 3 of its operations
// a pair instead of 4.  Where p q leaves the range (v0 + v1 below about -87) or
// an input is a NaN, r is not above 0: `good` is cleared, and the lane does its
// run again with lsigmoid (each lane for itself: a result must not depend on
// what the other lanes hold).
__device__ __forceinline__ Lane2 lsigmoid_pair(Lane2 v, bool &good) {
    const Lane2 t = lmul(v, Lane2::of(-kLog2e));
    const Lane2 qp = ladd(Lane2{make_float2(ex2_mufu(t.v.y), ex2_mufu(t.v.x))}, Lane2::of(1.0f));
    const float r = rcp_mufu(qp.v.x * qp.v.y);
    good = good && r > 0.0f;
    return lmul(qp, Lane2::of(r));
}
__device__ __forceinline__ Lane1 lsigmoid_pair(Lane1 v, bool &) { return lsigmoid(v); }

template <typename T, int VEC> struct GatedRaw;
template <> struct GatedRaw<float, 1> {
    using type = float;
    static __device__ __forceinline__ Lane1 get(type r) { return {r}; }
    static __device__ __forceinline__ type put(Lane1 v) { return v.v; }
};
template <> struct GatedRaw<__nv_bfloat16, 1> {
    using type = uint16_t;
    static __device__ __forceinline__ Lane1 get(type r) { return {__uint_as_float(uint32_t(r) << 16)}; }
    static __device__ __forceinline__ type put(Lane1 v) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(v.v));
    }
};
template <> struct GatedRaw<__nv_bfloat16, 2> {
    using type = uint32_t;
    static __device__ __forceinline__ Lane2 get(type r) {
        return {make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u))};
    }
    static __device__ __forceinline__ type put(Lane2 v) {
        __nv_bfloat162 h = __floats2bfloat162_rn(v.v.x, v.v.y);
        return *reinterpret_cast<uint32_t *>(&h);
    }
};

// ---------------------------------------------------------- the maps of runs
// A run of rows takes the state h to P h + b with P = prod(1 - u).  P in fp32 has
// an error of 2^-25 a row, which is nothing beside a decay that shows in a run,
// but adds up over a long sequence where hardly anything decays: with u = 5e-7 it
// is 5% of u, and a state that should stay at its input drifts by 2e-8 of it a row
// (4e-4 in 16384 rows).  So a run also sums what it loses, n = P - 1 = -sum(u P
// before the row), and its decay is held as q: n where P > 7/8, P where not, told
// apart by the sign (P is not negative: u is at most 1, but for its rounding).
// h + (n h + b) then rounds once, to the state's own last place.  The most runs that
// are joined to one map, 32, leave n above -0.99, so a decay of many slow runs keeps
// all but the last bits of P.  This takes an FMA a row and two operations a map more:
// 4096 x 8192 bf16 59 us for 57, 2 x 4096 x 4096 with the backward 169 for 162.
constexpr float kHeld = -1e-30f;  // the q of no decay
// 1 where q is P - 1
__device__ __forceinline__ float held_f32(float q) { return q < 0.0f ? 1.0f : 0.0f; }
__device__ __forceinline__ Lane1 lheld(Lane1 q) { return {held_f32(q.v)}; }
__device__ __forceinline__ Lane2 lheld(Lane2 q) { return {make_float2(held_f32(q.v.x), held_f32(q.v.y))}; }
__device__ __forceinline__ float decay_f32(float P, float n) {
    return P > 0.875f ? fminf(n, kHeld) : fmaxf(P, 0.0f);
}
__device__ __forceinline__ Lane1 ldecay(Lane1 P, Lane1 n) { return {decay_f32(P.v, n.v)}; }
__device__ __forceinline__ Lane2 ldecay(Lane2 P, Lane2 n) {
    return {make_float2(decay_f32(P.v.x, n.v.x), decay_f32(P.v.y, n.v.y))};
}
// The map (q, b) of h, and the decay of q1 and then q2 (either order).
template <int VEC> __device__ __forceinline__ Lane<VEC> lapply(Lane<VEC> q, Lane<VEC> h, Lane<VEC> b) {
    return lfma(lheld(q), h, lfma(q, h, b));
}
template <int VEC> __device__ __forceinline__ Lane<VEC> ljoin(Lane<VEC> q2, Lane<VEC> q1) {
    return lfma(q2, q1, lfma(q2, lheld(q1), lmul(q1, lheld(q2))));
}

// A map for a lane's channels, as it lies in shared memory.
template <int VEC> struct RunMap;
template <> struct RunMap<1> {
    float2 v;
    __device__ __forceinline__ Lane1 q() const { return {v.x}; }
    __device__ __forceinline__ Lane1 b() const { return {v.y}; }
    __device__ __forceinline__ static RunMap of(Lane1 q, Lane1 b) { return {make_float2(q.v, b.v)}; }
};
template <> struct RunMap<2> {
    float4 v;
    __device__ __forceinline__ Lane2 q() const { return {make_float2(v.x, v.y)}; }
    __device__ __forceinline__ Lane2 b() const { return {make_float2(v.z, v.w)}; }
    __device__ __forceinline__ static RunMap of(Lane2 q, Lane2 b) {
        return {make_float4(q.v.x, q.v.y, b.v.x, b.v.y)};
    }
};

// ------------------------------------------------------------------ clusters
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Stores to `rank`'s shared memory at the address that `saddr` has in this CTA.
__device__ __forceinline__ void st_cluster(uint32_t saddr, uint32_t rank, RunMap<1> m) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(m.v.x), "f"(m.v.y) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t saddr, uint32_t rank, RunMap<2> m) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(m.v.x), "f"(m.v.y),
                 "f"(m.v.z), "f"(m.v.w)
                 : "memory");
}

// The sequence that a cluster takes.  Clusters start in the order of their
// number, so of packed sequences the longest goes first (of equal ones the
// first), or a long one among the last would run on alone.  Up to as many
// sequences as threads; more come in their order.  `order`: THREADS + 1 ints.
template <int THREADS> __device__ __forceinline__ int gated_sequence(const GatedArgs &a, int nth, int *order) {
    if (!a.cu || a.batch > THREADS || a.batch < 2) return nth;
    int len = 0;
    if (threadIdx.x < a.batch) {
        int64_t row0, len64;
        gated_rows(a, threadIdx.x, row0, len64);
        order[threadIdx.x] = len = static_cast<int>(len64);
    }
    __syncthreads();
    if (threadIdx.x < a.batch) {
        int before = 0;
        for (int j = 0; j < a.batch; ++j) {
            const int l = order[j];
            before += l > len || (l == len && j < int(threadIdx.x));
        }
        if (before == nth) order[THREADS] = threadIdx.x;
    }
    __syncthreads();
    return order[THREADS];
}

// ------------------------------------------------------------------- staging
template <int BYTES> __device__ __forceinline__ void cp(uint32_t dst, const void *src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One array's rows of one warp.  A warp's lanes hold Q runs of S rows side by
// side, 32 / Q lanes of a row each; slot i of a stage is row i of every run, so
// that lane l's word of it lies at l * 4 whatever Q is.  The lane keeps the
// address of the part that it copies; a round's copy moves it on.  CP: bytes of
// one copy, by the alignment of the rows: 16, 4, or one 2-byte element at a
// time through a register.  Rows from n on and channels past the width are not
// read, and their places in the stage hold what they held: no lane that stores
// anything uses them.
template <typename T, int VEC, int S, int Q, int CP> struct GatedFeed {
    static constexpr int kSlot = 32 * VEC * int(sizeof(T));   // bytes of a slot
    static constexpr int kPer = CP == 16 ? kSlot / 16 : 32;   // lanes of one slot
    static constexpr int kSlots = 32 / kPer;                  // slots of one instruction
    static constexpr int kLanes = kPer / Q;                   // lanes of one row
    const char *p;       // this lane's part of its first row
    int64_t hop, round;  // bytes from one instruction's rows to the next, from one round's to the next

    // This lane's first row and first channel in the warp's rows.
    static __device__ __forceinline__ int row_of(int lane) { return lane % kPer / kLanes * S + lane / kPer; }
    static __device__ __forceinline__ int channel_of(int lane) {
        return lane % kLanes * (kSlot / kPer / int(sizeof(T)));
    }
    __device__ __forceinline__ void start(const void *base, int64_t row, int64_t rs, int c0, int lane,
                                          int64_t stride) {
        p = static_cast<const char *>(base) +
            ((row + row_of(lane)) * rs + c0 + channel_of(lane)) * int64_t(sizeof(T));
        hop = kSlots * rs * int64_t(sizeof(T));
        round = stride * rs * int64_t(sizeof(T));
    }
    __device__ __forceinline__ void copy(uint32_t dst, bool in, int n, int lane) {
        const char *q = p;
        dst += lane * (kSlot / kPer);  // slot lane / kPer, part lane % kPer
        if constexpr (CP == 2) {
            uint16_t v[S];
#pragma unroll
            for (int i = 0; i < S; ++i) {
                v[i] = in && row_of(lane) + i < n ? *reinterpret_cast<const uint16_t *>(q) : uint16_t(0);
                q += hop;
            }
#pragma unroll
            for (int i = 0; i < S; ++i)
                asm volatile("st.shared.b16 [%0], %1;" ::"r"(dst + i * kSlot), "h"(v[i]) : "memory");
        } else {
            const int mine = in ? n - row_of(lane) : 0;  // rows from the lane's first on
            if (mine > (S / kSlots - 1) * kSlots) {
#pragma unroll
                for (int i = 0; i < S / kSlots; ++i) {
                    cp<CP>(dst + i * kSlots * kSlot, q);
                    q += hop;
                }
            } else {
#pragma unroll 1
                for (int i = 0; i * kSlots < mine; ++i) {
                    cp<CP>(dst + i * kSlots * kSlot, q);
                    q += hop;
                }
            }
        }
        p += round;
    }
    __device__ __forceinline__ void skip() { p += round; }
    // Where a lane finds row i of its run: behind first_word, in raw values.
    static __device__ __forceinline__ int first_word(int lane) { return lane; }
    __device__ __forceinline__ int word_of(int i) const { return i * 32; }
};

// The same where the rows begin at any multiple of 4 bytes (the array itself at 16):
// 16-byte copies of the aligned bytes that hold a row's part, which is then read
// from its place in them.  A lane copies the same part of every kRows-th row.  A run's
// rows lie together, the runs apart so that their lanes' words fall into different
// banks.  Bytes of neighbouring rows and channels come along unused; nothing before
// the array is read, and behind it a copy is cut short.  A row of 64 bytes takes 5 of
// an instruction's lanes in place of 16: 13 x 4096 x 1026 bf16 with z 125 us for 184.
constexpr int kCpShifted = 0;
template <typename T, int VEC, int S, int Q> struct GatedShiftedFeed {
    static constexpr int kRow = 128 / Q;              // bytes of a row
    static constexpr int kParts = kRow / 16 + 1;      // copies of a row
    static constexpr int kRows = 32 / kParts;         // rows of one instruction
    static constexpr int kPitch = kParts * 16;
    static constexpr int kRun = S * kPitch + kRow % 128;
    static constexpr int kBytes = Q * kRun;           // of an array's rows of one warp
    static constexpr int kCopies = (S * Q + kRows - 1) / kRows;
    static_assert(VEC * sizeof(T) == 4, "");
    const char *p, *end;  // this lane's first row and its part of it (not rounded down), the array's end
    const char *safe;  // from here on this lane's copies of a round may reach past the end
    int64_t hop, round;
    int word[4];  // of this lane in its run's rows i, i + 4, ...

    static __device__ __forceinline__ int channel_of(int) { return 0; }
    __device__ __forceinline__ void start(const void *base, int64_t row, int64_t rs, int c0, int lane,
                                          int64_t stride, int64_t total, int d) {
        constexpr int64_t es = sizeof(T);
        const char *const b = static_cast<const char *>(base);
        end = b + ((total - 1) * rs + d) * es;
        p = b + ((row + lane / kParts) * rs + c0) * es + lane % kParts * 16;
        hop = kRows * rs * es;
        round = stride * rs * es;
        safe = end - (kCopies - 1) * hop - 15;  // a copy ends at most 16 bytes behind its part's start
        const int run = lane / (32 / Q), col = lane % (32 / Q);
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // S and the strides are multiples of 4 rows
            const int64_t at = ((row + i) * rs + c0) * es;
            word[i] = run * (kRun / 4) + col + (static_cast<int>(at >> 2) & 3);
        }
    }
    __device__ __forceinline__ void copy(uint32_t dst, bool, int n, int lane) {
        const char *q = p;
        const int first = lane / kParts;
        dst += first * kPitch + lane % kParts * 16;
        const bool on = first < kRows;
        if (n == S * Q && p < safe) {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int r = first + i * kRows;
                if (on && r < S * Q) cp<16>(dst + i * (kRows * kPitch) + r / S * (kRun - S * kPitch), down(q));
                q += hop;
            }
        } else if (on) {
#pragma unroll 1
            for (int r = first; r < n; r += kRows) {
                const char *const from = down(q);
                const int64_t left = end - from;
                if (left > 0)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                     dst + (r - first) * kPitch + r / S * (kRun - S * kPitch)),
                                 "l"(from), "r"(static_cast<int>(min(left, int64_t(16))))
                                 : "memory");
                q += hop;
            }
        }
        p += round;
    }
    static __device__ __forceinline__ const char *down(const char *q) {
        return reinterpret_cast<const char *>(reinterpret_cast<uintptr_t>(q) & ~uintptr_t(15));
    }
    static __device__ __forceinline__ int first_word(int) { return 0; }
    __device__ __forceinline__ int word_of(int i) const { return word[i & 3] + i * (kPitch / 4); }
};
template <typename T, int VEC, int S, int Q, int CP> struct GatedFeedOf {
    using type = GatedFeed<T, VEC, S, Q, CP>;
};
template <typename T, int VEC, int S, int Q> struct GatedFeedOf<T, VEC, S, Q, kCpShifted> {
    using type = GatedShiftedFeed<T, VEC, S, Q>;
};

__device__ __forceinline__ Lane1 lshfl_up(Lane1 a, int by) { return {__shfl_up_sync(~0u, a.v, by)}; }
__device__ __forceinline__ Lane2 lshfl_up(Lane2 a, int by) {
    return {make_float2(__shfl_up_sync(~0u, a.v.x, by), __shfl_up_sync(~0u, a.v.y, by))};
}

__device__ __forceinline__ Lane1 lshfl_down(Lane1 a, int by) { return {__shfl_down_sync(~0u, a.v, by)}; }
__device__ __forceinline__ Lane2 lshfl_down(Lane2 a, int by) {
    return {make_float2(__shfl_down_sync(~0u, a.v.x, by), __shfl_down_sync(~0u, a.v.y, by))};
}

// ------------------------------------------------------------------- the scan
// A step is h -> (1 - u) h + u x, so a run of steps is h -> P h + b with
// P = prod(1 - u) and b the state that the run reaches from zero; runs compose
// as (P2, b2) after (P1, b1) = (P2 P1, b2 + P2 b1).  A row's own state is P h + b
// with the rounded P, whose error goes no further; from run to run the maps are
// those above.
//
// A lane takes a run of S = 16 rows of its channels; a warp holds Q runs side by
// side, a CTA's W = 4 or 8 warps a chunk of 16 W Q rows, the CTAs of a cluster consecutive
// chunks, and the cluster walks its sequence in strides of all of them.  Each
// lane forms its rows' states from zero and products in registers; a shuffle,
// one exchange through shared memory and one through the cluster's distributed
// shared memory give it the map of everything before its run; then one FMA a
// row makes the true states.  Every input is read once, and no chunk waits for
// another but its cluster's.  A warp's rows come by asynchronous copies into
// two stages of its own, a row's g and x replaced as soon as the states are in
// registers: a stage needs no barrier but the warp's.
//
// Q and the cluster make the parallel work of few channels: Q = 2 and 4 halve
// and quarter the channels of a CTA (to 64 and 32 bytes of a row) and lengthen
// its chunk; a cluster splits the sequence further at the price of a cluster
// barrier per round.
//
// What bounds it: HBM in fp32 (4096 x 4096 with z: 44 us, 6.1 TB/s); in bf16,
// where an element is half the bytes for the same arithmetic, a round's latency at
// the 16 warps an SM that 128 registers leave: 13 x 4096 x 2048 takes 161 to 168 us
// (5.2 to 5.4 TB/s), and in the like 8 x 2048 x 4096 the issue slots and the
// special-function pipe are half used; 8192 channels by 4096 rows, with 256 tiles on
// 148 SMs, 59 us (4.6 TB/s).  The steps there, us at 13 x 4096 x 2048 before the maps
// held P - 1: runs of 8 rows and 8 warps 174, without the copies 143, without the
// sigmoids too 107; runs of 16 and 4 warps, which halve the exchange's share of a row,
// 158.  A reciprocal for each sigmoid, and three or four stages instead of two, were
// slower or no faster.
constexpr int kGatedMaxCluster = 8;
constexpr int kGatedRun = 16;

template <bool GATE, int W, int Q, int CP> struct GatedScanCfg {
    static constexpr int kThreads = 32 * W;
    static constexpr int kArrays = GATE ? 3 : 2;
    static constexpr int kArrayBytes =  // one array's rows of one warp
        CP == kCpShifted ? GatedShiftedFeed<float, 1, kGatedRun, Q>::kBytes : kGatedRun * 128;
    static constexpr int kStageBytes = kArrays * kArrayBytes;
    static constexpr int kSmemBytes = W * 2 * kStageBytes;
};

template <typename T, int VEC, bool GATE, int Q, int CP, bool CLUSTER, int W>
__global__ void __launch_bounds__(32 * W, 16 / W) gated_scan_kernel(const GatedArgs a, int cs) {
    using Raw = GatedRaw<T, VEC>;
    using R = typename Raw::type;
    using C = GatedScanCfg<GATE, W, Q, CP>;
    using L = Lane<VEC>;
    using Map = RunMap<VEC>;
    constexpr int S = kGatedRun, LPR = 32 / Q, kChunk = W * S * Q;
    constexpr int kBlockWarps = kGatedCkpt / (S * Q);  // warps of a checkpoint's 64 rows
    static_assert(kBlockWarps >= 1 && W % kBlockWarps == 0, "");
    using F = typename GatedFeedOf<T, VEC, S, Q, CP>::type;
    extern __shared__ __align__(128) uint8_t stages[];
    __shared__ Map runs[2][W][LPR];
    __shared__ Map chunks[CLUSTER ? 2 : 1][CLUSTER ? kGatedMaxCluster : 1][LPR];
    __shared__ L last[2][LPR];  // without a cluster: the state behind the last chunk
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = lane % LPR, run = lane / LPR;
    if (!CLUSTER) cs = 1;
    if (CLUSTER) cluster_arrive();  // waited for before the first store to another CTA
    const int rank = CLUSTER ? static_cast<int>(cluster_rank()) : 0;
    const int tiles = (a.d + LPR * VEC - 1) / (LPR * VEC);
    const int64_t unit = blockIdx.x / cs;
    __shared__ int order[C::kThreads + 1];
    const int b = gated_sequence<C::kThreads>(a, static_cast<int>(unit / tiles), order);
    const int c0 = static_cast<int>(unit % tiles) * LPR * VEC, c = c0 + col * VEC;
    const bool on = c < a.d;

    int64_t row0, len64;
    gated_rows(a, b, row0, len64);
    const int len = static_cast<int>(len64);  // at most 2^30
    const int stride = cs * kChunk;           // rows between this CTA's chunks
    const int rounds = (len + stride - 1) / stride;
    int t = rank * kChunk + warp * (S * Q);  // this warp's first row
    uint8_t *const mine = stages + warp * (2 * C::kStageBytes);
    F fg, fx, fz;
    const bool in = c0 + F::channel_of(lane) < a.d;
    if constexpr (CP == kCpShifted) {
        fg.start(a.g, row0 + t, a.gs, c0, lane, stride, a.total, a.d);
        fx.start(a.x, row0 + t, a.xs, c0, lane, stride, a.total, a.d);
        if (GATE) fz.start(a.z, row0 + t, a.zs, c0, lane, stride, a.total, a.d);
    } else {
        fg.start(a.g, row0 + t, a.gs, c0, lane, stride);
        fx.start(a.x, row0 + t, a.xs, c0, lane, stride);
        if (GATE) fz.start(a.z, row0 + t, a.zs, c0, lane, stride);
    }
    auto fill_gx = [&](int left, int stage) {  // left: rows from the copied round's first on
        if (left > 0) {
            const uint32_t to = smem_u32(mine) + stage * C::kStageBytes;
            fg.copy(to, in, min(left, S * Q), lane);
            fx.copy(to + C::kArrayBytes, in, min(left, S * Q), lane);
        }
        cp_async_commit();
    };
    auto fill_z = [&](int left, int stage) {
        if (!GATE) return;
        if (left > 0)
            fz.copy(smem_u32(mine) + stage * C::kStageBytes + 2 * C::kArrayBytes, in,
                    min(left, S * Q), lane);
        cp_async_commit();
    };
    fill_gx(len - t, 0);
    fill_z(len - t, 0);
    fill_gx(len - t - stride, 1);
    fill_z(len - t - stride, 1);
    // waits for the oldest of the copies in flight: g and x of two rounds, and z of two
    auto oldest = [&]() {
        cp_async_wait<GATE ? 3 : 1>();
        __syncwarp();
    };

    int64_t in_row = b, out_row = b;
    if (a.state_indices) {
        const bool report = threadIdx.x == 0 && rank == 0 && unit % tiles == 0;
        out_row = gated_slot(a, a.state_indices[b], report);
        in_row = a.initial_indices ? gated_slot(a, a.initial_indices[b], report) : out_row;
    }
    L carry, nrate, bias;  // nrate: -rate, so that -u comes out of one product
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        carry.set(v, on && a.h0 && in_row >= 0 ? a.h0[in_row * a.d + c + v] : 0.0f);
        nrate.set(v, on && a.rate ? -a.rate[c + v] : -1.0f);
        bias.set(v, on && a.bias ? a.bias[c + v] : 0.0f);
    }
    const L one = L::of(1.0f), zero = L::of(0.0f), held = L::of(kHeld);
    T *op = static_cast<T *>(a.out) + (row0 + t + run * S) * a.d + c;
    const bool store = on && a.out;
    float *ck = warp % kBlockWarps == 0 && run == 0 && on && a.ckpt
                    ? a.ckpt + (row0 / kGatedCkpt + b + t / kGatedCkpt) * a.d + c
                    : nullptr;
    if (CLUSTER) cluster_wait();  // every CTA of the cluster has started
    for (int k = 0; k < rounds; ++k, t += stride) {
        const int par = k & 1;
        const bool full = len - t >= S * Q;
        const int n = min(len - t - run * S, S);  // rows of this lane's run
        const uint8_t *st = mine + par * C::kStageBytes;
        const R *gp = reinterpret_cast<const R *>(st) + F::first_word(lane);
        const R *xp = reinterpret_cast<const R *>(st + C::kArrayBytes) + F::first_word(lane);
        const R *zp = reinterpret_cast<const R *>(st + 2 * C::kArrayBytes) + F::first_word(lane);
        auto gr = [&](int i) { return Raw::get(gp[fg.word_of(i)]); };
        auto xr = [&](int i) { return Raw::get(xp[fx.word_of(i)]); };
        auto zr = [&](int i) { return Raw::get(zp[fz.word_of(i)]); };
        oldest();  // this round's g and x
        // the states from zero and the products of (1 - u), row by row
        L h[S], P[S], ph = zero, pp = one, pn = zero;
        auto step = [&](int i, L s) {
            const L nu = lmul(s, nrate);
            ph = lfma(nu, lsub(ph, xr(i)), ph);
            pn = lfma(nu, pp, pn);
            pp = lfma(nu, pp, pp);
        };
        bool good = full;
        if (full) {
#pragma unroll
            for (int i = 0; i < S; ++i) {
                step(i, lsigmoid_pair(ladd(gr(i), bias), good));
                h[i] = ph, P[i] = pp;
            }
        }
        if (!good && on) {
            ph = pn = zero, pp = one;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                if (i < n) step(i, lsigmoid(ladd(gr(i), bias)));
                h[i] = ph, P[i] = pp;
            }
        }
        // the runs of this warp before the lane's own: sp, sb; all of them: ip, ib on the last
        L sp = held, sb = zero, ip = ldecay(pp, pn), ib = ph;
        if constexpr (Q > 1) {
#pragma unroll
            for (int by = LPR; by < 32; by *= 2) {
                const L op2 = lshfl_up(ip, by), ob = lshfl_up(ib, by);
                if (lane >= by) {
                    ib = lapply(ip, ob, ib);
                    ip = ljoin(ip, op2);
                }
            }
            const L ep = lshfl_up(ip, LPR), eb = lshfl_up(ib, LPR);
            if (run > 0) sp = ep, sb = eb;
        }
        if (run == Q - 1) runs[par][warp][col] = Map::of(ip, ib);
        __syncthreads();
        fill_gx(len - t - 2 * stride, par);  // g and x of this round have been read
        L mb;
        if constexpr (CLUSTER) {
            // the warps before this one, as a map
            Map r[W - 1];
#pragma unroll
            for (int w = 0; w < W - 1; ++w) r[w] = runs[par][w][col];
            L mp = held;
            mb = zero;
#pragma unroll
            for (int w = 0; w < W - 1; ++w) {
                if (w < warp) {
                    mb = lapply(r[w].q(), mb, r[w].b());
                    mp = ljoin(r[w].q(), mp);
                }
            }
            if (warp == W - 1 && run == Q - 1) {  // the chunk's map to every CTA of the cluster
                const Map m = Map::of(ljoin(ip, mp), lapply(ip, mb, ib));
                const uint32_t at = smem_u32(&chunks[par][rank][col]);
#pragma unroll
                for (int r = 0; r < kGatedMaxCluster; ++r)
                    if (r < cs) st_cluster(at, r, m);
            }
            __syncwarp();
            cluster_arrive();
            cluster_wait();
            L before = carry;
            Map q[kGatedMaxCluster];
#pragma unroll
            for (int r = 0; r < kGatedMaxCluster; ++r) q[r] = chunks[par][r][col];
#pragma unroll
            for (int r = 0; r < kGatedMaxCluster; ++r) {
                if (r == rank) before = carry;
                if (r < cs) carry = lapply(q[r].q(), carry, q[r].b());
            }
            mb = lapply(mp, before, mb);
        } else {
            // warp W - 1 left the last chunk's last state before this round's barrier
            if (k > 0) carry = last[par][col];
            Map r[W - 1];
#pragma unroll
            for (int w = 0; w < W - 1; ++w) r[w] = runs[par][w][col];
            mb = carry;
#pragma unroll
            for (int w = 0; w < W - 1; ++w)
                if (w < warp) mb = lapply(r[w].q(), mb, r[w].b());
            if (warp == W - 1 && run == Q - 1) last[par ^ 1][col] = lapply(ip, mb, ib);
        }
        // mb: the state before this warp's rows
        if (ck && t < len) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) ck[v] = mb.get(v);
            ck += int64_t(stride / kGatedCkpt) * a.d;
        }
        if (Q > 1) mb = lapply(sp, mb, sb);  // before this lane's
        if (GATE) oldest();  // this round's z
        good = full;
        if (full) {
            T *o = op;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                L ov = lfma(P[i], mb, h[i]);
                if (GATE) {
                    const L zv = zr(i);
                    ov = lmul(ov, lmul(zv, lsigmoid_pair(zv, good)));
                }
                if (store) *reinterpret_cast<R *>(o) = Raw::put(ov);
                o += a.d;
            }
        }
        if (!good && on) {
            T *o = op;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                L ov = lfma(P[i], mb, h[i]);
                if (GATE) {
                    const L zv = zr(i);
                    ov = lmul(ov, lmul(zv, lsigmoid(zv)));
                }
                if (store && i < n) *reinterpret_cast<R *>(o) = Raw::put(ov);
                o += a.d;
            }
        }
        op += int64_t(stride) * a.d;
        if (GATE) {
            __syncwarp();  // every lane has read the z that the next copy overwrites
            fill_z(len - t - 2 * stride, par);
        }
    }
    cp_async_wait<0>();
    if (a.h_final && out_row >= 0 && on && rank == 0 && warp == W - 1 && run == Q - 1) {
        if (!CLUSTER && rounds > 0) carry = last[rounds & 1][col];
#pragma unroll
        for (int v = 0; v < VEC; ++v) a.h_final[out_row * a.d + c + v] = carry.get(v);
    }
}

}  // namespace jssm
