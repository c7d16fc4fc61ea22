// i8_proj.cuh -- the 8-bit product with a scale for each token and each output
// channel: out[t, o] = (sum_k q[t, k] w[o, k]) q_scale[t] w_scale[o] + bias[o].
//
// The sums are tcgen05.mma of kind::i8 with 32-bit integer accumulators in
// TMEM, exact in any order.  The weight's rows are the product's M side (TMEM
// lanes) and the tokens its N side (columns), so that a decode step's few
// tokens fill an MMA as narrow as they are, and a thread holds one output
// channel: its scale and bias stay in registers, the tokens' scales come from
// shared memory, and a warp writes 32 neighbouring outputs of a token at once.
#pragma once

#include "device_utils.cuh"
#include "launch_order.cuh"
#include "tcgen05_utils.cuh"

namespace jssm {

struct I8ProjArgs {
    const float *qs, *ws, *bias;
    void *out;
    int ntok, n, kblocks;  // kblocks: 128-byte blocks of K
    int ks;                // CTAs that share a tile's K (the split kernel)
    bool pairs;            // two bf16 channels can be written as a word
    uint32_t withhold;     // test of the bounded waits: ranks (bits) that leave out their first copies
    uint64_t limit;
};

// Scales between 2^-60 and 2^60, and 0: no order of the factors overflows early.
__device__ __forceinline__ bool i8_tame(float s) {
    return s == 0.0f || (s >= 0x1p-60f && s <= 0x1p60f);
}
// acc * s * w.  Where a scale is not tame the smaller one comes first: acc * (the
// larger) could overflow where the whole product does not.  The order follows from
// the two scales alone, so an output has the same bits whatever tile, split or
// batch it is computed in (with s below 2^-60 and w tame, s is the smaller one).
// A NaN scale stays one.
__device__ __forceinline__ float i8_scaled(int acc, float s, float w, bool w_tame) {
    const bool s_first = s < w || (w_tame && s <= 0x1p60f);
    return static_cast<float>(acc) * (s_first ? s : w) * (s_first ? w : s);
}

// Columns [0, cols) of a lane's channel (tokens `out` on, n elements apart) from
// COLS accumulators.  `tame`: every scale is.  `pairs` (bf16, n even and the
// rows 4-byte aligned): neighbouring lanes exchange every other column, so that
// each writes two channels of one token as a word, and a warp's store 16 words
// of two tokens: half the store instructions, which with the rest of this loop
// bound the kernel's tiles where K is short.
template <typename T, bool TAME, bool WHOLE, int COLS>
__device__ __forceinline__ void i8_columns(T *out, int64_t n, const uint32_t (&v)[COLS], const float *sc,
                                           float w, float bias, bool on, int cols, bool pairs) {
    const bool w_tame = i8_tame(w);
    auto value = [&](int i) {
        const float s = sc[i];
        const float p = TAME ? static_cast<float>(int(v[i])) * s * w : i8_scaled(int(v[i]), s, w, w_tame);
        return p + bias;
    };
    if constexpr (sizeof(T) == 2) {
        if (pairs) {
            const bool odd = threadIdx.x & 1;
            T *at = odd ? out + n - 1 : out;
#pragma unroll
            for (int i = 0; i < COLS; i += 2) {
                const float a = value(i), b = value(i + 1);
                const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
                const uint32_t word = pack_bf16x2(odd ? got : a, odd ? b : got);
                if (WHOLE || (on && i + int(odd) < cols)) *reinterpret_cast<uint32_t *>(at) = word;
                at += 2 * n;
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < COLS; ++i) {
        if (WHOLE || (on && i < cols)) *out = from_f32<T>(value(i));
        out += n;
    }
}
template <typename T, int COLS>
__device__ __forceinline__ void i8_put(T *out, int64_t n, const uint32_t (&v)[COLS], const float *sc, float w,
                                       float bias, bool on, int cols, bool tame, bool pairs) {
    tame = __all_sync(0xffffffffu, tame && i8_tame(w));
    const bool whole = __all_sync(0xffffffffu, on && cols >= COLS);
    if (tame && whole)
        i8_columns<T, true, true>(out, n, v, sc, w, bias, on, cols, pairs);
    else if (tame)
        i8_columns<T, true, false>(out, n, v, sc, w, bias, on, cols, pairs);
    else
        i8_columns<T, false, false>(out, n, v, sc, w, bias, on, cols, pairs);
}

constexpr uint32_t i8_idesc(int m, int n) {
    return (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

template <int CTAS>
__device__ __forceinline__ void umma_i8(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
    if constexpr (CTAS == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
}

__device__ __forceinline__ uint32_t mapa(uint32_t saddr, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    return a;
}
__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The pair's forms: a copy into this CTA's shared memory that completes on the
// leader's barrier, a commit that arrives on both CTAs' barriers, an arrival on
// the leader's barrier, and the pair's TMEM.
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, int c0, int c1,
                                                 uint32_t bar_cluster) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar_cluster)
        : "memory");
}
__device__ __forceinline__ void tc_commit_pair(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar_cluster) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster)
                 : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t *slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}

// A wait for a barrier that this thread gives up when `limit` cycles pass or
// another thread of the CTA gave one up.
struct I8Wait {
    uint64_t limit;
    volatile int *abort;
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) const {
        if (mbar_wait_or_abort(bar, parity, limit, abort)) return true;
        fail();
        return false;
    }
    __device__ __forceinline__ void fail() const {
        if (!*abort) record_status(nullptr, kStTimeout);
        *abort = 1;
    }
};

// ------------------------------------------------------------- many tokens
// Persistent CTA pairs on tiles of 256 channels x 256 tokens: one MMA spans the
// pair (cta_group::2), each CTA staging its 128 channels and 128 of the tokens,
// so a 128-byte block of K costs an SM 32 KB for 256 x 256 x 128 products of
// the pair -- a third less from L2 than a CTA of its own with 128 x 256.  Six
// stages; two accumulators of 256 TMEM columns, so a tile's outputs are written
// while the next tile's products run.  4096 x 4096 x 16384: 158 to 175 us alone, by
// the clock, the tensor pipe 83% active; 178 to 205 back to back, where the power
// limit lowers the clock.  What the outputs cost shows at K 4096 and below: 205 us with 4 warps
// that wrote one bf16 channel at a time, 181 with two channels a word, 178 with 8.
struct I8PairCfg {
    static constexpr int kTile = 256;               // channels and tokens of a pair's tile
    static constexpr int kHalf = 128;
    static constexpr int kStages = 6;
    static constexpr int kOperand = kHalf * 128;    // bytes of one operand's stage
    static constexpr int kStage = 2 * kOperand;
    static constexpr int kOffScale = kStages * kStage;            // 2 x 256 token scales
    static constexpr int kOffBar = kOffScale + 2 * kTile * 4;
    static constexpr int kSmem = kOffBar + 256 + 1024;            // and up to 1024 to align
    static constexpr int kOutWarps = 8;             // two to a quarter of the TMEM lanes
    static constexpr int kThreads = 64 + 32 * kOutWarps;  // and the copies' warp and the MMAs'
    static constexpr uint32_t kIdesc = i8_idesc(256, 256);
};

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(I8PairCfg::kThreads, 1)
    i8_proj_pair_kernel(const __grid_constant__ CUtensorMap map_w,
                        const __grid_constant__ CUtensorMap map_q, const I8ProjArgs a) {
    using C = I8PairCfg;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    float *scales = reinterpret_cast<float *>(smem + C::kOffScale);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *empty = full + C::kStages, *acc_full = empty + C::kStages, *acc_empty = acc_full + 2;
    uint64_t *drain = acc_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();
    const bool leader = rank == 0;
    const I8Wait wait{a.limit, abort_flag};
    const int tok_tiles = (a.ntok + C::kTile - 1) / C::kTile, ch_tiles = (a.n + C::kTile - 1) / C::kTile;
    const int64_t tiles = int64_t(tok_tiles) * ch_tiles;
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 2 * C::kOutWarps);  // both CTAs'
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
        prefetch_tensormap(&map_w);
        prefetch_tensormap(&map_q);
    }
    if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    cluster_barrier();
    tc_fence_after();
    after_earlier_work();
    let_next_begin();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(tmem_slot);

    if (warp == 0) {
        if (lane == 0) {
            int wi = 0;
            bool ok = true;
            for (int64_t it = pair; it < tiles && ok; it += pairs) {
                const int m0 = static_cast<int>(it % tok_tiles) * C::kTile + int(rank) * C::kHalf;
                const int n0 = static_cast<int>(it / tok_tiles) * C::kTile + int(rank) * C::kHalf;
                for (int kb = 0; kb < a.kblocks; ++kb, ++wi) {
                    const int s = wi % C::kStages;
                    if (wi >= C::kStages && !wait(&empty[s], ((wi / C::kStages) & 1) ^ 1)) {
                        ok = false;
                        break;
                    }
                    if (wi == 0 && ((a.withhold >> rank) & 1u)) continue;
                    uint8_t *st = smem + s * C::kStage;
                    if (leader) mbar_arrive_expect_tx(&full[s], 2 * C::kStage);
                    const uint32_t bar = mapa(smem_u32(&full[s]), 0);
                    tma_load_2d_pair(st, &map_w, kb * 128, n0, bar);
                    tma_load_2d_pair(st + C::kOperand, &map_q, kb * 128, m0, bar);
                }
            }
            // No copy may still be landing when the pair moves on: the leader sees both CTAs'.
            if (leader)
                for (int j = max(wi - C::kStages, 0); j < wi; ++j)
                    if (!mbar_wait_bounded(&full[j % C::kStages], (j / C::kStages) & 1, a.limit)) wait.fail();
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leader && lane == 0) {
            int wi = 0, j = 0;
            bool ok = true;
            for (int64_t it = pair; it < tiles && ok; it += pairs, ++j) {
                const int buf = j & 1;
                if (j >= 2 && !wait(&acc_empty[buf], ((j / 2) - 1) & 1)) break;
                tc_fence_after();
                for (int kb = 0; kb < a.kblocks; ++kb, ++wi) {
                    const int s = wi % C::kStages;
                    if (!wait(&full[s], (wi / C::kStages) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t at = smem_u32(smem + s * C::kStage);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_i8<2>(tmem + uint32_t(buf) * C::kTile, umma_desc_sw128(at + k * 32),
                                   umma_desc_sw128(at + C::kOperand + k * 32), C::kIdesc,
                                   (kb | k) != 0 ? 1u : 0u);
                    tc_commit_pair(&empty[s]);
                }
                if (!ok) break;
                tc_commit_pair(&acc_full[buf]);
            }
            // TMEM is not freed while MMAs run.
            tc_commit_pair(drain);
            if (!mbar_wait_bounded(drain, 0, a.limit)) wait.fail();
        }
        __syncwarp();
    } else {
        // this warp's TMEM lanes, 32 q .. 32 q + 31, and its half of the columns
        constexpr int kOut = 32 * C::kOutWarps, kCols = C::kTile / (C::kOutWarps / 4);
        const int q = warp & 3, c0 = (warp - 2) / 4 * kCols;
        int j = 0;
        for (int64_t it = pair; it < tiles; it += pairs, ++j) {
            const int buf = j & 1;
            const int m0 = static_cast<int>(it % tok_tiles) * C::kTile;
            const int o = static_cast<int>(it / tok_tiles) * C::kTile + int(rank) * C::kHalf + q * 32 + lane;
            const bool on = o < a.n;
            const float w = on ? a.ws[o] : 0.0f, bias = on && a.bias ? a.bias[o] : 0.0f;
            float *sc = scales + buf * C::kTile;
            bool tame = true;
            for (int i = threadIdx.x - 64; i < C::kTile; i += kOut) {
                sc[i] = m0 + i < a.ntok ? a.qs[m0 + i] : 0.0f;
                tame = tame && i8_tame(sc[i]);
            }
            tame = epilogue_all(tame, kOut);  // and the scales are staged
            if (!epilogue_all(wait(&acc_full[buf], (j / 2) & 1), kOut)) break;
            tc_fence_after();
            T *out = static_cast<T *>(a.out) + int64_t(m0) * a.n + o;
            const int cols = min(C::kTile, a.ntok - m0);
            const uint32_t at = tmem + (uint32_t(q * 32) << 16) + uint32_t(buf * C::kTile);
#pragma unroll 1
            for (int c = c0; c < min(c0 + kCols, cols); c += 32) {
                float f[32];
                tmem_ld32(at + uint32_t(c), f);
                uint32_t v[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(f[i]);
                i8_put<T>(out + int64_t(c) * a.n, a.n, v, sc + c, w, bias, on, cols - c, tame, a.pairs);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa(smem_u32(&acc_empty[buf]), 0));
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_barrier();  // neither CTA leaves while the other's copies, MMAs or arrivals may reach it
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// -------------------------------------------------------------- few tokens
// One CTA to a tile of 128 channels x NT tokens and a part of K: what bounds a
// decode step is reading the weight once, so the CTAs of a cluster share a
// tile's K until the device is full, every CTA with up to 200 KB of the weight
// on its way.  The cluster then adds its partial sums: each CTA sends every
// other one the columns that it finishes, through distributed shared memory.
// 8 tokens, K 8192, 4096 channels, 4 CTAs to a tile: 10.9 us with the weight from HBM
// (3.1 TB/s of it), 9.4 where L2 still holds a part; K 4096, 16384 channels 15.4 (4.4).
template <int NT> struct I8SplitCfg {
    static constexpr int kM = 128;
    static constexpr int kA = kM * 128, kB = NT * 128;
    static constexpr int kStage = kA + kB;
    static constexpr int kStages = NT <= 32 ? 10 : NT == 64 ? 8 : 6;
    static constexpr int kOffScale = kStages * kStage;
    static constexpr int kOffBar = kOffScale + NT * 4;
    static constexpr int kSmem = kOffBar + 256 + 1024;
    static constexpr int kThreads = 192;
    static constexpr int kTmemCols = NT < 32 ? 32 : NT;
    static constexpr uint32_t kIdesc = i8_idesc(kM, NT);
    static_assert(kStages * kStage >= NT * kM * 4, "the partial sums fit the stages");
};
constexpr int kI8MaxSplit = 8;

template <typename T, int NT>
__global__ void __launch_bounds__(I8SplitCfg<NT>::kThreads, 1)
    i8_proj_split_kernel(const __grid_constant__ CUtensorMap map_w,
                         const __grid_constant__ CUtensorMap map_q, const I8ProjArgs a) {
    using C = I8SplitCfg<NT>;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    float *scales = reinterpret_cast<float *>(smem + C::kOffScale);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *empty = full + C::kStages, *acc_full = empty + C::kStages;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_full + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *sums_lost = abort_flag + 1;  // another CTA of the cluster gave a wait up
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = a.ks > 1 ? static_cast<int>(cta_rank()) : 0;
    const I8Wait wait{a.limit, abort_flag};
    const int tok_tiles = (a.ntok + NT - 1) / NT;
    const int64_t it = blockIdx.x / a.ks;
    const int m0 = static_cast<int>(it % tok_tiles) * NT;
    const int n0 = static_cast<int>(it / tok_tiles) * C::kM;
    const int kb0 = static_cast<int>(int64_t(a.kblocks) * rank / a.ks);
    const int cnt = static_cast<int>(int64_t(a.kblocks) * (rank + 1) / a.ks) - kb0;  // >= 1

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        *abort_flag = *sums_lost = 0;
        fence_mbarrier_init();
        prefetch_tensormap(&map_w);
        prefetch_tensormap(&map_q);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    after_earlier_work();
    let_next_begin();
    bool tame = true;
    for (int i = threadIdx.x; i < NT; i += C::kThreads) {
        scales[i] = m0 + i < a.ntok ? a.qs[m0 + i] : 0.0f;
        tame = tame && i8_tame(scales[i]);
    }
    tc_fence_before();
    tame = __syncthreads_and(tame);  // and the scales are staged
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(tmem_slot);

    if (warp == 0) {
        if (lane == 0) {
            int issued = 0;
            for (; issued < cnt; ++issued) {
                const int s = issued % C::kStages;
                if (issued >= C::kStages && !wait(&empty[s], ((issued / C::kStages) & 1) ^ 1)) break;
                if (issued == 0 && ((a.withhold >> rank) & 1u)) continue;
                uint8_t *st = smem + s * C::kStage;
                mbar_arrive_expect_tx(&full[s], C::kStage);
                tma_load_2d(st, &map_w, (kb0 + issued) * 128, n0, &full[s]);
                tma_load_2d(st + C::kA, &map_q, (kb0 + issued) * 128, m0, &full[s]);
            }
            for (int j = max(issued - C::kStages, 0); j < issued; ++j)  // none still landing
                if (!mbar_wait_bounded(&full[j % C::kStages], (j / C::kStages) & 1, a.limit)) wait.fail();
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            for (int i = 0; i < cnt; ++i) {
                const int s = i % C::kStages;
                if (!wait(&full[s], (i / C::kStages) & 1)) break;
                tc_fence_after();
                const uint32_t at = smem_u32(smem + s * C::kStage);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_i8<1>(tmem, umma_desc_sw128(at + k * 32), umma_desc_sw128(at + C::kA + k * 32),
                               C::kIdesc, (i | k) != 0 ? 1u : 0u);
                tc_commit(&empty[s]);
            }
            tc_commit(acc_full);  // arrives once every MMA issued above has completed
            if (!mbar_wait_bounded(acc_full, 0, a.limit)) wait.fail();
        }
        __syncwarp();
    }
    __syncthreads();  // every copy has landed and every MMA has completed, or the wait was given up
    tc_fence_after();
    const int q = warp & 3;
    const int o = n0 + q * 32 + lane;
    bool on = o < a.n && !*abort_flag;
    const float w = on ? a.ws[o] : 0.0f, bias = on && a.bias ? a.bias[o] : 0.0f;
    const int cols = min(NT, a.ntok - m0);
    T *out = static_cast<T *>(a.out) + int64_t(m0) * a.n + o;
    const uint32_t lanes = tmem + (uint32_t(q * 32) << 16);
    if (a.ks == 1) {
        if (warp >= 2) {
#pragma unroll 1
            for (int c = 0; c < cols; c += 16) {
                uint32_t v[16];
                tmem_ld16_async(lanes + c, v);
                tmem_wait_ld();
                tmem_regs_ready(v);
                i8_put<T>(out + int64_t(c) * a.n, a.n, v, scales + c, w, bias, on, cols - c, tame, a.pairs);
            }
        }
    } else {
        // CTA r finishes the columns from r * own on, in pairs and fours of columns:
        // slot [group][source rank][channel][column of the group]
        uint8_t *sums = smem;
        const int own = NT / a.ks, log_own = __ffs(own) - 1;
        cluster_barrier();  // every CTA's stages are free
        if (threadIdx.x < a.ks && *abort_flag)  // no CTA takes this one's part for a sum
            asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(
                             mapa(smem_u32(const_cast<int *>(sums_lost)), threadIdx.x)),
                         "r"(1)
                         : "memory");
        __syncwarp();
        if (warp >= 2) {
            const int width = own >= 4 ? 4 : 2;  // columns of a group
            const uint32_t at = smem_u32(sums) + (rank * C::kM + q * 32 + lane) * width * 4;
            const uint32_t group = a.ks * C::kM * width * 4;
#pragma unroll 1
            for (int c = 0; c < cols; c += 16) {
                uint32_t v[16];
                tmem_ld16_async(lanes + c, v);
                tmem_wait_ld();
                tmem_regs_ready(v);
                if (own >= 4) {
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const uint32_t to = mapa(at + (((c + i) & (own - 1)) >> 2) * group, (c + i) >> log_own);
                        asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(v[i]),
                                     "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3])
                                     : "memory");
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; i += 2)
                        asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(mapa(at, (c + i) >> 1)),
                                     "r"(v[i]), "r"(v[i + 1])
                                     : "memory");
                }
            }
        }
        cluster_barrier();
        on = on && !*sums_lost;
        if (warp >= 2) {
            const int c0 = rank * own, end = min(c0 + own, cols);
            if (own >= 4) {
                const int4 *mine = reinterpret_cast<const int4 *>(sums) + q * 32 + lane;
                for (int c = c0; c < end; c += 4) {
                    int4 t = make_int4(0, 0, 0, 0);
                    for (int r = 0; r < a.ks; ++r) {
                        const int4 p = mine[r * C::kM];
                        t.x += p.x, t.y += p.y, t.z += p.z, t.w += p.w;
                    }
                    mine += a.ks * C::kM;
                    const uint32_t acc[4] = {uint32_t(t.x), uint32_t(t.y), uint32_t(t.z), uint32_t(t.w)};
                    i8_put<T>(out + int64_t(c) * a.n, a.n, acc, scales + c, w, bias, on, end - c, tame,
                              a.pairs);
                }
            } else {
                const int2 *mine = reinterpret_cast<const int2 *>(sums) + q * 32 + lane;
                int2 t = make_int2(0, 0);
                for (int r = 0; r < a.ks; ++r) {
                    const int2 p = mine[r * C::kM];
                    t.x += p.x, t.y += p.y;
                }
                const uint32_t acc[2] = {uint32_t(t.x), uint32_t(t.y)};
                i8_put<T>(out + int64_t(c0) * a.n, a.n, acc, scales + c0, w, bias, on, end - c0, tame, a.pairs);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

}  // namespace jssm
