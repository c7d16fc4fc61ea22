// batch_maps.cuh -- the maps of a continuous batch from its requests' lengths.
//
// Everything follows from three running sums over the requests: of the tokens,
// of the cache blocks that a request needs beyond those it has, and of the
// requests that start and take a state slot.  A new block's first token is one
// of this step's, so the thread that maps that token writes the block's table
// entry too, and nothing loops over a long request.
//
// Up to 2048 requests the call is one launch of CTAs that each compute all the
// sums in shared memory (the lengths come from L2) and then map 1024 tokens: a
// second launch, or a wait for one CTA's sums, would cost more than the few
// thousand additions.  It is bound by latency: a load of the lengths, two block
// scans, a search and a store (256 requests of one token: 5.5 us; 1000 requests,
// 131072 tokens: 6.4 us, of which the 2.1 MB of maps would take 0.3).  More
// requests take two launches, the second searching the first's cu_seqlens.
#pragma once

#include "device_utils.cuh"
#include "launch_order.cuh"

namespace jssm {

struct BatchMapsArgs {
    int requests, max_tokens, max_blocks, block_size;
    const int32_t *new_lens, *ctx_lens, *free_blocks, *free_slots;
    int num_free_blocks, num_free_slots;
    int32_t *block_tables, *request_slots, *cu_seqlens, *positions, *token_request;
    int64_t *slot_map;
    int32_t *state_indices, *initial_indices, *counts;
    bool wide;  // the per-token maps are 16-byte aligned
};

constexpr int kMapsThreads = 256, kMapsTokens = 4, kMapsFused = 2048;
constexpr int kMapsManyThreads = 1024;

constexpr int64_t kMapsPositions = int64_t(1) << 31;  // a position is an int32

// v / by rounded up; v is at most 2^31 and by 2^20, so 32 bits hold the sum.
__device__ __forceinline__ int64_t ceil_div(int64_t v, int by) {
    return (static_cast<uint32_t>(v) + uint32_t(by) - 1) / uint32_t(by);
}

// One request's share, given n, the tokens of it that fit.
struct MapsRequest {
    int ctx, had, take;
    bool starts, too_long;
};
__device__ __forceinline__ int maps_ctx(const BatchMapsArgs &a, int b) {
    return a.ctx_lens ? max(a.ctx_lens[b], 0) : 0;
}
__device__ __forceinline__ MapsRequest maps_request(const BatchMapsArgs &a, int ctx, int n) {
    MapsRequest r;
    r.ctx = ctx;
    const int64_t most = a.max_blocks, end = int64_t(r.ctx) + n;
    r.had = static_cast<int>(min(ceil_div(r.ctx, a.block_size), most));
    const int64_t need = n > 0 ? ceil_div(min(end, kMapsPositions), a.block_size) : r.had;
    r.too_long = need > most || (n > 0 && end > kMapsPositions);
    r.take = max(static_cast<int>(min(need, most)) - r.had, 0);
    r.starts = n > 0 && r.ctx == 0;
    return r;
}

// Sum of v over the threads before this one; *total over all.  Two barriers.
template <int THREADS>
__device__ __forceinline__ int64_t maps_scan(int64_t v, int64_t *part, int64_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t s = v;
#pragma unroll
    for (int by = 1; by < 32; by *= 2) {
        const int64_t o = __shfl_up_sync(0xffffffffu, s, by);
        if (lane >= by) s += o;
    }
    if (lane == 31) part[warp] = s;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += part[w];
        all += part[w];
    }
    __syncthreads();  // `part` may be written again
    *total = all;
    return before + s - v;
}

// A request's state slots (`slot`: the one it holds), and the step's totals.
__device__ __forceinline__ void maps_state(const BatchMapsArgs &a, int b, int n, const MapsRequest &r,
                                           int64_t nth, int slot) {
    if (r.starts) {
        slot = nth < a.num_free_slots ? a.free_slots[nth] : -1;
        a.request_slots[b] = slot;
    }
    a.state_indices[b] = n > 0 ? slot : -1;
    a.initial_indices[b] = n > 0 && !r.starts ? slot : -1;
}
__device__ __forceinline__ void maps_totals(const BatchMapsArgs &a, int64_t tokens, int64_t blocks,
                                            int64_t slots, int longest, bool bad) {
    a.counts[0] = static_cast<int>(min(tokens, int64_t(a.max_tokens)));
    a.counts[1] = static_cast<int>(min(blocks, int64_t(a.num_free_blocks)));
    a.counts[2] = static_cast<int>(min(slots, int64_t(a.num_free_slots)));
    a.counts[3] = longest;
    if (bad || tokens > a.max_tokens || blocks > a.num_free_blocks || slots > a.num_free_slots)
        record_status(nullptr, kStInvalidArg);
}

// The request of token t: the last b with cu[b] <= t, where t < cu[n].
__device__ __forceinline__ int maps_find(const int *cu, int n, int t) {
    int lo = 0, hi = n;  // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (cu[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// kMapsTokens tokens from t0 on.  `block_of(b, ctx, j)`: the cache block that
// holds request b's block j, or a negative number.
template <typename C, typename F>
__device__ __forceinline__ void maps_tokens(const BatchMapsArgs &a, const int *cu, C ctx_of, int64_t t0,
                                            F block_of) {
    if (t0 >= a.max_tokens) return;
    const int total = cu[a.requests];
    int pos[kMapsTokens], req[kMapsTokens];
    int64_t slot[kMapsTokens];
    int b = -1, ctx = 0;
#pragma unroll
    for (int i = 0; i < kMapsTokens; ++i) {
        const int64_t t = t0 + i;
        pos[i] = req[i] = -1;
        slot[i] = -1;
        if (t < total) {
            if (b < 0 || t >= cu[b + 1]) {
                b = maps_find(cu, a.requests, static_cast<int>(t));
                ctx = ctx_of(b);
            }
            req[i] = b;
            const int64_t p = ctx + (t - cu[b]);
            if (p >= kMapsPositions) continue;  // no position: -1, as of a row without a token
            pos[i] = static_cast<int>(p);
            const int j = pos[i] / a.block_size, in = pos[i] - j * a.block_size;
            if (j < a.max_blocks) {
                const int blk = block_of(b, ctx, j, in);
                if (blk >= 0) slot[i] = int64_t(blk) * a.block_size + in;
            }
        }
    }
    if (a.wide && t0 + kMapsTokens <= a.max_tokens) {
        *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        *reinterpret_cast<int4 *>(a.token_request + t0) = make_int4(req[0], req[1], req[2], req[3]);
        *reinterpret_cast<longlong2 *>(a.slot_map + t0) = make_longlong2(slot[0], slot[1]);
        *reinterpret_cast<longlong2 *>(a.slot_map + t0 + 2) = make_longlong2(slot[2], slot[3]);
    } else {
#pragma unroll
        for (int i = 0; i < kMapsTokens; ++i) {
            if (t0 + i < a.max_tokens) {
                a.positions[t0 + i] = pos[i];
                a.token_request[t0 + i] = req[i];
                a.slot_map[t0 + i] = slot[i];
            }
        }
    }
}

// Up to kMapsFused requests; CTA i maps tokens from i * 1024 on, CTA 0 writes
// what there is of each request.  PER: requests of a thread, whose lengths stay
// in registers; one scan sums the blocks and, in the low 13 bits, the starts
// (blocks stay below 2^11 2^24).
template <int PER> __global__ void __launch_bounds__(kMapsThreads) batch_maps_kernel(const BatchMapsArgs a) {
    constexpr int kMost = kMapsThreads * PER;
    static_assert(kMost < 1 << 13 && kMost <= kMapsFused, "");
    __shared__ int cu[kMost + 1];
    __shared__ int first[kMost];  // a request's first place in free_blocks
    __shared__ int ctx_of[kMost];
    __shared__ int64_t part[kMapsThreads / 32];
    __shared__ int longest_of[kMapsThreads / 32];
    after_earlier_work();
    let_next_begin();
    const int b0 = int(threadIdx.x) * PER;
    int want[PER], ctx[PER], held[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool on = b0 + i < a.requests;
        want[i] = on ? max(a.new_lens[b0 + i], 0) : 0;
        ctx[i] = on ? maps_ctx(a, b0 + i) : 0;
        held[i] = on && blockIdx.x == 0 ? a.request_slots[b0 + i] : -1;
    }
    int64_t sum = 0, tokens, all;
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += want[i];
    int64_t before = maps_scan<kMapsThreads>(sum, part, &tokens);
    const int64_t cap = a.max_tokens;
    int n[PER], longest = 0;
    MapsRequest r[PER];
    int64_t add = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int lo = static_cast<int>(min(before, cap));
        cu[b0 + i] = lo;
        ctx_of[b0 + i] = ctx[i];
        before += want[i];
        n[i] = static_cast<int>(min(before, cap)) - lo;
        r[i] = maps_request(a, ctx[i], n[i]);
        longest = max(longest, n[i]);
        bad |= r[i].too_long;
        add += (int64_t(r[i].take) << 13) + r[i].starts;
    }
    if (threadIdx.x == kMapsThreads - 1) cu[kMost] = static_cast<int>(min(tokens, cap));
    int64_t at = maps_scan<kMapsThreads>(add, part, &all);
    const int64_t at0 = at;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        first[b0 + i] = static_cast<int>(min(at >> 13, int64_t(0x7fffffff)));
        at += (int64_t(r[i].take) << 13) + r[i].starts;
    }
    __syncthreads();
    maps_tokens(a, cu, [&](int b) { return ctx_of[b]; },
                (int64_t(blockIdx.x) * kMapsThreads + threadIdx.x) * kMapsTokens,
                [&](int b, int c, int j, int in) {
                    int32_t *entry = a.block_tables + int64_t(b) * a.max_blocks + j;
                    const int64_t fresh = j - ceil_div(c, a.block_size);
                    if (fresh < 0) return *entry;
                    const int64_t f = int64_t(first[b]) + fresh;
                    const int blk = f < a.num_free_blocks ? a.free_blocks[f] : -1;
                    if (in == 0) *entry = blk;  // the block's first token
                    return blk;
                });
    if (blockIdx.x != 0) return;
    at = at0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (b0 + i < a.requests) {
            a.cu_seqlens[b0 + i] = cu[b0 + i];
            maps_state(a, b0 + i, n[i], r[i], at & 8191, held[i]);
        }
        at += (int64_t(r[i].take) << 13) + r[i].starts;
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if ((threadIdx.x & 31) == 0) longest_of[threadIdx.x >> 5] = longest;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        a.cu_seqlens[a.requests] = cu[kMost];
        for (int w = 1; w < kMapsThreads / 32; ++w) longest = max(longest, longest_of[w]);
        maps_totals(a, tokens, all >> 13, all & 8191, longest, bad);
    }
}

// More requests, first launch (one CTA): what there is of each request, the
// table entries among it.
__global__ void __launch_bounds__(kMapsManyThreads) batch_maps_requests_kernel(const BatchMapsArgs a) {
    __shared__ int64_t part[kMapsManyThreads / 32];
    __shared__ int64_t upto[kMapsManyThreads];  // new blocks of the group's requests up to and with this
    __shared__ int at[kMapsManyThreads];        // a request's first new entry
    after_earlier_work();
    let_next_begin();
    int64_t tokens = 0, blocks = 0, slots = 0;
    int longest = 0;
    bool bad = false;
    for (int g = 0; g < a.requests; g += kMapsManyThreads) {
        const int b = g + threadIdx.x;
        const bool on = b < a.requests;
        const int64_t want = on ? max(a.new_lens[b], 0) : 0;
        int64_t all;
        const int64_t w = tokens + maps_scan<kMapsManyThreads>(want, part, &all);
        tokens += all;
        const int64_t cap = a.max_tokens;
        const int lo = static_cast<int>(min(w, cap)), n = static_cast<int>(min(w + want, cap)) - lo;
        MapsRequest r{};
        if (on) r = maps_request(a, maps_ctx(a, b), n);
        bad |= r.too_long;
        longest = max(longest, n);
        const int64_t nth = slots + maps_scan<kMapsManyThreads>(r.starts, part, &all);
        slots += all;
        if (on) {
            a.cu_seqlens[b] = lo;
            maps_state(a, b, n, r, nth, a.request_slots[b]);
        }
        const int64_t f0 = maps_scan<kMapsManyThreads>(r.take, part, &all);
        upto[threadIdx.x] = f0 + r.take;
        at[threadIdx.x] = r.had;
        __syncthreads();
        for (int64_t e = threadIdx.x; e < all; e += kMapsManyThreads) {
            int i = 0;  // the request of the group's e-th new block: the first with upto > e
#pragma unroll
            for (int s = kMapsManyThreads / 2; s > 0; s /= 2)
                if (upto[i + s - 1] <= e) i += s;
            const int64_t k = e - (i > 0 ? upto[i - 1] : 0), f = blocks + e;
            a.block_tables[int64_t(g + i) * a.max_blocks + at[i] + k] =
                f < a.num_free_blocks ? a.free_blocks[f] : -1;
        }
        blocks += all;
        __syncthreads();
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if ((threadIdx.x & 31) == 0) at[threadIdx.x >> 5] = longest;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        for (int w = 1; w < kMapsManyThreads / 32; ++w) longest = max(longest, at[w]);
        a.cu_seqlens[a.requests] = static_cast<int>(min(tokens, int64_t(a.max_tokens)));
        maps_totals(a, tokens, blocks, slots, longest, bad);
    }
}

// More requests, second launch: the tokens.
__global__ void __launch_bounds__(kMapsThreads) batch_maps_tokens_kernel(const BatchMapsArgs a) {
    after_earlier_work();
    let_next_begin();
    maps_tokens(a, a.cu_seqlens, [&](int b) { return maps_ctx(a, b); }, (int64_t(blockIdx.x) * kMapsThreads + threadIdx.x) * kMapsTokens,
                [&](int b, int, int j, int) { return a.block_tables[int64_t(b) * a.max_blocks + j]; });
}

}  // namespace jssm
