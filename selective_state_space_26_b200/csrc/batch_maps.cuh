// batch_maps.cuh -- the maps of a continuous batch from its requests' lengths.
//
// Everything follows from three running sums over the requests: of the tokens
// that fit, of the cache blocks that a request needs beyond those it has, and
// of the requests that start and take a state slot.  The sums are a few
// thousand additions, so every CTA computes them for itself (the lengths come
// from L2) rather than one CTA computing them for the others, which would cost
// a second launch or a wait: the call is one launch.
#pragma once

#include "device_utils.cuh"

namespace jssm {

struct BatchMapsArgs {
    int requests, max_tokens, max_blocks, block_size;
    const int32_t *new_lens, *ctx_lens, *free_blocks, *free_slots;
    int num_free_blocks, num_free_slots;
    int32_t *block_tables, *request_slots, *cu_seqlens, *positions, *token_request;
    int64_t *slot_map;
    int32_t *state_indices, *initial_indices, *counts;
};

constexpr int kMapsThreads = 256;

struct MapsItem {
    int64_t tokens, blocks;
    int slots;
};

// One request's share, given the tokens before it.
struct MapsRequest {
    int n, want, ctx, had, take;
    bool starts, too_long;
};
__device__ __forceinline__ int ceil_div(int64_t v, int by) { return static_cast<int>((v + by - 1) / by); }
__device__ __forceinline__ MapsRequest maps_request(const BatchMapsArgs &a, int b, int64_t before) {
    MapsRequest r;
    r.want = max(a.new_lens[b], 0);
    r.ctx = a.ctx_lens ? max(a.ctx_lens[b], 0) : 0;
    r.n = static_cast<int>(min(max(int64_t(a.max_tokens) - before, int64_t(0)), int64_t(r.want)));
    r.had = min(ceil_div(r.ctx, a.block_size), a.max_blocks);
    const int need = r.n > 0 ? ceil_div(int64_t(r.ctx) + r.n, a.block_size) : r.had;
    r.too_long = need > a.max_blocks;
    r.take = max(min(need, a.max_blocks) - r.had, 0);
    r.starts = r.n > 0 && r.ctx == 0;
    return r;
}

// The simplest form: one thread.
__global__ void batch_maps_simple_kernel(const BatchMapsArgs a) {
    int64_t before = 0, blocks = 0;
    int slots = 0, longest = 0;
    bool bad = false;
    if (a.cu_seqlens) a.cu_seqlens[0] = 0;
    for (int b = 0; b < a.requests; ++b) {
        const MapsRequest r = maps_request(a, b, before);
        bad |= r.n < r.want || r.too_long;
        int32_t *table = a.block_tables + int64_t(b) * a.max_blocks;
        for (int j = 0; j < r.take; ++j) {
            const int64_t f = blocks + j;
            table[r.had + j] = f < a.num_free_blocks ? a.free_blocks[f] : -1;
            bad |= f >= a.num_free_blocks;
        }
        blocks += r.take;
        int slot = a.request_slots[b];
        if (r.starts) {
            slot = slots < a.num_free_slots ? a.free_slots[slots] : -1;
            bad |= slots >= a.num_free_slots;
            ++slots;
            a.request_slots[b] = slot;
        }
        a.state_indices[b] = r.n > 0 ? slot : -1;
        a.initial_indices[b] = r.n > 0 && !r.starts ? slot : -1;
        for (int i = 0; i < r.n; ++i) {
            const int64_t t = before + i;
            const int pos = r.ctx + i, j = pos / a.block_size;
            const int blk = j < a.max_blocks ? table[j] : -1;
            a.positions[t] = pos;
            a.token_request[t] = b;
            a.slot_map[t] = blk >= 0 ? int64_t(blk) * a.block_size + pos % a.block_size : -1;
        }
        before += r.n;
        a.cu_seqlens[b + 1] = static_cast<int>(before);
        longest = max(longest, r.n);
    }
    for (int64_t t = before; t < a.max_tokens; ++t) {
        a.positions[t] = -1;
        a.token_request[t] = -1;
        a.slot_map[t] = -1;
    }
    a.counts[0] = static_cast<int>(before);
    a.counts[1] = static_cast<int>(min(blocks, int64_t(a.num_free_blocks)));
    a.counts[2] = min(slots, a.num_free_slots);
    a.counts[3] = longest;
    if (bad) record_status(nullptr, kStInvalidArg);
}

}  // namespace jssm
