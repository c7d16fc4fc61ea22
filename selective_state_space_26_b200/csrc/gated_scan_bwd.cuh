// gated_scan_bwd.cuh -- the gated recurrence's backward pass.
//
// With gh_t = dL/dh_t and s = sigmoid(g + bias), u = rate s:
//   gh_t = dout_t silu(z_t) + c_{t+1},   c_t = (1 - u_t) gh_t   (the gradient of h_{t-1}),
//   dx = u gh,  du = gh (x - h_{t-1}),  dg = du u (1 - s),  dz = dout h silu'(z),
//   drate = sum du s,  dbias = sum dg.
//
// c runs backwards through the sequence as the state runs forwards: a run of
// rows maps the c behind it to P c + R with the same P = prod(1 - u), held as the
// scan's maps hold it, and runs compose.  So the kernel is the scan's with the order reversed: a lane takes a
// run of 8 rows, a warp Q runs, a CTA's 8 warps a chunk of 64 Q rows, a cluster
// consecutive chunks, from the sequence's end to its start.  The states that du
// and dz need come from the forward's checkpoints, one for every 64 rows, so
// they need no exchange beyond the 64 rows' own runs.  One barrier a round
// carries both directions' maps.  dz is written on the way forward through a
// run, dx and dg on the way back; the sums of drate and dbias stay in registers
// and are added over runs, warps, the cluster and, in a second small launch,
// the sequences, each in a fixed order.
//
// It reads x, g, z and dout once and writes dx, dg and dz once: with the
// forward and its checkpoints, 8 x 2048 x 4096 bf16 take 302 us (4.9 TB/s, 75%
// of a plain copy), 2 x 4096 x 4096, whose 256 CTAs leave an SM two at most, 169.
// What bounds it is latency at the 16 warps an SM that 128 registers leave: a row
// and warp takes 123 instructions, and 56% of the issue slots are used.  Before the
// maps held P - 1 (292 and 166 us): runs of 16 rows on 4 warps (381 and 209) spread
// the exchange over more rows but leave half the warps to hide each other's latency;
// testing a row for the run's end inside the loops costs 328 and 179.
#pragma once

#include "gated_scan.cuh"
#include "launch_order.cuh"

namespace jssm {

constexpr int kGatedBwdWarps = 8, kGatedBwdRun = 8, kGatedBwdThreads = 32 * kGatedBwdWarps;
static_assert(kGatedBwdWarps * kGatedBwdRun == kGatedCkpt, "W / Q warps take a checkpoint's rows");

struct Yes {
    static constexpr bool value = true;
};
struct No {
    static constexpr bool value = false;
};

template <bool GATE> struct GatedBwdCfg {
    static constexpr int kArrays = GATE ? 4 : 3;
    static constexpr int kArrayBytes = kGatedBwdRun * 128;
    static constexpr int kStageBytes = kArrays * kArrayBytes;
    static constexpr int kSmemBytes = kGatedBwdWarps * 2 * kStageBytes;
};

#pragma nv_diag_suppress 549  // s[i] and dy[i] are set just before `ahead` reads them
template <typename T, int VEC, bool GATE, int Q, int CP, bool CLUSTER>
__global__ void __launch_bounds__(kGatedBwdThreads, 2) gated_scan_bwd_kernel(const GatedArgs a, int cs) {
    using Raw = GatedRaw<T, VEC>;
    using R = typename Raw::type;
    using C = GatedBwdCfg<GATE>;
    using L = Lane<VEC>;
    using Map = RunMap<VEC>;
    constexpr int S = kGatedBwdRun, W = kGatedBwdWarps, LPR = 32 / Q, kChunk = W * S * Q;
    constexpr int kBlockWarps = W / Q;  // warps of a checkpoint's 64 rows
    using F = GatedFeed<T, VEC, S, Q, CP>;
    extern __shared__ __align__(128) uint8_t stages[];
    __shared__ Map runs[2][W][LPR];   // (P, b): the states' direction
    __shared__ L back[2][W][LPR];     // R: the gradients' direction
    __shared__ Map chunks[CLUSTER ? 2 : 1][CLUSTER ? kGatedMaxCluster : 1][LPR];
    __shared__ L last[2][LPR];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = lane % LPR, run = lane / LPR;
    if (!CLUSTER) cs = 1;
    if (CLUSTER) cluster_arrive();  // waited for before the first store to another CTA
    const int rank = CLUSTER ? static_cast<int>(cluster_rank()) : 0;
    const int tiles = (a.d + LPR * VEC - 1) / (LPR * VEC);
    const int64_t unit = blockIdx.x / cs;
    __shared__ int order[kGatedBwdThreads + 1];
    const int b = gated_sequence<kGatedBwdThreads>(a, static_cast<int>(unit / tiles), order);
    const int c0 = static_cast<int>(unit % tiles) * LPR * VEC, c = c0 + col * VEC;
    const bool on = c < a.d;

    int64_t row0, len64;
    gated_rows(a, b, row0, len64);
    const int len = static_cast<int>(len64);
    const int stride = cs * kChunk;
    const int rounds = (len + stride - 1) / stride;
    int t = (rounds - 1) * stride + rank * kChunk + warp * (S * Q);  // this warp's first row
    uint8_t *const mine = stages + warp * (2 * C::kStageBytes);
    const bool in = c0 + F::channel_of(lane) < a.d;
    F fg, fx, fz, fd;
    fg.start(a.g, row0 + t, a.gs, c0, lane, -stride);
    fx.start(a.x, row0 + t, a.xs, c0, lane, -stride);
    fd.start(a.dout, row0 + t, a.d, c0, lane, -stride);
    if (GATE) fz.start(a.z, row0 + t, a.zs, c0, lane, -stride);
    auto fill = [&](int at, int stage) {  // at: the copied round's first row
        if (at >= 0 && at < len) {
            const uint32_t to = smem_u32(mine) + stage * C::kStageBytes;
            const int n = min(len - at, S * Q);
            fg.copy(to, in, n, lane);
            fx.copy(to + C::kArrayBytes, in, n, lane);
            fd.copy(to + 2 * C::kArrayBytes, in, n, lane);
            if (GATE) fz.copy(to + 3 * C::kArrayBytes, in, n, lane);
        } else {
            fg.skip(), fx.skip(), fd.skip();
            if (GATE) fz.skip();
        }
        cp_async_commit();
    };
    fill(t, 0);
    fill(t - stride, 1);

    L carry, rate, bias;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        carry.set(v, on && a.dh_final ? a.dh_final[int64_t(b) * a.d + c + v] : 0.0f);
        rate.set(v, on && a.rate ? a.rate[c + v] : 1.0f);
        bias.set(v, on && a.bias ? a.bias[c + v] : 0.0f);
    }
    const L one = L::of(1.0f), zero = L::of(0.0f), held = L::of(kHeld), nrate = lmul(rate, L::of(-1.0f));
    L drate = zero, dbias = zero;
    const float *ck = a.ckpt + (row0 / kGatedCkpt + b) * a.d + c;  // the sequence's first entry
    auto checkpoint = [&](int at) {  // the state before the 64 rows around row `at`
        L h = zero;
#pragma unroll
        for (int v = 0; v < VEC; ++v)
            if (on && at >= 0 && at < len) h.set(v, ck[int64_t(at / kGatedCkpt) * a.d + v]);
        return h;
    };
    L block = checkpoint(t);
    int64_t o0 = (row0 + t + run * S) * a.d + c;  // the lane's first output
    if (CLUSTER) cluster_wait();  // every CTA of the cluster has started
    for (int k = 0; k < rounds; ++k, t -= stride) {
        const int par = k & 1;
        const bool full = len - t >= S * Q;
        const int n = min(len - t - run * S, S);  // rows of this lane's run
        uint8_t *st = mine + par * C::kStageBytes;
        const R *gr = reinterpret_cast<const R *>(st) + lane;
        const R *xr = reinterpret_cast<const R *>(st + C::kArrayBytes) + lane;
        const R *dr = reinterpret_cast<const R *>(st + 2 * C::kArrayBytes) + lane;
        // x - h_{t-1} takes the place of g and x once they have been used
        float *d0 = reinterpret_cast<float *>(st) + lane;
        float *d1 = reinterpret_cast<float *>(st + C::kArrayBytes) + lane;
        const R *zr = reinterpret_cast<const R *>(st + 3 * C::kArrayBytes) + lane;
        const L next_block = checkpoint(t - stride);
        cp_async_wait<1>();
        __syncwarp();
        // the run's maps: of the state, P h + hb, and of the gradient, P c + rb.  The
        // latter is a sum forwards too: row i's dy reaches the rows before the run
        // through the product of (1 - u) up to and with its own.
        L s[S], dy[S], P = one, pn = zero, hb = zero, rb = zero;  // dy holds sigmoid(z) until z has been used
        auto ahead = [&](int i) {
            const L nu = lmul(s[i], nrate);
            hb = lfma(nu, lsub(hb, Raw::get(xr[i * 32])), hb);
            pn = lfma(nu, P, pn);
            P = lfma(nu, P, P);
            L d = Raw::get(dr[i * 32]);
            if (GATE) d = lmul(d, lmul(Raw::get(zr[i * 32]), dy[i]));
            rb = lfma(P, d, rb);
        };
        bool good = full;
        if (full) {
#pragma unroll
            for (int i = 0; i < S; ++i) {
                s[i] = lsigmoid_pair(ladd(Raw::get(gr[i * 32]), bias), good);
                if (GATE) dy[i] = lsigmoid_pair(Raw::get(zr[i * 32]), good);
                ahead(i);
            }
        }
        if (!good && on) {
            P = one, pn = hb = rb = zero;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                if (i < n) {
                    s[i] = lsigmoid(ladd(Raw::get(gr[i * 32]), bias));
                    if (GATE) dy[i] = lsigmoid(Raw::get(zr[i * 32]));
                    ahead(i);
                }
            }
        }
        // the warp's runs before and behind this one; P and both totals over the warp
        const L q = ldecay(P, pn);
        L bp = held, bb = zero, ap = held, ab = zero, wp = q, wb = hb, wr = rb;
        if constexpr (Q > 1) {
            L ip = q, ib = hb;
#pragma unroll
            for (int by = LPR; by < 32; by *= 2) {
                const L op = lshfl_up(ip, by), ob = lshfl_up(ib, by);
                if (lane >= by) {
                    ib = lapply(ip, ob, ib);
                    ip = ljoin(ip, op);
                }
            }
            const L ep = lshfl_up(ip, LPR), eb = lshfl_up(ib, LPR);
            if (run > 0) bp = ep, bb = eb;
            L jp = q, jr = rb;
#pragma unroll
            for (int by = LPR; by < 32; by *= 2) {
                const L op = lshfl_down(jp, by), orr = lshfl_down(jr, by);
                if (lane + by < 32) {
                    jr = lapply(jp, orr, jr);
                    jp = ljoin(jp, op);
                }
            }
            const L fp = lshfl_down(jp, LPR), fr = lshfl_down(jr, LPR);
            if (run < Q - 1) ap = fp, ab = fr;
            wp = ip, wb = ib;  // of the whole warp on the last run's lanes
            wr = jr;           // and on the first run's
        }
        if (run == Q - 1) runs[par][warp][col] = Map::of(wp, wb);
        if (run == 0) back[par][warp][col] = wr;
        __syncthreads();
        // the state before this run: the block's checkpoint through the runs between
        L h = block;
        const int w0 = warp / kBlockWarps * kBlockWarps;
        Map maps[W];
        L backs[W];
#pragma unroll
        for (int w = 0; w < W; ++w) maps[w] = runs[par][w][col], backs[w] = back[par][w][col];
#pragma unroll
        for (int w = 0; w < W - 1; ++w)
            if (w >= w0 && w < warp) h = lapply(maps[w].q(), h, maps[w].b());
        if (Q > 1) h = lapply(bp, h, bb);
        // c behind this warp's rows
        L cb;
        if constexpr (CLUSTER) {
            L mp = held;
            cb = zero;
#pragma unroll
            for (int w = W - 1; w > 0; --w) {
                if (w > warp) {
                    cb = lapply(maps[w].q(), cb, backs[w]);
                    mp = ljoin(maps[w].q(), mp);
                }
            }
            if (warp == 0 && run == 0) {  // the chunk's map to every CTA of the cluster
                const L p = maps[0].q();
                const Map m = Map::of(ljoin(p, mp), lapply(p, cb, wr));
                const uint32_t at = smem_u32(&chunks[par][rank][col]);
#pragma unroll
                for (int r = 0; r < kGatedMaxCluster; ++r)
                    if (r < cs) st_cluster(at, r, m);
            }
            __syncwarp();
            cluster_arrive();
            cluster_wait();
            L behind = carry;
#pragma unroll
            for (int r = kGatedMaxCluster - 1; r >= 0; --r) {
                if (r == rank) behind = carry;
                if (r < cs) {
                    const Map m = chunks[par][r][col];
                    carry = lapply(m.q(), carry, m.b());
                }
            }
            cb = lapply(mp, behind, cb);
        } else {
            if (k > 0) carry = last[par][col];
            cb = carry;
#pragma unroll
            for (int w = W - 1; w > 0; --w)
                if (w > warp) cb = lapply(maps[w].q(), cb, backs[w]);
            if (warp == 0 && run == 0) last[par ^ 1][col] = lapply(maps[0].q(), cb, wr);
        }
        if (Q > 1) cb = lapply(ap, cb, ab);  // behind this run
        L sr = zero, sg = zero;
        auto rest = [&](auto whole) {  // whole: every row and channel of the run is there
            constexpr bool kWhole = decltype(whole)::value;
            // forwards again from the true state: dz, and x - h_{t-1}
            T *dz = static_cast<T *>(a.dz) + o0;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                if (kWhole || i < n) {
                    const L diff = lsub(Raw::get(xr[i * 32]), h);
                    h = lfma(lmul(s[i], rate), diff, h);
                    L d = Raw::get(dr[i * 32]);
                    if (GATE) {
                        // silu' = sz + z sz (1 - sz)
                        const L sz = dy[i], zs = lmul(Raw::get(zr[i * 32]), sz);
                        const L slope = lfma(lsub(one, sz), zs, sz);
                        const R v = Raw::put(lmul(lmul(d, h), slope));
                        if (kWhole || on) *reinterpret_cast<R *>(dz) = v;
                        d = lmul(d, zs);
                    }
                    dy[i] = d;
                    d0[i * 32] = diff.get(0);
                    if constexpr (VEC == 2) d1[i * 32] = diff.get(1);
                }
                if (GATE) dz += a.d;
            }
            // and back: dx, dg and the sums
            T *dx = static_cast<T *>(a.dx) + o0 + int64_t(S) * a.d;
            T *dg = static_cast<T *>(a.dg) + o0 + int64_t(S) * a.d;
#pragma unroll
            for (int i = S - 1; i >= 0; --i) {
                dx -= a.d, dg -= a.d;
                if (kWhole || i < n) {
                    L diff;
                    diff.set(0, d0[i * 32]);
                    if constexpr (VEC == 2) diff.set(1, d1[i * 32]);
                    const L gh = ladd(dy[i], cb);
                    const L x = lmul(lmul(s[i], rate), gh), du = lmul(gh, diff);
                    const L dus = lmul(du, s[i]);
                    const L g = lmul(lmul(dus, rate), lsub(one, s[i]));
                    sr = ladd(sr, dus);
                    sg = ladd(sg, g);
                    cb = lsub(gh, x);
                    const R xr2 = Raw::put(x), gr2 = Raw::put(g);
                    if (kWhole || on) {
                        *reinterpret_cast<R *>(dx) = xr2;
                        *reinterpret_cast<R *>(dg) = gr2;
                    }
                }
            }
        };
        if (full && on)
            rest(Yes{});
        else
            rest(No{});
        drate = ladd(drate, sr);
        dbias = ladd(dbias, sg);
        o0 -= int64_t(stride) * a.d;
        block = next_block;
        __syncwarp();  // every lane has read the stage that the next copy overwrites
        fill(t - 2 * stride, par);
    }
    cp_async_wait<0>();
    // the sums: runs of a warp, warps, ranks
#pragma unroll
    for (int by = LPR; by < 32; by *= 2) {
        drate = ladd(drate, lshfl_down(drate, by));
        dbias = ladd(dbias, lshfl_down(dbias, by));
    }
    if (!CLUSTER && rounds > 0) {
        __syncthreads();
        carry = last[rounds & 1][col];
    }
    __syncthreads();  // runs[] has been read
    if (run == 0) runs[0][warp][col] = Map::of(drate, dbias);
    __syncthreads();
    if (warp == 0 && run == 0) {
        drate = dbias = zero;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const Map r = runs[0][w][col];
            drate = ladd(drate, r.q());
            dbias = ladd(dbias, r.b());
        }
    }
    if constexpr (CLUSTER) {
        // the ranks' sums to rank 0; nobody's maps are read any more after this barrier
        cluster_arrive();
        cluster_wait();
        if (warp == 0 && run == 0)
            st_cluster(smem_u32(&chunks[0][rank][col]), 0, Map::of(drate, dbias));
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (warp == 0 && run == 0) {
            drate = dbias = zero;
            for (int r = 0; r < cs; ++r) {
                const Map m = chunks[0][r][col];
                drate = ladd(drate, m.q());
                dbias = ladd(dbias, m.b());
            }
        }
    }
    if (rank == 0 && warp == 0 && run == 0 && on) {
        float *pr = a.partial ? a.partial + int64_t(2 * b) * a.d : a.drate;
        float *pb = a.partial ? a.partial + int64_t(2 * b + 1) * a.d : a.dbias;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            if (a.dh0) a.dh0[int64_t(b) * a.d + c + v] = carry.get(v);
            if (pr) pr[c + v] = drate.get(v);
            if (pb) pb[c + v] = dbias.get(v);
        }
    }
}

// drate and dbias: the sequences' sums added in their order.
__global__ void gated_reduce_kernel(const float *partial, float *drate, float *dbias, int batch, int d) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    after_earlier_work();
    let_next_begin();
    if (c >= d) return;
    double r = 0.0, s = 0.0;
    for (int b = 0; b < batch; ++b) {
        r += partial[int64_t(2 * b) * d + c];
        s += partial[int64_t(2 * b + 1) * d + c];
    }
    if (drate) drate[c] = static_cast<float>(r);
    if (dbias) dbias[c] = static_cast<float>(s);
}

}  // namespace jssm
