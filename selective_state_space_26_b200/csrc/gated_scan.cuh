// gated_scan.cuh -- the gated linear recurrence over whole sequences.
//
//   u_t = rate * sigmoid(g_t + bias),  h_t = h_{t-1} + u_t (x_t - h_{t-1}),
//   out_t = h_t silu(z_t)
//
// One thread walks one channel of one sequence.
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

template <typename T> __global__ void gated_scan_kernel(const GatedArgs a) {
    const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    const int b = static_cast<int>(i / a.d), c = static_cast<int>(i % a.d);
    if (b >= a.batch) return;
    int64_t row0, len;
    gated_rows(a, b, row0, len);
    int64_t in_row = b, out_row = b;
    if (a.state_indices) {
        out_row = gated_slot(a, a.state_indices[b], c == 0);
        in_row = a.initial_indices ? gated_slot(a, a.initial_indices[b], c == 0) : out_row;
    }
    float h = a.h0 && in_row >= 0 ? a.h0[in_row * a.d + c] : 0.0f;
    const float rate = a.rate ? a.rate[c] : 1.0f, bias = a.bias ? a.bias[c] : 0.0f;
    const T *x = static_cast<const T *>(a.x), *g = static_cast<const T *>(a.g),
            *z = static_cast<const T *>(a.z);
    T *out = static_cast<T *>(a.out);
    for (int64_t t = 0; t < len; ++t) {
        const int64_t r = row0 + t;
        if (a.ckpt && t % kGatedCkpt == 0)
            a.ckpt[(row0 / kGatedCkpt + b + t / kGatedCkpt) * a.d + c] = h;
        const float u = rate * sigmoid_f32(to_f32(g[r * a.gs + c]) + bias);
        h = fmaf(u, to_f32(x[r * a.xs + c]) - h, h);
        if (out) out[r * a.d + c] = from_f32<T>(z ? h * silu_f32(to_f32(z[r * a.zs + c])) : h);
    }
    if (a.h_final && out_row >= 0) a.h_final[out_row * a.d + c] = h;
}

// Backward: per 64-step block, last block first, the states again from the
// block's checkpoint, then the gradients in reverse.
template <typename T> __global__ void gated_scan_bwd_kernel(const GatedArgs a) {
    const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    const int b = static_cast<int>(i / a.d), c = static_cast<int>(i % a.d);
    if (b >= a.batch) return;
    int64_t row0, len;
    gated_rows(a, b, row0, len);
    const float rate = a.rate ? a.rate[c] : 1.0f, bias = a.bias ? a.bias[c] : 0.0f;
    const T *x = static_cast<const T *>(a.x), *g = static_cast<const T *>(a.g),
            *z = static_cast<const T *>(a.z), *dout = static_cast<const T *>(a.dout);
    T *dx = static_cast<T *>(a.dx), *dg = static_cast<T *>(a.dg), *dz = static_cast<T *>(a.dz);
    float carry = a.dh_final ? a.dh_final[int64_t(b) * a.d + c] : 0.0f;
    float drate = 0.0f, dbias = 0.0f;
    float hp[kGatedCkpt];
    for (int64_t k = (len + kGatedCkpt - 1) / kGatedCkpt - 1; k >= 0; --k) {
        const int64_t t0 = k * kGatedCkpt;
        const int n = static_cast<int>(min(int64_t(kGatedCkpt), len - t0));
        float h = a.ckpt[(row0 / kGatedCkpt + b + k) * a.d + c];
        for (int t = 0; t < n; ++t) {
            const int64_t r = row0 + t0 + t;
            hp[t] = h;
            h = fmaf(rate * sigmoid_f32(to_f32(g[r * a.gs + c]) + bias), to_f32(x[r * a.xs + c]) - h, h);
        }
        for (int t = n - 1; t >= 0; --t) {
            const int64_t r = row0 + t0 + t;
            const float s = sigmoid_f32(to_f32(g[r * a.gs + c]) + bias), u = rate * s;
            const float xv = to_f32(x[r * a.xs + c]), dv = to_f32(dout[r * a.d + c]);
            float gh = carry;
            if (z) {
                const float zv = to_f32(z[r * a.zs + c]), sz = sigmoid_f32(zv);
                const float ht = fmaf(u, xv - hp[t], hp[t]);
                gh += dv * (zv * sz);
                dz[r * a.d + c] = from_f32<T>(dv * ht * (sz * fmaf(zv, 1.0f - sz, 1.0f)));
            } else {
                gh += dv;
            }
            const float du = gh * (xv - hp[t]);
            const float dgv = du * u * (1.0f - s);
            dx[r * a.d + c] = from_f32<T>(u * gh);
            dg[r * a.d + c] = from_f32<T>(dgv);
            drate += du * s;
            dbias += dgv;
            carry = fmaf(-u, gh, gh);
        }
    }
    if (a.dh0) a.dh0[int64_t(b) * a.d + c] = carry;
    a.partial[int64_t(2 * b) * a.d + c] = drate;
    a.partial[int64_t(2 * b + 1) * a.d + c] = dbias;
}

// drate and dbias: the sequences' partial sums added in their order.
__global__ void gated_reduce_kernel(const float *partial, float *drate, float *dbias, int batch, int d) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= d) return;
    float r = 0.0f, s = 0.0f;
    for (int b = 0; b < batch; ++b) {
        r += partial[int64_t(2 * b) * d + c];
        s += partial[int64_t(2 * b + 1) * d + c];
    }
    if (drate) drate[c] = r;
    if (dbias) dbias[c] = s;
}

// One token for each request, one thread for each channel of it.
struct GatedUpdateArgs {
    float *state;
    const void *x, *g, *z;
    int64_t xs, gs, zs;
    const float *rate, *bias;
    void *out;
    const int32_t *state_indices;
    int64_t num_slots;
    int *status;
    int d, batch;
};
template <typename T> __global__ void gated_update_kernel(const GatedUpdateArgs a) {
    const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    const int64_t b = i / a.d;
    const int c = static_cast<int>(i % a.d);
    if (b >= a.batch) return;
    int64_t row = b;
    if (a.state_indices) {
        row = a.state_indices[b];
        if (row >= a.num_slots && c == 0) record_status(a.status, kStInvalidArg);
        if (row < 0 || row >= a.num_slots) return;
    }
    const float u = (a.rate ? a.rate[c] : 1.0f) *
                    sigmoid_f32(to_f32(static_cast<const T *>(a.g)[b * a.gs + c]) +
                                (a.bias ? a.bias[c] : 0.0f));
    float h = a.state[row * a.d + c];
    h = fmaf(u, to_f32(static_cast<const T *>(a.x)[b * a.xs + c]) - h, h);
    a.state[row * a.d + c] = h;
    static_cast<T *>(a.out)[b * a.d + c] =
        from_f32<T>(a.z ? h * silu_f32(to_f32(static_cast<const T *>(a.z)[b * a.zs + c])) : h);
}

}  // namespace jssm
