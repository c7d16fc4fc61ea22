// gated_update.cuh -- one token of the gated recurrence for each request, the
// state updated in place:
//   h <- h + u (x - h),  u = rate * sigmoid(g + bias),  out = h silu(z).
//
// A thread takes V neighbouring channels of one request: 8 bf16 or 4 fp32 (one
// 16-byte load each of x, g and z, two of the state for bf16) where rows begin
// at 16-byte boundaries, else 1.  Every byte moves once: 256 x 8192 bf16 from HBM
// take 7.6 us (4.4 TB/s, start and tail of one wave among it), 5.5 where L2 still
// holds a part; few requests are bound by the launch (5 x 1027 fp32: 1.6 us), so it
// begins while the work before it ends.
#pragma once

#include "device_utils.cuh"
#include "launch_order.cuh"
#include "s6_math.cuh"

namespace jssm {

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

template <typename T, int V> struct UpdateVec {
    __device__ __forceinline__ static void load(const T *p, float (&v)[V]) {
        if constexpr (V == 1) {
            v[0] = to_f32(*p);
        } else {
            const uint4 r = *reinterpret_cast<const uint4 *>(p);
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 2) {
                    v[2 * i] = __uint_as_float(w[i] << 16);
                    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                } else {
                    v[i] = __uint_as_float(w[i]);
                }
            }
        }
    }
    __device__ __forceinline__ static void store(T *p, const float (&v)[V]) {
        if constexpr (V == 1) {
            *p = from_f32<T>(v[0]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 2) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t *>(&h);
                } else {
                    w[i] = __float_as_uint(v[i]);
                }
            }
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    __device__ __forceinline__ static void load32(const float *p, float (&v)[V]) {
        if constexpr (V == 1) {
            v[0] = *p;
        } else {
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                const float4 r = reinterpret_cast<const float4 *>(p)[i];
                v[4 * i] = r.x, v[4 * i + 1] = r.y, v[4 * i + 2] = r.z, v[4 * i + 3] = r.w;
            }
        }
    }
    __device__ __forceinline__ static void store32(float *p, const float (&v)[V]) {
        if constexpr (V == 1) {
            *p = v[0];
        } else {
#pragma unroll
            for (int i = 0; i < V / 4; ++i)
                reinterpret_cast<float4 *>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
    }
};

constexpr int kUpdateThreads = 128;

// Block x: channels, block y (and on, by the grid's height): requests.
template <typename T, int V>
__global__ void __launch_bounds__(kUpdateThreads) gated_update_kernel(const GatedUpdateArgs a) {
    using U = UpdateVec<T, V>;
    const int c = (blockIdx.x * kUpdateThreads + threadIdx.x) * V;
    after_earlier_work();
    let_next_begin();
    if (c >= a.d) return;
    float rate[V], bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i) rate[i] = 1.0f, bias[i] = 0.0f;
    if (a.rate) U::load32(a.rate + c, rate);
    if (a.bias) U::load32(a.bias + c, bias);
    for (int64_t b = blockIdx.y; b < a.batch; b += gridDim.y) {
        int64_t row = b;
        if (a.state_indices) {
            row = a.state_indices[b];
            if (row >= a.num_slots && c == 0) record_status(a.status, kStInvalidArg);
            if (row < 0 || row >= a.num_slots) continue;
        }
        float *state = a.state + row * a.d + c;
        float x[V], g[V], z[V], h[V];
        U::load(static_cast<const T *>(a.x) + b * a.xs + c, x);
        U::load(static_cast<const T *>(a.g) + b * a.gs + c, g);
        if (a.z) U::load(static_cast<const T *>(a.z) + b * a.zs + c, z);
        U::load32(state, h);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float u = rate[i] * rcp_mufu(1.0f + ex2_mufu(-(g[i] + bias[i]) * kLog2e));
            h[i] = fmaf(u, x[i] - h[i], h[i]);
        }
        U::store32(state, h);
        if (a.z)
#pragma unroll
            for (int i = 0; i < V; ++i) h[i] *= silu_f32(z[i]);
        U::store(static_cast<T *>(a.out) + b * a.d + c, h);
    }
}

}  // namespace jssm
