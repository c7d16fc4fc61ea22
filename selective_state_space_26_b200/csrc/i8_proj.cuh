// i8_proj.cuh -- the 8-bit product with a scale for each token and each output
// channel: out = (q . w) q_scale w_scale + bias.
#pragma once

#include "device_utils.cuh"

namespace jssm {

struct I8ProjArgs {
    const int8_t *q, *w;
    const float *qs, *ws, *bias;
    void *out;
    int64_t ntok;
    int n, pitch;
};

// acc * s * w with the smaller scale first: acc * (the larger) could overflow
// where the whole product does not.  A NaN scale stays one.
__device__ __forceinline__ float i8_scaled(int acc, float s, float w) {
    const bool less = s < w;
    return static_cast<float>(acc) * (less ? s : w) * (less ? w : s);
}

// One thread for each output.
template <typename T> __global__ void i8_proj_simple_kernel(const I8ProjArgs a) {
    const int o = blockIdx.x * 32 + threadIdx.x;
    const int64_t t = int64_t(blockIdx.y) * 8 + threadIdx.y;
    if (o >= a.n || t >= a.ntok) return;
    const int *q = reinterpret_cast<const int *>(a.q + t * a.pitch);
    const int *w = reinterpret_cast<const int *>(a.w + int64_t(o) * a.pitch);
    int acc = 0;
    for (int k = 0; k < a.pitch / 4; ++k) acc = __dp4a(q[k], w[k], acc);
    float v = i8_scaled(acc, a.qs[t], a.ws[o]);
    if (a.bias) v += a.bias[o];
    static_cast<T *>(a.out)[t * a.n + o] = from_f32<T>(v);
}

}  // namespace jssm
