// i8_quant.cuh -- rows to 8 bits, each with its own scale:
//   scale = max|x| / 127,  q = x / scale rounded to the nearest integer.
#pragma once

#include "device_utils.cuh"

namespace jssm {

struct I8QuantArgs {
    const void *x;
    int64_t xs;  // row stride in elements
    int8_t *q;
    float *scale;
    int64_t rows;
    int k, pitch;
};

// The nearest integer (ties to even) of the exact quotient x / s, given inv =
// 1 / s rounded.  x * inv is within 2^-22 relative of the quotient, so its
// floor m has m + 1/2 as the only half-integer that can matter, and the sign of
// x - (m + 1/2) s, which one FMA gives exactly, says on which side of it the
// quotient lies.  (x * inv alone rounds the common case max/2, whose quotient
// is next to 63.5, by chance.)
__device__ __forceinline__ int i8_round(float x, float s, float inv) {
    const float m = floorf(x * inv);
    const float t = fmaf(-(m + 0.5f), s, x);
    const int i = static_cast<int>(m);
    const int q = t > 0.0f ? i + 1 : t < 0.0f ? i : i + (i & 1);
    return min(max(q, -127), 127);
}

// Of a row's largest |x| (as bits, so that an infinity or a NaN is above all
// finite values): the stored scale, and the factors for i8_round.  Rows of tiny
// values are raised by 2^100 first, or 1 / s would overflow and the FMA's
// result underflow.
struct I8Scale {
    float scale, up, s, inv;
    bool zero;  // q is 0 throughout
};
__device__ __forceinline__ I8Scale i8_scale(uint32_t amax_bits) {
    I8Scale r;
    const float amax = __uint_as_float(amax_bits);
    r.scale = amax_bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __fdiv_rn(amax, 127.0f);
    r.up = amax < 0x1p-60f ? 0x1p100f : 1.0f;
    r.s = r.scale * r.up;
    r.inv = __fdiv_rn(1.0f, r.s);
    r.zero = !(r.scale > 0.0f);
    return r;
}

template <typename T> __global__ void i8_quant_kernel(const I8QuantArgs a) {
    __shared__ uint32_t part[4];
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.xs;
    uint32_t m = 0;
    for (int c = threadIdx.x; c < a.k; c += 128)
        m = max(m, __float_as_uint(to_f32(x[c])) & 0x7fffffffu);
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    m = max(max(part[0], part[1]), max(part[2], part[3]));
    const I8Scale sc = i8_scale(m);
    if (threadIdx.x == 0) a.scale[row] = sc.scale;
    int8_t *q = a.q + row * a.pitch;
    for (int c = threadIdx.x; c < a.pitch; c += 128)
        q[c] = c < a.k && !sc.zero ? static_cast<int8_t>(i8_round(to_f32(x[c]) * sc.up, sc.s, sc.inv))
                                   : int8_t(0);
}

}  // namespace jssm
