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

// Eight neighbouring elements; those from n on read as 0.
template <bool VECTOR> __device__ __forceinline__ void i8_load8(const __nv_bfloat16 *p, int n, float (&v)[8]) {
    if (VECTOR && n >= 8) {
        const uint4 r = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? __bfloat162float(p[i]) : 0.0f;
    }
}
template <bool VECTOR> __device__ __forceinline__ void i8_load8(const float *p, int n, float (&v)[8]) {
    if (VECTOR && n >= 8) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 r = reinterpret_cast<const float4 *>(p)[i];
            v[4 * i] = r.x, v[4 * i + 1] = r.y, v[4 * i + 2] = r.z, v[4 * i + 3] = r.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
    }
}

// LANES threads take a row, eight elements at a time; the first kKept of a
// thread's eights stay in registers between the two passes (every row of up to
// 8 * LANES * kKept elements is read once), the others are read again, from L2.
// VECTOR: rows begin at 16-byte boundaries.
constexpr int kQuantThreads = 256, kQuantKept = 4;
template <typename T, int LANES, bool VECTOR>
__global__ void __launch_bounds__(kQuantThreads) i8_quant_kernel(const I8QuantArgs a) {
    __shared__ uint32_t part[kQuantThreads / 32];
    const int64_t row = int64_t(blockIdx.x) * (kQuantThreads / LANES) + threadIdx.x / LANES;
    const int l = threadIdx.x % LANES;
    const bool on = row < a.rows;
    const T *x = static_cast<const T *>(a.x) + (on ? row : 0) * a.xs;
    const int k = on ? a.k : 0;
    float kept[kQuantKept][8];
    uint32_t m = 0;
    auto most = [&](const float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    };
#pragma unroll
    for (int j = 0; j < kQuantKept; ++j) {
        const int c = (j * LANES + l) * 8;
        i8_load8<VECTOR>(x + c, k - c, kept[j]);
        most(kept[j]);
    }
    for (int c = (kQuantKept * LANES + l) * 8; c < k; c += LANES * 8) {
        float v[8];
        i8_load8<VECTOR>(x + c, k - c, v);
        most(v);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if constexpr (LANES > 32) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
        __syncthreads();
        const int w0 = threadIdx.x / LANES * (LANES / 32);
#pragma unroll
        for (int w = 0; w < LANES / 32; ++w) m = max(m, part[w0 + w]);
    }
    if (!on) return;
    const I8Scale sc = i8_scale(m);
    if (l == 0) a.scale[row] = sc.scale;
    int8_t *q = a.q + row * a.pitch;
    auto put = [&](int c, const float (&v)[8]) {
        uint32_t w[2] = {0, 0};
        if (!sc.zero) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i / 4] |= (uint32_t(i8_round(v[i] * sc.up, sc.s, sc.inv)) & 0xffu) << (8 * (i % 4));
        }
        *reinterpret_cast<uint2 *>(q + c) = make_uint2(w[0], w[1]);
    };
#pragma unroll
    for (int j = 0; j < kQuantKept; ++j) {
        const int c = (j * LANES + l) * 8;
        if (c < a.pitch) put(c, kept[j]);
    }
    for (int c = (kQuantKept * LANES + l) * 8; c < a.pitch; c += LANES * 8) {
        float v[8];
        i8_load8<VECTOR>(x + c, k - c, v);
        put(c, v);
    }
}

}  // namespace jssm
