// i8_quant.cuh -- rows to 8 bits, each with its own scale:
//   scale = max|x| / 127,  q = x / scale rounded to the nearest integer.
#pragma once

#include "device_utils.cuh"
#include "launch_order.cuh"

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

// Two at once.  Adding 1.5 * 2^23 rounds to the nearest integer and leaves it in
// the low bits: no conversion instruction, which would run at an eighth of the
// rate.  Right wherever y = x * inv is not within 2^-12 of a half (its error is
// below 2^-15 for |y| <= 128); `off`, the largest distance from the integer,
// shows where it is.
__device__ __forceinline__ float2 i8_round_fast(float2 x, float inv, float &off) {
    const float big = 12582912.0f;
    const float2 y = mul2(x, make_float2(inv, inv)), one = make_float2(1.0f, 1.0f);
    const float2 t = fma2(y, one, make_float2(big, big)), r = fma2(t, one, make_float2(-big, -big));
    const float2 d = fma2(r, make_float2(-1.0f, -1.0f), y);
    off = fmaxf(off, fmaxf(fabsf(d.x), fabsf(d.y)));
    return t;
}
// The low bytes of four words.
__device__ __forceinline__ uint32_t i8_pack(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Of a row's largest |x|, as bits: the stored scale, and the factors for
// i8_round.  Rows of tiny values are raised by 2^100 first, or 1 / s would
// overflow and the FMA's result underflow.
struct I8Scale {
    float scale, up, s, inv;
    bool zero;  // q is 0 throughout
};
__device__ __forceinline__ I8Scale i8_scale(uint32_t bits) {
    I8Scale r;
    const float amax = __uint_as_float(bits);
    r.scale = bits < 0x7f800000u ? __fdiv_rn(amax, 127.0f) : __uint_as_float(0x7fc00000u);
    r.up = amax < 0x1p-60f ? 0x1p100f : 1.0f;
    r.s = r.scale * r.up;
    r.inv = __fdiv_rn(1.0f, r.s);
    r.zero = !(r.scale > 0.0f);
    return r;
}

// Eight neighbouring elements as they lie in memory; those from n on are 0.
template <typename T> struct I8Eight;
template <> struct I8Eight<__nv_bfloat16> {
    uint32_t w[4];
    template <bool VECTOR> __device__ __forceinline__ void load(const __nv_bfloat16 *p, int n) {
        if (VECTOR && n >= 8) {
            const uint4 r = *reinterpret_cast<const uint4 *>(p);
            w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
        } else {
            const uint16_t *u = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = (2 * i < n ? uint32_t(u[2 * i]) : 0u) | (2 * i + 1 < n ? uint32_t(u[2 * i + 1]) << 16 : 0u);
        }
    }
    // The largest |element| so far, as bits, in two halves of a word: an infinity
    // or a NaN is above all finite values.
    __device__ __forceinline__ uint32_t most(uint32_t m) const {
#pragma unroll
        for (int i = 0; i < 4; i += 2)
            m = __vimax3_u16x2(m, w[i] & 0x7fff7fffu, w[i + 1] & 0x7fff7fffu);
        return m;
    }
    static __device__ __forceinline__ uint32_t bits(uint32_t m) { return max(m << 16, m & 0xffff0000u); }
    __device__ __forceinline__ float2 pair(int i) const {
        return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
};
template <> struct I8Eight<float> {
    float v[8];
    template <bool VECTOR> __device__ __forceinline__ void load(const float *p, int n) {
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
    __device__ __forceinline__ uint32_t most(uint32_t m) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
        return m;
    }
    static __device__ __forceinline__ uint32_t bits(uint32_t m) { return m; }
    __device__ __forceinline__ float2 pair(int i) const { return make_float2(v[2 * i], v[2 * i + 1]); }
};

// LANES threads take a row, eight elements at a time; the first kKept of a
// thread's eights stay in registers between the two passes (every row of up to
// 8 * LANES * kKept elements is read once), the others are read again, from L2.
// VECTOR: rows begin at 16-byte boundaries.  4096 x 4096 bf16: 13.3 us, 3.8 TB/s;
// bound by the arithmetic, about 6 instructions an element (with floor and
// convert instructions in their place 19 us).
constexpr int kQuantThreads = 256, kQuantKept = 4;
template <typename T, int LANES, bool VECTOR>
__global__ void __launch_bounds__(kQuantThreads) i8_quant_kernel(const I8QuantArgs a) {
    using E = I8Eight<T>;
    __shared__ uint32_t part[kQuantThreads / 32];
    const int64_t row = int64_t(blockIdx.x) * (kQuantThreads / LANES) + threadIdx.x / LANES;
    const int l = threadIdx.x % LANES;
    const bool on = row < a.rows;
    const T *x = static_cast<const T *>(a.x) + (on ? row : 0) * a.xs;
    const int k = on ? a.k : 0;
    E kept[kQuantKept];
    uint32_t m = 0;
    after_earlier_work();
    let_next_begin();
#pragma unroll
    for (int j = 0; j < kQuantKept; ++j) {
        const int c = (j * LANES + l) * 8;
        kept[j].template load<VECTOR>(x + c, k - c);
    }
#pragma unroll
    for (int j = 0; j < kQuantKept; ++j) m = kept[j].most(m);
    for (int c = (kQuantKept * LANES + l) * 8; c < k; c += LANES * 8) {
        E v;
        v.template load<VECTOR>(x + c, k - c);
        m = v.most(m);
    }
    m = __reduce_max_sync(0xffffffffu, E::bits(m));
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
    auto put = [&](int c, const E &v) {
        uint32_t w[2] = {0, 0};
        if (!sc.zero) {
            float off = sc.up != 1.0f ? 1.0f : 0.0f;
            uint32_t t[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 r = i8_round_fast(v.pair(i), sc.inv, off);
                t[2 * i] = __float_as_uint(r.x);
                t[2 * i + 1] = __float_as_uint(r.y);
            }
            if (off > 0.5f - 0x1p-12f)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    t[2 * i] = uint32_t(i8_round(v.pair(i).x * sc.up, sc.s, sc.inv));
                    t[2 * i + 1] = uint32_t(i8_round(v.pair(i).y * sc.up, sc.s, sc.inv));
                }
            w[0] = i8_pack(t[0], t[1], t[2], t[3]);
            w[1] = i8_pack(t[4], t[5], t[6], t[7]);
        }
        *reinterpret_cast<uint2 *>(q + c) = make_uint2(w[0], w[1]);
    };
#pragma unroll
    for (int j = 0; j < kQuantKept; ++j) {
        const int c = (j * LANES + l) * 8;
        if (c < a.pitch) put(c, kept[j]);
    }
    for (int c = (kQuantKept * LANES + l) * 8; c < a.pitch; c += LANES * 8) {
        E v;
        v.template load<VECTOR>(x + c, k - c);
        put(c, v);
    }
}

}  // namespace jssm
