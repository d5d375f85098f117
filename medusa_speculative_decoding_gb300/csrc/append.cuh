// append.cuh -- what the kernels share that write rows into the 8-bit paged cache: rows
// as they were loaded, the choice of a page's scale, and conversions to the nearest code
// of an exact quotient.
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "q8.cuh"

namespace medusa {
namespace append {

// Eight neighbouring elements of a row, as they were loaded.
struct Bf16x8 {
    uint4 w;
    __device__ __forceinline__ void load(const uint16_t* p) { w = ld_stream16(p); }
    // where the same kernel writes there later
    __device__ __forceinline__ void load_plain(const uint16_t* p) { w = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void unpack(float (&x)[8]) const {
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) { x[2 * i] = bf16_lo(v[i]); x[2 * i + 1] = bf16_hi(v[i]); }
    }
    // largest |x|, NaN left out
    __device__ __forceinline__ float top() const {
        const uint32_t m = max_abs2(max_abs2(w.x, w.y), max_abs2(w.z, w.w));
        return fmaxf(fmaxf(fabsf(bf16_lo(m)), fabsf(bf16_hi(m))), 0.f);
    }
    // the larger of the magnitudes, pair by pair, under some sign
    static __device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
};
struct F32x8 {
    uint4 w[2];
    __device__ __forceinline__ void load(const float* p) { w[0] = ld_stream16(p); w[1] = ld_stream16(p + 4); }
    __device__ __forceinline__ void load_plain(const float* p) {
        w[0] = *reinterpret_cast<const uint4*>(p);
        w[1] = *reinterpret_cast<const uint4*>(p + 4);
    }
    __device__ __forceinline__ void unpack(float (&x)[8]) const {
        const uint32_t v[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(v[i]);
    }
    __device__ __forceinline__ float top() const {
        float x[8], m = 0.f;
        unpack(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
        return m;
    }
};
// largest finite |x| of a page's share, once some |x| is infinite
template <typename Raw>
__device__ __forceinline__ float finite_top(const Raw& x) {
    float y[8], top = 0.f;
    x.unpack(y);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (fabsf(y[e]) < INFINITY) top = fmaxf(top, fabsf(y[e]));
    return top;
}
template <typename T> struct Raw8;
template <> struct Raw8<uint16_t> { using type = Bf16x8; };
template <> struct Raw8<float> { using type = F32x8; };

// the smallest 2^e with top <= MOST * 2^e, e held to [-64, 64]
template <int MOST>
__device__ __forceinline__ float page_scale(float top) {
    static_assert(MOST >= 256 && MOST < 512, "the leading bit of MOST is 2^8");
    if (!(top > 0.f)) return q8::kMinScale;
    const uint32_t u = __float_as_uint(top);
    int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > (uint32_t)(MOST - 256) << 15 ? 1 : 0);
    if ((u >> 23) == 0) e = -64;  // subnormal
    e = q8::clamp_int(e, -64, 64);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// q is a quotient or product rounded to float32, r what the exact one lies above it: the
// exact one's neighbour with an odd last bit (or itself).  The middle of two codes ends in
// zeros, so rounding the result to a code is rounding the exact value.
__device__ __forceinline__ float to_odd(float q, float r) {
    uint32_t u = __float_as_uint(q);
    if (r != 0.f) {
        if ((r < 0.f) != (q < 0.f)) u -= 1;  // towards zero first
        u |= 1;
    }
    return __uint_as_float(u);
}
__device__ __forceinline__ float divide_to_odd(float x, float s) {
    const float q = x / s;
    // (below, the code is zero whatever the bits; above, it is held at 448)
    return fabsf(q) > 0x1p-12f && fabsf(q) < 1024.f ? to_odd(q, fmaf(-q, s, x)) : q;
}
__device__ __forceinline__ float multiply_to_odd(float x, float s) {
    const float p = x * s;
    return to_odd(p, fmaf(x, s, -p));
}
// top <= MOST * s, of the exact product
template <int MOST>
__device__ __forceinline__ bool fits(float top, float s) {
    const float p = (float)MOST * s;
    return top < p || (top == p && fmaf((float)MOST, s, -p) >= 0.f);
}

}  // namespace append
}  // namespace medusa
