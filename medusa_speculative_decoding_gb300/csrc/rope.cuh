// rope.cuh -- rotary positions: which values of a head are a pair, and the sine and cosine
// of position * frequency for positions of any size.
//
// A head's first 2n values are n pairs (i, n + i), or (2i, 2i + 1) where `interleaved`; pair
// i of the row at position p turns by p * inv_freq[i]:
//   (a, b) -> (a cos - b sin, b cos + a sin),
// in float32, rounded once by the caller.  Values behind 2n stay as they are.
//
// p * inv_freq in float32 is off by 2^-25 p radians: 0.03 at a million tokens.  Here a
// frequency is a 64-bit fraction of a revolution, so that p times it modulo 2^64 is the angle
// after whole turns, off by p * 2^-64 revolutions and the 2^-53 of the fraction itself; two
// integer products instead of 64-bit floating ones, of which an SM does two a cycle.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace medusa {
namespace rope {

struct Freqs {
    const float* inv_freq;  // [n]
    int n, interleaved;
};

// inv_freq / 2 pi modulo 1, in units of 2^-64
__device__ __forceinline__ uint64_t turn(float inv_freq) {
    double t = (double)inv_freq * 0.15915494309189535;
    t -= floor(t);
    return __double2ull_rn(t * 18446744073709551616.0);
}

// (cos, sin) of p turns
__device__ __forceinline__ float2 cos_sin(uint64_t turn, int p) {
    const uint32_t w = (uint32_t)((turn * (uint64_t)(int64_t)p) >> 32);  // units of 2^-32 revolutions
    const uint32_t quarter = (w + (1u << 29)) >> 30;
    const float x = (float)(int32_t)(w - (quarter << 30)) * 0x1p-31f;  // half turns, within a quarter
    float s, c;
    sincospif(x, &s, &c);
    const float cs = quarter & 1 ? s : c, sn = quarter & 1 ? c : s;
    return make_float2((quarter + 1) & 2 ? -cs : cs, quarter & 2 ? -sn : sn);
}

// The sixteen values that a thread works on: eight pairs in two pieces of eight values, or
// sixteen values behind the pairs.  item = 0 .. D / 16 - 1 of a head.
struct Item {
    int first, second;  // where the two pieces begin
    int freq;           // of the first pair, -1: not rotated
};
__device__ __forceinline__ Item item_at(const Freqs& f, int item) {
    const int i = item * 8;
    if (i >= f.n) return Item{2 * i, 2 * i + 8, -1};
    return f.interleaved ? Item{2 * i, 2 * i + 8, i} : Item{i, f.n + i, i};
}

// a, b: the two pieces; cs: (cos, sin) of the eight pairs
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const float2* cs, bool interleaved) {
    float2 t[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float4 v = *reinterpret_cast<const float4*>(cs + i);
        t[i] = make_float2(v.x, v.y);
        t[i + 1] = make_float2(v.z, v.w);
    }
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], w = b[2 * i + 1];
            a[2 * i] = x * t[i].x - y * t[i].y;
            a[2 * i + 1] = y * t[i].x + x * t[i].y;
            b[2 * i] = z * t[i + 4].x - w * t[i + 4].y;
            b[2 * i + 1] = w * t[i + 4].x + z * t[i + 4].y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = a[i], y = b[i];
            a[i] = x * t[i].x - y * t[i].y;
            b[i] = y * t[i].x + x * t[i].y;
        }
    }
}

__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
    uint4 w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(x[1]), "f"(x[0]));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(x[3]), "f"(x[2]));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.z) : "f"(x[5]), "f"(x[4]));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.w) : "f"(x[7]), "f"(x[6]));
    *reinterpret_cast<uint4*>(p) = w;
}

// The limits that the entry points share.
inline int check_freqs(const char* who, const float* inv_freq, int n, int D) {
    if (!inv_freq) return fail(MEDUSA_ERR_INVALID_ARG, "%s: null pointer", who);
    if (n < 8 || n % 8 || 2 * n > D)
        return fail(MEDUSA_ERR_UNSUPPORTED, "%s: %d frequencies must be a multiple of 8, at most half of head dim %d", who, n, D);
    return MEDUSA_OK;
}

}  // namespace rope
}  // namespace medusa
