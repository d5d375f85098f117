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
// after whole turns, two integer products instead of 64-bit floating ones, of which an SM does
// two a cycle.  The fraction comes from a double, off by 2^-52 of inv_freq / 2 pi and by 2^-65, so that
// the angle is off by p (2^-52 |inv_freq| + 2^-62) radians, and is then rounded to 2^-32 revolutions:
// by 2 pi * 2^-33 < 2^-30 radians.
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

// (cos, sin) of p turns.  Within an eighth of a revolution of a multiple of a quarter, the series
// of sine and cosine to the 9th and 10th power are off by 2^-29 and 2^-33 (the next terms, x^11 /
// 11! and x^12 / 12!); what is left is the rounding of the angle to float32 (2^-25 at an eighth of a
// revolution) and of the sums, 2^-24 each.
__device__ __forceinline__ float2 cos_sin(uint64_t turn, int p) {
    const uint32_t w = (uint32_t)((turn * (uint64_t)(int64_t)p + (1ull << 31)) >> 32);  // units of 2^-32 revolutions
    const uint32_t quarter = (w + (1u << 29)) >> 30;
    const float x = (float)(int32_t)(w - (quarter << 30)) * 1.46291807926715968e-9f;  // 2 pi / 2^32
    const float z = x * x;
    const float s = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), x);
    const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f), 1.f);
    const float cs = quarter & 1 ? s : c, sn = quarter & 1 ? c : s;
    return make_float2((quarter + 1) & 2 ? -cs : cs, quarter & 2 ? -sn : sn);
}

// The sixteen values that a thread works on, item = 0 .. D / 16 - 1 of a head: eight pairs, or
// sixteen values behind the pairs, in two pieces of eight that lie as far apart as they can, so that
// neighbouring threads read neighbouring pieces.
struct Item {
    int first, second;  // where the two pieces begin
    int turns;          // its place in a row of the table, -1: not rotated
};
__device__ __forceinline__ Item item_at(const Freqs& f, int item, int D) {
    const int i = item * 8;
    return i < f.n ? Item{i, f.n + i, item} : Item{f.n + i, (D - 2 * f.n) / 2 + f.n + i, -1};
}

// A row's cosines and sines in shared memory, [4][n / 8] float4 of two pairs each: the threads of
// neighbouring items read side by side (sixteen bytes of every 64 took four times as long).
// Entry e of n: frequency freq_at(e) at float2 number place(e).
__device__ __forceinline__ int freq_at(const Freqs& f, int e) {  // the pair that an item's k-th is, e = 8 * item + k
    const int item = e >> 3, k = e & 7;
    return !f.interleaved ? e : k < 4 ? item * 4 + k : f.n / 2 + item * 4 + k - 4;
}
__device__ __forceinline__ int place(const Freqs& f, int e) { return ((e & 7) >> 1) * (f.n / 4) + (e >> 3) * 2 + (e & 1); }

// The rows first .. first + count - 1 of the table; row r stands at position pos(r).  Called by
// every thread of the block.
template <typename Pos>
__device__ __forceinline__ void fill_table(const Freqs& f, float2* table, int first, int count, Pos pos) {
    const int per = blockDim.x / f.n, e = threadIdx.x % f.n;  // threads per entry
    if ((int)threadIdx.x >= per * f.n) return;
    const uint64_t step = turn(f.inv_freq[freq_at(f, e)]);
    const int at = place(f, e);
    for (int r = first + threadIdx.x / f.n; r < first + count; r += per) table[r * f.n + at] = cos_sin(step, pos(r));
}

// a, b: the two pieces; turns: the item's first float4 of the row's table
__device__ __forceinline__ void rotate(const Freqs& f, float (&a)[8], float (&b)[8], const float4* turns) {
    float2 t[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = turns[i * (f.n / 8)];
        t[2 * i] = make_float2(v.x, v.y);
        t[2 * i + 1] = make_float2(v.z, v.w);
    }
    if (f.interleaved) {
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
