// q8.cuh -- the 8-bit paged KV cache: what a page holds, which scales are
// readable, e4m3 conversions, and the even split of attention work over CTAs.
//
// A pool of n_pages pages serves every sequence: codes [n_pages][Hkv][P][D] in
// e4m3 for K and for V, one float scale per (page, KV head), value = code *
// scale.  One (page, head) is P * D contiguous bytes: the unit that a TMA box,
// an append and a page copy move.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace medusa {
namespace q8 {

constexpr float kE4m3Max = 448.f;
constexpr int kMaxBatch = 1024;  // sequences a call takes (row tables fit shared memory)
// readable scales: far from the ends of float32, so that sums of codes times
// scales (and their inverses) over a million keys stay finite
constexpr float kMinScale = 5.421010862427522e-20f;  // 2^-64
constexpr float kMaxScale = 18446744073709551616.f;  // 2^64

// Limits every entry point of the paged cache shares.
inline int check_pool(const char* who, int B, int Hkv, int D, int P, int n_pages, int M) {
    if ((D != 64 && D != 128) || (P != 16 && P != 32 && P != 64 && P != 128))
        return fail(MEDUSA_ERR_UNSUPPORTED, "%s: head dim %d must be 64 or 128, page %d tokens 16, 32, 64 or 128", who, D, P);
    if (B > kMaxBatch) return fail(MEDUSA_ERR_UNSUPPORTED, "%s: batch %d above %d", who, B, kMaxBatch);
    if (Hkv > 1024) return fail(MEDUSA_ERR_UNSUPPORTED, "%s: %d KV heads above 1024", who, Hkv);
    if ((long long)n_pages * Hkv * P > 0x7fffffffll)
        return fail(MEDUSA_ERR_UNSUPPORTED, "%s: a pool of %d pages x %d heads x %d rows exceeds 2^31 rows", who, n_pages,
                    Hkv, P);
    if ((long long)M * P > (1ll << 30) || (long long)B * M > (1ll << 30))
        return fail(MEDUSA_ERR_UNSUPPORTED, "%s: a table of %d x %d pages is too large", who, B, M);
    return MEDUSA_OK;
}

__host__ __device__ __forceinline__ bool scale_ok(float s) { return s >= kMinScale && s <= kMaxScale; }

// two e4m3 codes (low, high byte) -> two floats, exactly
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    float2 f;
    asm("{\n.reg .f16 a, b;\nmov.b32 {a, b}, %2;\ncvt.f32.f16 %0, a;\ncvt.f32.f16 %1, b;\n}"
        : "=f"(f.x), "=f"(f.y) : "r"(h));
    return f;
}
// two floats -> two e4m3 codes (lo in the low byte): nearest even, held at 448,
// NaN stays NaN
__device__ __forceinline__ uint16_t float2_to_e4m3x2(float lo, float hi) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
    return c;
}

// two products on the paired float32 pipe
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b) {
    asm("{\n.reg .b64 ra, rb, rd;\nmov.b64 ra, {%2, %3};\nmov.b64 rb, {%4, %4};\n"
        "mul.rn.f32x2 rd, ra, rb;\nmov.b64 {%0, %1}, rd;\n}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b));
}

__device__ __forceinline__ int clamp_int(int x, int lo, int hi) { return x < lo ? lo : (x > hi ? hi : x); }

// ---------------------------------------------------------------------------
// Attention work.  A unit is (sequence, KV head, block of query rows); its keys
// are cut into tiles of T: first the prefix's, then the tree's.  The tiles of all
// units, laid end to end, are shared out evenly over the CTAs (the lengths are
// known on the device only, so the host cannot choose a split); a unit counts V
// tiles more, in front of its own, for what taking it up and handing its result out
// costs.  A CTA's share is a run of segments, each a range of one unit's tiles; a
// unit that several CTAs share leaves one partial result per CTA, joined by a merge
// kernel.  Where no unit can have more than a few tiles (the tables' width bounds them on
// the host) the units themselves are shared out, and there is nothing to join.
struct Work {
    // U units per sequence, T keys per tile, cap slots per sequence, whole: no unit is cut
    int B, N, U, T, V, cap, ctas, whole;
    __device__ __forceinline__ int len(const int32_t* kv_len, int b) const { return clamp_int(kv_len[b], 0, cap); }
    __device__ __forceinline__ int prefix_tiles(int L) const { return (L + T - 1) / T; }
    __device__ __forceinline__ int tree_tiles() const { return (N + T - 1) / T; }
    __device__ __forceinline__ int span(int L) const { return V + prefix_tiles(L) + tree_tiles(); }
    // total * c / ctas, in 32 bits
    __device__ __forceinline__ uint32_t cta_begin(uint32_t total, int c) const {
        const uint32_t q = total / (uint32_t)ctas, r = total - q * (uint32_t)ctas;
        return q * (uint32_t)c + r * (uint32_t)c / (uint32_t)ctas;
    }
    // the CTA whose share holds position g: the largest c with total * c / ctas <= g
    __device__ __forceinline__ int cta_of(uint32_t total, uint32_t g) const {
        return (int)((((unsigned long long)g + 1) * ctas - 1) / total);
    }
};

// Two tables in shared memory: first[b] (b <= B), where the units of sequence b begin, and rest[b], the length of b less the whole tiles before its last one.
// (Tiles are counted in 32 bits: the entry point bounds their number.)
constexpr int kMaxSmem = 232448;  // shared memory of a CTA on sm_103
__host__ __device__ constexpr int offsets_bytes(int B) { return (B + 1) * 4 + (B + 3) / 4 * 4; }
struct Offsets {
    uint32_t* first;
    uint8_t* rest;
    __device__ __forceinline__ Offsets(void* smem, int B)
        : first(static_cast<uint32_t*>(smem)), rest(reinterpret_cast<uint8_t*>(first + B + 1)) {}
    __device__ __forceinline__ uint32_t total(const Work& w) const { return first[w.B]; }
};

// Fills the tables; called by every thread of the block.  last, where given: a sequence whose
// last is negative counts as one without slots.
__device__ __forceinline__ void tile_offsets(const Work& w, const int32_t* __restrict__ kv_len, const Offsets& t,
                                             const int32_t* __restrict__ last = nullptr) {
    for (int b = threadIdx.x; b < w.B; b += blockDim.x) {
        const int L = last && last[b] < 0 ? 0 : w.len(kv_len, b);
        t.rest[b] = (uint8_t)(L ? (L - 1) % w.T : 0);
        t.first[b + 1] = (uint32_t)w.U * w.span(L);
    }
    if (threadIdx.x == 0) t.first[0] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {  // inclusive scan by one warp, 32 sequences at a time
        uint32_t carry = 0;
        for (int b0 = 0; b0 < w.B; b0 += 32) {
            const int b = b0 + (int)threadIdx.x;
            uint32_t v = b < w.B ? t.first[b + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
                if ((int)threadIdx.x >= o) v += u;
            }
            v += carry;
            if (b < w.B) t.first[b + 1] = v;
            carry = __shfl_sync(0xffffffffu, v, 31);
        }
    }
    __syncthreads();
}

// The sequence whose units hold g (first[b] <= g < first[b + 1]).
__device__ __forceinline__ int find_sequence(const uint32_t* first, int B, uint32_t g) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= g) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Where the share of CTA c begins (c = ctas: where the last one ends).
__device__ __forceinline__ uint32_t share_begin(const Work& w, const Offsets& t, int c) {
    const uint32_t total = t.total(w);
    if (!w.whole) return w.cta_begin(total, c);
    const uint32_t units = (uint32_t)w.B * w.U, u = (uint32_t)c * units / (uint32_t)w.ctas;
    if (u == units) return total;
    const uint32_t b = u / (uint32_t)w.U;
    return t.first[b] + (u - b * w.U) * ((t.first[b + 1] - t.first[b]) / (uint32_t)w.U);
}

// Tiles [t0, t1) of unit `unit` of sequence b.
struct Segment {
    int b, unit, t0, t1, tiles, L;
    uint32_t begin, end;  // positions of the unit's span
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
    // a CTA has at most one segment that begins inside a unit (its first) and one
    // that begins a unit without ending it (its last): its two partial slots
    __device__ __forceinline__ int slot(int cta) const { return 2 * cta + (t0 > 0 ? 0 : 1); }
};
// The segment at position g of a share that ends at g_end.
__device__ __forceinline__ Segment segment_at(const Work& w, const Offsets& t, uint32_t g, uint32_t g_end) {
    Segment s;
    s.b = find_sequence(t.first, w.B, g);
    const int span = (int)((t.first[s.b + 1] - t.first[s.b]) / (uint32_t)w.U);
    s.tiles = span - w.V;
    const int pt = s.tiles - w.tree_tiles();
    s.L = pt ? (pt - 1) * w.T + t.rest[s.b] + 1 : 0;
    const uint32_t x = g - t.first[s.b];
    s.unit = (int)(x / (uint32_t)span);
    s.begin = t.first[s.b] + (uint32_t)s.unit * span;
    s.end = s.begin + span;
    s.t0 = max(0, (int)(g - s.begin) - w.V);
    s.t1 = max(0, (int)(min(g_end, s.end) - s.begin) - w.V);
    return s;
}
// Moves g to the next segment that has tiles; false: the share has none left.
__device__ __forceinline__ bool next_segment(const Work& w, const Offsets& t, uint32_t& g, uint32_t g_end, Segment& s) {
    while (g < g_end) {
        s = segment_at(w, t, g, g_end);
        if (s.t1 > s.t0) return true;
        g = s.end;
    }
    return false;
}

}  // namespace q8

// Attention of one row a sequence over the slots that it holds, at most 16 query heads a KV head,
// bf16 (attention_q8.cu; the arguments are checked, the workspace is large enough).
size_t row_attention_q8_workspace(int G, int D);
int row_attention_q8(const char* who, const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
                     const float* v_scale, const int32_t* page_table, const int32_t* kv_len, const int32_t* last, int B, int Hq,
                     int Hkv, int D, int P, int n_pages, int M, float scale, void* out, void* ws, void* stream);
}  // namespace medusa
