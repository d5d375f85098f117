// chunks.cuh -- how the attention of a chunk of new tokens over the 8-bit paged cache is cut
// into work.
//
// Row i < n of a sequence sees the slots [0, L - n + i] of its L: the chunk's own keys are in
// the pages.  A unit is (sequence, block of `tb` tokens, KV head); it has the tiles of `tile`
// slots up to the last one that its last row sees, so that nothing behind the diagonal is
// looked at but in its last tiles.  The tiles of all units, laid end to end, are shared out
// evenly over the CTAs (lengths are known on the device only); a unit counts `setup` tiles
// more, in front of its own, for what taking it up and handing its result out costs.  A unit
// that several CTAs share leaves one partial result per CTA, joined by a merge kernel.  Where
// no unit can have more than a few tiles the units themselves are shared out (`whole`).
#pragma once

#include <stdint.h>

#include "q8.cuh"

namespace medusa {
namespace chunks {

struct Work {
    int B, T, heads, blocks, tb, tile, setup, cap, ctas, whole;  // heads: KV heads; cap: slots of a table row
    // tiles of block j of a sequence with L slots, the last n of them the chunk's
    __device__ __forceinline__ int tiles(int L, int n, int j) const {
        const int lo = j * tb;
        if (lo >= n) return 0;
        const int lim = L - n + min(lo + tb, n) - 1;  // last slot that the block's last row sees
        return lim < 0 ? 0 : lim / tile + 1;
    }
    // positions of a unit with so many tiles; one that sees nothing has its rows set to zero and no more
    __device__ __forceinline__ int span_of(int tiles) const { return whole || !tiles ? 1 : setup + tiles; }
    __device__ __forceinline__ int span(int L, int n, int j) const { return span_of(tiles(L, n, j)); }
    // total * c / ctas, in 32 bits
    __device__ __forceinline__ uint32_t share(uint32_t total, int c) const {
        const uint32_t q = total / (uint32_t)ctas, r = total - q * (uint32_t)ctas;
        return q * (uint32_t)c + r * (uint32_t)c / (uint32_t)ctas;
    }
    __device__ __forceinline__ int cta_of(uint32_t total, uint32_t g) const {
        return (int)((((unsigned long long)g + 1) * ctas - 1) / total);
    }
};

// Tables in shared memory: first[b], where the units of sequence b begin (b <= B), and its
// lengths (L, n).
__host__ __device__ constexpr int table_bytes(int B) { return (B + 1) * 12; }
struct Tables {
    int2* len;
    uint32_t* first;
    __device__ __forceinline__ Tables(void* smem, int B) : len(static_cast<int2*>(smem)), first(reinterpret_cast<uint32_t*>(len + B)) {}
};

// Called by every thread of the block.
__device__ __forceinline__ void fill_tables(const Work& w, const int32_t* __restrict__ kv_len, const int32_t* __restrict__ last,
                                            const Tables& t) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    for (int b = threadIdx.x; b < w.B; b += blockDim.x)
        t.len[b] = make_int2(q8::clamp_int(kv_len[b], 0, w.cap), last ? q8::clamp_int(last[b], -1, w.T - 1) + 1 : w.T);
    __syncthreads();
    if (w.blocks <= 8) {
        for (int b = threadIdx.x; b < w.B; b += blockDim.x) {
            uint32_t sum = 0;
            for (int j = 0; j < w.blocks; ++j) sum += w.span(t.len[b].x, t.len[b].y, j);
            t.first[b + 1] = sum * (uint32_t)w.heads;
        }
    } else {
        for (int b = warp; b < w.B; b += warps) {
            uint32_t sum = 0;
            for (int j = lane; j < w.blocks; j += 32) sum += w.span(t.len[b].x, t.len[b].y, j);
            sum = __reduce_add_sync(0xffffffffu, sum);
            if (lane == 0) t.first[b + 1] = sum * (uint32_t)w.heads;
        }
    }
    if (threadIdx.x == 0) t.first[0] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {  // inclusive scan by one warp, 32 sequences at a time
        uint32_t carry = 0;
        for (int b0 = 0; b0 < w.B; b0 += 32) {
            const int b = b0 + lane;
            uint32_t v = b < w.B ? t.first[b + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            v += carry;
            if (b < w.B) t.first[b + 1] = v;
            carry = __shfl_sync(0xffffffffu, v, 31);
        }
    }
    __syncthreads();
}

// A unit and the position where it begins.
struct Cursor {
    int b, j, h, L, n, tiles;
    uint32_t begin;
    __device__ __forceinline__ void set(const Work& w, const Tables& t) {
        L = t.len[b].x;
        n = t.len[b].y;
        tiles = w.tiles(L, n, j);
    }
    __device__ __forceinline__ uint32_t end(const Work& w) const { return begin + w.span_of(tiles); }
    // the next unit; not called behind the last one
    __device__ __forceinline__ void next(const Work& w, const Tables& t) {
        begin = end(w);
        if (++h < w.heads) return;
        h = 0;
        if (++j == w.blocks) { j = 0; ++b; }
        if (b < w.B) set(w, t);
    }
    // its tiles that the share [g0, g1) has
    __device__ __forceinline__ int first_tile(const Work& w, uint32_t g0) const {
        return w.whole || g0 <= begin ? 0 : max(0, (int)(g0 - begin) - w.setup);
    }
    __device__ __forceinline__ int end_tile(const Work& w, uint32_t g1) const {
        return w.whole || g1 >= end(w) ? tiles : max(0, (int)(g1 - begin) - w.setup);
    }
};

// The unit at position g < first[B]; called by one whole warp.
__device__ __forceinline__ Cursor cursor_at(const Work& w, const Tables& t, uint32_t g) {
    const int lane = threadIdx.x & 31;
    Cursor c;
    c.b = q8::find_sequence(t.first, w.B, g);
    c.L = t.len[c.b].x;
    c.n = t.len[c.b].y;
    uint32_t base = t.first[c.b];
    c.j = 0;
    for (int j0 = 0; j0 < w.blocks; j0 += 32) {
        const int j = j0 + lane;
        const uint32_t v = j < w.blocks ? (uint32_t)w.heads * w.span(c.L, c.n, j) : 0;
        uint32_t upto = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += u;
        }
        const unsigned behind = __ballot_sync(0xffffffffu, base + upto > g);
        if (behind) {
            const int at = __ffs(behind) - 1;
            c.j = j0 + at;
            base += __shfl_sync(0xffffffffu, upto - v, at);
            break;
        }
        base += __shfl_sync(0xffffffffu, upto, 31);
    }
    const uint32_t span = (uint32_t)w.span(c.L, c.n, c.j);
    c.h = (int)((g - base) / span);
    c.begin = base + (uint32_t)c.h * span;
    c.tiles = w.tiles(c.L, c.n, c.j);
    return c;
}

// What the merge has to know about the share [g0, g1): the unit that it begins and leaves to
// others to finish, as (last share of it, sequence, block, KV head); x = -1: none.  Called by
// one whole warp.
__device__ __forceinline__ int4 plan_share(const Work& w, const Tables& t, uint32_t g0, uint32_t g1) {
    int4 p = make_int4(-1, 0, 0, 0);
    if (w.whole || g0 >= g1) return p;
    const Cursor c = cursor_at(w, t, g1 - 1);
    const uint32_t tile0 = c.begin + w.setup;
    if (g0 <= tile0 && tile0 < g1 && g1 < c.end(w)) p = make_int4(w.cta_of(t.first[w.B], c.end(w) - 1), c.b, c.j, c.h);
    return p;
}

}  // namespace chunks
}  // namespace medusa
