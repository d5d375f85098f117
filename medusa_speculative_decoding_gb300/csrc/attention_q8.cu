// attention_q8.cu -- tree attention over the 8-bit paged cache ("Medusa Heads"
// glossary page, "Tree attention and acceptance").
//
// Query i attends to the prefix keys in the pages (code * scale) and to the
// tree rows m whose bit m of mask row i is set:
//   out = softmax(scale * q.k) v
// The tree's own K and V rows are given in the model's type, next to the cache:
// rejected candidates never reach a page.
//
//   tree_attn_q8_umma_kernel   : bf16, on the tensor cores
//   tree_attn_q8_simple_kernel : float32, on the CUDA cores
//   attn_q8_merge_kernel       : joins the partial results of units that several
//                                CTAs share (q8.cuh, Work)
#include <float.h>

#include <type_traits>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "q8.cuh"
#include "tmap.cuh"
#include "umma.cuh"

namespace medusa {
namespace {

MEDUSA_WAIT_CONTROL()

constexpr float kLog2e = 1.4426950408889634f;

struct AttnQ8Args {
    const void *q, *k_tree, *v_tree;
    const uint8_t *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    const int32_t *page_table, *kv_len;
    const uint64_t* mask;
    void* out;
    float* part_o;   // ws [2 * ctas][rows][D]: sums relative to the row's reference
    float2* part_ml;  // ws [2 * ctas][rows]: (reference in log2 units, sum)
    int4* plan;       // ws [ctas]: see plan_share
    q8::Work work;
    int Hq, Hkv, G, P, M, n_pages, W, qblocks;
    float scale_log2;
};

__device__ __forceinline__ void store1(uint16_t* p, float v) {
    uint16_t r;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(v));
    *p = r;
}

__device__ __forceinline__ void store4(float* p, float4 v, float f) {
    *reinterpret_cast<float4*>(p) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
}
__device__ __forceinline__ void store4(uint16_t* p, float4 v, float f) {
    uint2 w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(v.y * f), "f"(v.x * f));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(v.w * f), "f"(v.z * f));
    *reinterpret_cast<uint2*>(p) = w;
}

// 2^x with x <= 0 or -inf; exp2f is within 2 units in the last place
__device__ __forceinline__ float weight(float x) { return exp2f(x); }

// What the merge has to know about share c = blockIdx.x: the unit that it begins and
// leaves to others to finish, as (last share of it, sequence, KV head, first row); x =
// -1: none.  One thread; it is off every path that others wait for.
__device__ __forceinline__ void plan_share(const AttnQ8Args& a, const q8::Offsets& first, int rows_block) {
    const q8::Work& w = a.work;
    if (w.whole) return;  // there is no merge
    const uint32_t total = first.total(w);
    const uint32_t g_begin = w.cta_begin(total, blockIdx.x), g_end = w.cta_begin(total, blockIdx.x + 1);
    int4 p = make_int4(-1, 0, 0, 0);
    if (g_begin < g_end) {
        const q8::Segment s = q8::segment_at(w, first, g_end - 1, g_end);
        const uint32_t tiles = s.begin + w.V;  // the unit's first tile
        if (g_begin <= tiles && tiles < g_end && g_end < s.end)
            p = make_int4(w.cta_of(total, s.end - 1), s.b, s.unit / a.qblocks, s.unit % a.qblocks * rows_block);
    }
    a.plan[blockIdx.x] = p;
}

// ---------------------------------------------------------------------------
// One CTA works through its share of (unit, tile) pairs; a unit's block has
// ROWS query rows, 16 or 64.  Each tile of kKeys keys is dequantised into shared
// memory once for all rows; scores, softmax and sums are float32.  A thread has four
// rows and KT keys (then CP columns) of each product.  Small calls are bound by
// latency: 14 us with the merge for nine rows, four heads of 64 and 128 keys.  Large
// ones by issue and shared memory: with blocks of 16 rows, whose every key is
// dequantised anew, 147 us for three sequences of 2730 keys, 8 heads of 64 and 64 rows, with
// 64 rows 67 (85 with 512 threads); at D = 128, 2000 keys and two sequences 83 and 69 (78
// with 256 threads, of which an SM holds one block).  One token goes through a block
// of 16 rows, most of them zero: 509 us for sixteen sequences of 777 to 16384 keys, 8 heads
// of 4 rows, where reading the codes takes 42.
// ---------------------------------------------------------------------------
constexpr int kKeys = 64;

template <int D, int ROWS>
struct SimpleSmem {
    static constexpr int kStride = D + 4, kStrideP = kKeys + 4;  // rows 16 bytes apart in the banks
    static constexpr int kOffV = kKeys * kStride * 4;
    static constexpr int kOffQ = kOffV + kKeys * D * 4;
    static constexpr int kOffP = kOffQ + ROWS * kStride * 4;
    static constexpr int kOffStat = kOffP + ROWS * kStrideP * 4;  // corr, m, l
    static constexpr int kOffFirst = kOffStat + 3 * ROWS * 4;  // tile offsets
    static constexpr int bytes(int B) { return kOffFirst + q8::offsets_bytes(B); }
};

template <int D, int ROWS, int THREADS>
__global__ void __launch_bounds__(THREADS) tree_attn_q8_simple_kernel(const AttnQ8Args a) {
    using L = SimpleSmem<D, ROWS>;
    extern __shared__ __align__(16) uint8_t smem[];
    float* sk = reinterpret_cast<float*>(smem);
    float* sv = reinterpret_cast<float*>(smem + L::kOffV);
    float* sq = reinterpret_cast<float*>(smem + L::kOffQ);
    float* sp = reinterpret_cast<float*>(smem + L::kOffP);
    float* s_corr = reinterpret_cast<float*>(smem + L::kOffStat);
    float* s_m = s_corr + ROWS;
    float* s_l = s_m + ROWS;
    const q8::Offsets first(smem + L::kOffFirst, a.work.B);
    __shared__ uint64_t s_seen[kKeys];  // rows that see the key, one bit each
    __shared__ int s_bad[kKeys];        // tree key whose V row holds an infinity or NaN
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const q8::Work w = a.work;
    pdl_wait();
    pdl_trigger();
    q8::tile_offsets(w, a.kv_len, first);
    const uint32_t g_begin = q8::share_begin(w, first, blockIdx.x), g_end = q8::share_begin(w, first, blockIdx.x + 1);
    uint32_t g = g_begin;
    const int rows_all = w.N * a.G;
    // this thread's four rows; its KT keys, KL apart; its CP columns, CW side by side
    constexpr int KT = ROWS * kKeys / (4 * THREADS), KL = kKeys / KT, CP = D * ROWS / (4 * THREADS), CW = CP < 4 ? CP : 4;
    const int r0 = tid / KL * 4, kl = tid % KL;
    auto column = [&](int j) { return (j / CW * KL + kl) * CW + j % CW; };
    for (q8::Segment s; q8::next_segment(w, first, g, g_end, s); g = s.end) {
        const int hk = s.unit / a.qblocks, row0 = s.unit % a.qblocks * ROWS;
        const int nrows = min(ROWS, rows_all - row0);
        for (int i = tid; i < ROWS * D; i += THREADS) {
            const int r = row0 + i / D;
            float v = 0.f;
            if (i / D < nrows)
                v = static_cast<const float*>(a.q)[(((size_t)s.b * w.N + r / a.G) * a.Hq + hk * a.G + r % a.G) * D + i % D];
            sq[i / D * L::kStride + i % D] = v;
        }
        if (tid < ROWS) { s_m[tid] = -INFINITY; s_l[tid] = 0.f; }
        if (tid < kKeys) s_bad[tid] = 0;
        float acc[4][CP];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < CP; ++j) acc[i][j] = 0.f;
        const int pt = w.prefix_tiles(s.L);
        for (int t = s.t0; t < s.t1; ++t) {
            __syncthreads();
            const bool tree = t >= pt;
            const int k0 = tree ? (t - pt) * kKeys : t * kKeys;
            const int nk = min(kKeys, (tree ? w.N : s.L) - k0);
            // keys of the tile, 8 elements a step; absent ones read zero
            for (int i = tid; i < kKeys * (D / 8); i += THREADS) {
                const int key = i / (D / 8), c = i % (D / 8) * 8;
                float kx[8], vx[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) kx[e] = vx[e] = 0.f;
                bool there = key < nk;
                if (there && tree) {
                    const size_t o = (((size_t)s.b * w.N + k0 + key) * a.Hkv + hk) * D + c;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        kx[e] = static_cast<const float*>(a.k_tree)[o + e];
                        vx[e] = static_cast<const float*>(a.v_tree)[o + e];
                        // 0 * inf of a masked row would spoil rows that do not see it
                        if (!isfinite(vx[e])) { vx[e] = 0.f; s_bad[key] = 1; }
                    }
                } else if (there) {
                    const int slot = k0 + key;
                    const int page = a.page_table[(size_t)s.b * a.M + slot / a.P];
                    there = page >= 0 && page < a.n_pages;
                    if (there) {
                        const size_t unit = (size_t)page * a.Hkv + hk;
                        const float ks = a.k_scale[unit], vs = a.v_scale[unit];
                        there = q8::scale_ok(ks) && q8::scale_ok(vs);
                        if (there) {
                            const size_t o = (unit * a.P + slot % a.P) * D + c;
                            const uint2 kw = *reinterpret_cast<const uint2*>(a.k_pages + o);
                            const uint2 vw = *reinterpret_cast<const uint2*>(a.v_pages + o);
                            const uint32_t kk[2] = {kw.x, kw.y}, vv[2] = {vw.x, vw.y};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 kf = q8::e4m3x2_to_float2((uint16_t)(kk[e >> 1] >> (16 * (e & 1))));
                                const float2 vf = q8::e4m3x2_to_float2((uint16_t)(vv[e >> 1] >> (16 * (e & 1))));
                                kx[2 * e] = kf.x * ks; kx[2 * e + 1] = kf.y * ks;
                                vx[2 * e] = vf.x * vs; vx[2 * e + 1] = vf.y * vs;
                            }
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    *reinterpret_cast<float4*>(sk + key * L::kStride + c + e) = make_float4(kx[e], kx[e + 1], kx[e + 2], kx[e + 3]);
                    *reinterpret_cast<float4*>(sv + key * D + c + e) = make_float4(vx[e], vx[e + 1], vx[e + 2], vx[e + 3]);
                }
                if (c == 0) {
                    uint64_t seen = there ? ~0ull : 0ull;
                    if (there && tree) {
                        seen = 0;
                        const int m = k0 + key;
                        for (int r = 0; r < nrows; ++r)
                            seen |= ((a.mask[(size_t)((row0 + r) / a.G) * a.W + (m >> 6)] >> (m & 63)) & 1) << r;
                    }
                    s_seen[key] = seen;
                }
            }
            __syncthreads();
            {
                float z[4][KT];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < KT; ++j) z[i][j] = 0.f;
#pragma unroll 4
                for (int c = 0; c < D; c += 4) {
                    float4 kx[KT], qx[4];
#pragma unroll
                    for (int j = 0; j < KT; ++j) kx[j] = *reinterpret_cast<const float4*>(sk + (kl + j * KL) * L::kStride + c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) qx[i] = *reinterpret_cast<const float4*>(sq + (r0 + i) * L::kStride + c);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < KT; ++j)
                            z[i][j] = fmaf(qx[i].x, kx[j].x, fmaf(qx[i].y, kx[j].y, fmaf(qx[i].z, kx[j].z, fmaf(qx[i].w, kx[j].w, z[i][j]))));
                }
#pragma unroll
                for (int j = 0; j < KT; ++j) {
                    const uint64_t seen = s_seen[kl + j * KL];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sp[(r0 + i) * L::kStrideP + kl + j * KL] = (seen >> (r0 + i)) & 1 ? z[i][j] * a.scale_log2 : -INFINITY;
                }
            }
            __syncthreads();
            // running maximum and sum, several rows per warp
            constexpr int RW = ROWS * 32 / THREADS;
#pragma unroll 4
            for (int r = RW * warp; r < RW * (warp + 1); ++r) {
                const float x0 = sp[r * L::kStrideP + lane], x1 = sp[r * L::kStrideP + lane + 32];
                float mx = fmaxf(x0, x1);
                // a NaN score makes the row NaN: the sum below carries it
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float m0 = s_m[r], m1 = fmaxf(m0, mx);
                const float ref = m1 == -INFINITY ? 0.f : m1;
                const float p0 = weight(x0 - ref), p1 = weight(x1 - ref);
                float sum = warp_sum(p0 + p1);
                const bool bad = (s_bad[lane] && (s_seen[lane] >> r & 1)) || (s_bad[lane + 32] && (s_seen[lane + 32] >> r & 1));
                if (__any_sync(0xffffffffu, bad)) sum = NAN;
                sp[r * L::kStrideP + lane] = p0;
                sp[r * L::kStrideP + lane + 32] = p1;
                if (lane == 0) {
                    const float c = weight(m0 - ref);  // 0 where nothing was seen before
                    s_corr[r] = c;
                    s_m[r] = m1;
                    s_l[r] = s_l[r] * c + sum;
                }
            }
            __syncthreads();
            if (tid < kKeys) s_bad[tid] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float c = s_corr[r0 + i];
#pragma unroll
                for (int j = 0; j < CP; ++j) acc[i][j] *= c;
            }
#pragma unroll 2
            for (int k = 0; k < kKeys; k += 4) {
                float p[4][4], v[4][CP];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<float4*>(p[i]) = *reinterpret_cast<const float4*>(sp + (r0 + i) * L::kStrideP + k);
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int j = 0; j < CP; j += CW) {
                        const float* from = sv + (k + e) * D + column(j);
                        if constexpr (CW == 4) *reinterpret_cast<float4*>(v[e] + j) = *reinterpret_cast<const float4*>(from);
                        else if constexpr (CW == 2) *reinterpret_cast<float2*>(v[e] + j) = *reinterpret_cast<const float2*>(from);
                        else v[e][j] = *from;
                    }
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < CP; ++j) acc[i][j] = fmaf(p[i][e], v[e][j], acc[i][j]);
            }
        }
        const bool whole = s.whole();
        const size_t part = (size_t)s.slot(blockIdx.x) * ROWS;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = row0 + r0 + i;
            const float l = s_l[r0 + i];
            if (whole && r0 + i >= nrows) continue;
            float* out = static_cast<float*>(a.out) + (((size_t)s.b * w.N + r / a.G) * a.Hq + hk * a.G + r % a.G) * D;
#pragma unroll
            for (int j = 0; j < CP; ++j) {
                if (whole) out[column(j)] = l == 0.f ? 0.f : acc[i][j] / l;
                else a.part_o[(part + r0 + i) * D + column(j)] = acc[i][j];
            }
        }
        if (!whole && tid < ROWS) a.part_ml[part + tid] = make_float2(s_m[tid], s_l[tid]);
        __syncthreads();  // q, statistics free again
    }
    // an empty share gives nothing to the units around it
    if (tid < ROWS && g_begin == g_end)
        a.part_ml[(size_t)2 * blockIdx.x * ROWS + tid] = make_float2(-INFINITY, 0.f);
    if (tid == 0) plan_share(a, first, ROWS);
}

// ---------------------------------------------------------------------------
// tcgen05 kernel (bf16 queries).
//
// Products on the 8-bit codes themselves.  The codes go from the page into the
// matrix instruction as they are; what has more than e4m3's four significant
// bits is split into planes that the instruction takes:
//   scores   bf16 has 8 bits: q = q_hi + q_lo, two e4m3 planes under one power of
//            two for the block (exact down to 2^-17 of its largest |q|), both added
//            into S = K q; the page's scale multiplies S
//   output   weight times V scale = p_1 + p_2 + p_3, three e5m2 planes side by side
//            in one product: 9 bits, down to 2^-17 of the row's largest, and fewer from
//            there to 2^-26 (e5m2 has the range that a softmax needs: with an
//            attention sink the weights that count can be 2^-12 of the largest)
// so no key or value is ever converted: converting them would cost more
// instructions than the whole softmax of 64 rows, and twice the shared memory.
//
// Transposed: S^T = K Q^T and O^T = V^T P^T, the 128 keys of a tile (then the D
// output columns) in the TMEM lanes and the query rows in the columns.  A thread
// owns one key: its scale is one register, the work is in proportion to the
// query rows (from 16 on) rather than to the 128 rows of a matrix tile, and the
// row sums are added up per thread and joined once per segment.  What crosses
// threads is the rows' maximum, and that only when a weight times its V scale rises
// 2^6.9 above the reference it is held against (the first tile and few others), which
// one barrier vote per tile finds out.
//
// Two streams per CTA (four warps each, one per lane quarter), each with its own S and O in
// TMEM, so that one stream's softmax runs while the other's products do:
//   SHARED = false  blocks of NB rows; the streams take alternate tiles, each an
//                   online softmax of its own, joined at the end
//   SHARED = true   blocks of 2 NB rows; each stream has NB of them, both use
//                   every tile
// Steps x = 0, 1, 2, ...: stream x & 1, tile x (or x / 2).  S has two buffers a
// stream, so its MMA warp forms scores up to two steps ahead, and a stream waits
// for its last PV only before it writes the next weights or rescales O.
//
// Warps 0-7 softmax, warps 8 and 9 MMA (one per stream), warp 10 TMA (page tables,
// scales and tiles run ahead through a ring of slots; a slot is K and V of one tile
// of 128 keys).
// The tree's rows are bf16: such a tile takes two slots, and its products are
// kind::f16 with q and P in bf16, added to the same sums.
// Every wait is bounded; a CTA that gives up marks its results NaN.
//
// Measured, merge included: 96 us for eight sequences of 1024 to 4096 keys, 40 heads, 64
// rows (231 MB, 2.4 TB/s); 386 us for four of 8192 keys, 32 heads, 341 rows (191 GFLOP, 494
// TFLOP/s); 50 us for sixteen of 777 to 16384 keys, 8 heads of 4 rows (282 MB, 5.6 TB/s); 22
// us for one of 2048 keys, 32 heads, 64 rows.  With 64 rows and more no unit is near full
// (341 rows: issue slots 44%, tensor pipe 31%, DRAM 30%; eight sequences: 33, 16 and 29%): a
// scheduler has two softmax warps, and both wait in turn for a tile's vote, the stream's
// last PV and the scores' way out of TMEM.  With 16 rows it is the tiles under way.
// ---------------------------------------------------------------------------
constexpr int kTile = 128;  // keys per tile
constexpr int kUSoftmax = 256, kUThreads = kUSoftmax + 96;
constexpr int kUMmaWarp = kUSoftmax / 32, kUTmaWarp = kUMmaWarp + 2;  // an MMA warp per stream
constexpr int kUStream = kUSoftmax / 2;  // threads of a stream
// Tiles that a unit counts more (q8.cuh, Work): first references, tree tile and results
// cost as much as several tiles, and more where they are of more rows.  Measured with
// 3 / 5 / 7 / 9 / 12 / 16: eight ragged sequences of 64 rows 103 / 100 / 97 / 96 / 97 / 97
// us, four of 341 rows 392 / 390 / 388 / 386 / 386 / 386 us, one of 2048 keys 20 / 20 / 22 /
// 22 / 22 / 22 us (the price of 9 where there are few units a CTA); sixteen sequences of
// one token 51 / 50 / 51 / 52 / 53 / 55 us.
constexpr int kSetup = 9, kSetup16 = 5;
// What enters the sum over V is weight * V scale, w = 2^(x + log2 vs - m) with x the score
// in log2 units and m the row's reference, the largest x + log2 vs when set.  So a page's
// scale counts only as far as its weight does, row by row.  The planes hold w * 2^kLift,
// which may grow to 2^15.9, below f16's largest 65504, before the references move; a tree
// row's (vs = 1, bf16) to 2^27.9: 512 of them times 2^91 stay below 2^128 (too_large).
// The row sums hold w / vs * 2^(kLift - kUnit), from 2^-112 for the largest scale to
// 2^116 for the smallest and a w that is taken back.
constexpr float kLift = 9.f, kUnit = 57.f;
constexpr float kTopPage = 15.9f, kTopTree = 27.9f;
// A reference that moves by more drops what was summed up before, the weights' sum as
// well: keys whose w is below 2^-100 of a later one's.  (Their weight is below 2^-36 of its
// weight where the scales of the two differ by 2^64 at most.)
constexpr float kDrop = 100.f;
constexpr long long kDrainCycles = kDefaultWaitCycles;

template <int D, int NB, bool SHARED>
struct USmem {
    // Slots of the ring.  Split streams take alternate tiles, so an even number keeps a
    // slot with its stream: what a stream's tile replaces is an earlier tile of its own,
    // and a look at the slot's barrier cannot mistake one phase for another.
    static constexpr int kRing = SHARED ? 3 : 4;
    static constexpr int kBlocks = SHARED ? 2 : 1;             // row blocks of NB
    static constexpr int kRowsBlock = NB * kBlocks;
    static constexpr int kQ8 = 2 * NB * D;                     // hi rows, lo rows
    static constexpr int kQB = NB * D * 2;                     // bf16, for the tree tiles
    static constexpr int kHalf = kTile * D;                    // K or V codes of a tile
    static constexpr int kSlot = 2 * kHalf;
    static constexpr int kPlane = kTile * 64;                  // one plane of weights: rows of 64 bytes
    static constexpr int kP = NB == 64 ? 3 * kPlane : 2 * kPlane;  // (two: bf16 weights of a tree tile)
    static constexpr int kOffRing = 0;
    static constexpr int kOffP = kOffRing + kRing * kSlot;
    static constexpr int kOffQ8 = kOffP + 2 * kP;
    static constexpr int kOffQB = kOffQ8 + (kBlocks * kQ8 + 1023) / 1024 * 1024;
    static constexpr int kOffM = kOffQB + (kBlocks * kQB + 1023) / 1024 * 1024;  // float -m[2][NB], m = row reference
    static constexpr int kOffCorr = kOffM + 2 * NB * 4;        // float corr[2][NB], later coefficients
    static constexpr int kOffRed = kOffCorr + 2 * NB * 4;      // float red[2][4][NB]
    static constexpr int kOffRow = kOffRed + 8 * NB * 4;       // int [2][kRowsBlock]: (node, head) of a row, in rows of D
    static constexpr int kOffMask = kOffRow + 2 * kRowsBlock * 4;      // uint32 [kRowsBlock][16]: mask rows
    static constexpr int kOffInfo = kOffMask + kRowsBlock * 64;  // float2 (k scale, log2 of v scale)[kRing][8]
    static constexpr int kOffBad = kOffInfo + kRing * 8 * 8;   // uint32 [2][4]: keys of a tree tile with a non-finite V
    static constexpr int kOffMisc = kOffBad + 32;              // see below, 256 bytes
    static constexpr int kOffBar = kOffMisc + 256;
    // full[R] empty[R] s_full[2][2] p_full[2] pv_done[2] qfull seen checked[2] drain[2]
    static constexpr int kNumBar = 2 * kRing + 14;
    static constexpr int kOffFirst = (kOffBar + kNumBar * 8 + 15) / 16 * 16;
    static constexpr int bytes(int B) { return kOffFirst + q8::offsets_bytes(B) + 1024; }  // + alignment slack
};

__device__ __forceinline__ float redux_max_nan(float v) {  // NaN if any is
    float r;
    asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float redux_max(float v) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
// (the barrier takes whole warps in step: lanes that left a wait or a branch at
// different times meet first)
__device__ __forceinline__ void bar_sync(int id, int n) {
    __syncwarp();
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
// All lanes wait; the same answer in all of them.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, long long lim) {
    return __all_sync(0xffffffffu, umma::mbar_wait(bar, parity, lim));
}
// pairs of floats on the paired float32 pipe
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b, float c0, float c1) {
    asm("{\n.reg .b64 ra, rb, rc, rd;\nmov.b64 ra, {%2, %3};\nmov.b64 rb, {%4, %4};\nmov.b64 rc, {%5, %6};\n"
        "fma.rn.f32x2 rd, ra, rb, rc;\nmov.b64 {%0, %1}, rd;\n}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1) {
    asm("{\n.reg .b64 ra, rb, rd;\nmov.b64 ra, {%0, %1};\nmov.b64 rb, {%2, %3};\n"
        "add.rn.f32x2 rd, ra, rb;\nmov.b64 {%0, %1}, rd;\n}"
        : "+f"(d0), "+f"(d1) : "f"(a0), "f"(a1));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two weights (times V scale) into their planes.  e5m2 is the upper byte of f16: the
// first two planes cut the f16 value off behind that byte (three bits each, and what
// is left is exact in f16), the third rounds.  Returns the planes' values in the upper
// bytes of each half.
__device__ __forceinline__ void split_weights(float a, float b, uint32_t (&plane)[3]) {
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(plane[0]) : "f"(b), "f"(a));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(plane[1]) : "r"(plane[0]), "r"(plane[0] & 0xff00ff00u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(plane[2]) : "r"(plane[1]), "r"(plane[1] & 0xff00ff00u));
    plane[2] += 0x00800080u;
}
// Any of eight bf16 values infinite, NaN or of 2^91 and more: a weight may be 2^27.9 in the
// sums' units, and 512 of them times 2^91 stay below float32's 2^128.
__device__ __forceinline__ bool too_large(const uint4& v) {
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) bad = bad || (x[e] & 0x7f80u) >= 0x6d00u || (x[e] & 0x7f800000u) >= 0x6d000000u;
    return bad;
}
__device__ __forceinline__ uint32_t join16(uint16_t lo, uint16_t hi) { return (uint32_t)lo | (uint32_t)hi << 16; }

template <int D, int NB, bool SHARED>
__global__ void __launch_bounds__(kUThreads, 1) tree_attn_q8_umma_kernel(
    const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
    const __grid_constant__ CUtensorMap tmkt, const __grid_constant__ CUtensorMap tmvt, const AttnQ8Args a) {
    using namespace umma;
    using L = USmem<D, NB, SHARED>;
    constexpr int R = L::kRing;
    // TMEM: S of stream s at NB (2 s + buffer); O behind it, OP sums of NB columns a
    // stream.  NB = 64: the third plane is added to the second's sum, so that two
    // buffers of S have room.
    constexpr int OP = NB == 64 ? 2 : 3, kCols = NB == 64 ? 512 : 256;
    constexpr uint32_t kO = 4 * NB;
    extern __shared__ uint8_t smem_raw[];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const q8::Work w = a.work;

    const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
    uint8_t* base = smem_raw + pad;
    const uint32_t base_a = smem_addr(base);
    const uint32_t ring_a = base_a + L::kOffRing, p_a = base_a + L::kOffP, q8_a = base_a + L::kOffQ8,
                   qb_a = base_a + L::kOffQB;
    const uint32_t bar_a = base_a + L::kOffBar;
    const uint32_t full0 = bar_a, empty0 = full0 + 8 * R, s_full0 = empty0 + 8 * R, p_full0 = s_full0 + 32,
                   pv_done0 = p_full0 + 16, qfull = pv_done0 + 16, seen = qfull + 8, checked0 = seen + 8, drain = checked0 + 16;
    float* s_m = reinterpret_cast<float*>(base + L::kOffM);
    float* s_corr = reinterpret_cast<float*>(base + L::kOffCorr);
    float* s_red = reinterpret_cast<float*>(base + L::kOffRed);
    float2* s_info = reinterpret_cast<float2*>(base + L::kOffInfo);
    uint32_t* s_bad = reinterpret_cast<uint32_t*>(base + L::kOffBad);
    int* s_row = reinterpret_cast<int*>(base + L::kOffRow);
    uint32_t* s_mask = reinterpret_cast<uint32_t*>(base + L::kOffMask);
    float* s_misc = reinterpret_cast<float*>(base + L::kOffMisc);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_misc);
    volatile int* s_fail = reinterpret_cast<volatile int*>(s_misc + 2);    // [2] per stream
    float* s_qmax = s_misc + 16;                                           // [2][kUSoftmax / 32] per warp
    uint32_t* s_hurt = reinterpret_cast<uint32_t*>(s_misc + 32);           // [2][2] rows of a stream that saw a bad V, one bit each
    const q8::Offsets first(base + L::kOffFirst, w.B);
    const long long lim = g_wait_limit;

    if (warp == kUTmaWarp && lane == 0) {
        for (int i = 0; i < L::kNumBar; ++i) mbar_init(bar_a + 8 * i, 1);
        mbar_init(p_full0, kUStream / 32);
        mbar_init(p_full0 + 8, kUStream / 32);
        if (SHARED)  // a slot is free when both streams' products are through
            for (int i = 0; i < R; ++i) mbar_init(empty0 + 8 * i, 2);
        for (int i = 0; i < 4; ++i) mbar_init(s_full0 + 8 * i, 2);  // the products, and the MMA warp itself
        mbar_init(qfull, kUSoftmax / 32);
        mbar_init(seen, 2);
        mbar_init(checked0, 4);
        mbar_init(checked0 + 8, 4);
        mbar_init_fence();
        s_fail[0] = s_fail[1] = 0;
        for (int i = 0; i < 4; ++i) s_hurt[i] = 0;
        prefetch_tmap(&tmk);
        prefetch_tmap(&tmv);
        prefetch_tmap(&tmkt);
        prefetch_tmap(&tmvt);
    }
    if (warp == 0) tmem_alloc(tmem_slot, kCols);
    pdl_wait();
    pdl_trigger();
    q8::tile_offsets(w, a.kv_len, first);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint32_t g_begin = q8::share_begin(w, first, blockIdx.x), g_end = q8::share_begin(w, first, blockIdx.x + 1);
    const int ppt = kTile / a.P;  // pages per tile
    const int rows_all = w.N * a.G;
    uint32_t g_failed = g_end;   // first segment whose results are not there
    bool gave_up = false;

    // tiles of a segment: n_pre of the prefix, then n_tree of the tree
    auto prefix_of = [&](const q8::Segment& s, int& n_pre, int& n_tree) {
        const int pt = w.prefix_tiles(s.L);
        n_pre = max(0, min(s.t1, pt) - s.t0);
        n_tree = s.t1 - s.t0 - n_pre;
    };

    if (warp >= kUMmaWarp && warp < kUTmaWarp) {
        // ------------------------ MMA warp of a stream ------------------------
        const int st = warp - kUMmaWarp;
        constexpr uint32_t id_s = idesc_f8(128, NB, 0, 0, 0, 0);
        constexpr uint32_t id_pv = idesc_f8(128, (NB == 64 ? 2 : 3) * NB, 0, 1, 1, 1), id_p3 = idesc_f8(128, NB, 0, 1, 1, 1);
        constexpr uint32_t id_st = idesc_bf16(128, NB, 0, 0), id_pt = idesc_bf16(128, NB, 1, 1);
        const uint32_t s_full = s_full0 + 16 * st, p_full = p_full0 + 8 * st, pv_done = pv_done0 + 8 * st;
        const uint32_t tS = tmem + 2 * st * NB, tO = tmem + kO + st * OP * NB, p = p_a + st * L::kP;
        const uint32_t q8s = q8_a + (SHARED ? st : 0) * L::kQ8, qbs = qb_a + (SHARED ? st : 0) * L::kQB;
        auto desc8 = [](uint32_t addr) {  // codes: rows of D bytes, either major
            return D == 128 ? desc_sw128(addr, 16, 1024) : desc_sw64(addr, 0, 512);
        };
        bool fail = false;
        int slot0 = 0;      // first slot of the segment
        uint32_t p_par = 0;  // parity of the next step's weights
        int seg = 0;
        uint32_t g = g_begin;
        for (q8::Segment s; !fail && q8::next_segment(w, first, g, g_end, s); g = s.end, ++seg) {
            int n_pre, n_tree;
            prefix_of(s, n_pre, n_tree);
            // (the shuffles tell the compiler that these are the same in all lanes)
            n_pre = __shfl_sync(0xffffffffu, n_pre, 0);
            n_tree = __shfl_sync(0xffffffffu, n_tree, 0);
            const int n = n_pre + n_tree, steps = SHARED ? n : (n + 1 - st) >> 1;
            auto tile_of = [&](int i) { return SHARED ? i : 2 * i + st; };
            auto slot_of = [&](int t) { return slot0 + t + max(0, t - n_pre); };
            if (!warp_wait(qfull, (uint32_t)(seg & 1), lim)) fail = true;
            if (lane == 0) mbar_arrive(seen);  // (a stream without steps must not fall segments behind)
            // S runs up to two steps ahead of PV; whichever of the next S and the next PV
            // has its inputs goes, S first when the stream has no scores left
            int ns = 0, np = 0, spins = 0;
            int sl = slot_of(tile_of(0));
            uint32_t s_stage = sl % R, s_bar = full0 + 8 * s_stage, s_par = (sl / R) & 1;  // K of step ns
            long long t_last = 0;
            while (np < steps && !fail) {
                const bool can_s = ns < steps && ns < np + 2 && mbar_test(s_bar, s_par);
                bool can_pv = np < ns && mbar_test(p_full, p_par);
                const int t = tile_of(np);
                if (can_pv && t >= n_pre) {
                    const int sv = slot_of(t) + 1;
                    can_pv = mbar_test(full0 + 8 * (sv % R), (uint32_t)((sv / R) & 1));
                }
                if (__all_sync(0xffffffffu, can_s) && (ns <= np + 1 || !__all_sync(0xffffffffu, can_pv))) {
                    fence_after_sync();
                    const uint32_t k = ring_a + s_stage * L::kSlot, d = tS + (ns & 1) * NB;
                    if (tile_of(ns) < n_pre) {
                        const uint64_t dk = desc8(k), dq = desc8(q8s);
#pragma unroll
                        for (int ks = 0; ks < D / 32; ++ks) {
                            mma_f8_warp(d, dk + 2 * ks, dq + 2 * ks, id_s, ks > 0);
                            mma_f8_warp(d, dk + 2 * ks, dq + ((NB * D) >> 4) + 2 * ks, id_s, 1);
                        }
                    } else {
                        const uint64_t dk = desc_sw128(k, 16, 1024), dq = desc_sw128(qbs, 16, 1024);
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks)
                            mma_bf16_warp(d, dk + (((ks >> 2) * (kTile * 128) + (ks & 3) * 32) >> 4),
                                          dq + (((ks >> 2) * (NB * 128) + (ks & 3) * 32) >> 4), id_st, ks > 0);
                    }
                    commit_warp(s_full + 8 * (ns & 1));
                    // (this arrival hands on the scales, which came with the slot)
                    if (lane == 0) mbar_arrive(s_full + 8 * (ns & 1));
                    ++ns;
                    sl = slot_of(tile_of(ns));
                    s_stage = sl % R;
                    s_bar = full0 + 8 * s_stage;
                    s_par = (sl / R) & 1;
                    spins = 0;
                } else if (__all_sync(0xffffffffu, can_pv)) {
                    fence_after_sync();
                    const int slv = slot_of(t);
                    const uint32_t stage = slv % R;
                    if (t < n_pre) {
                        const uint64_t dv = desc8(ring_a + stage * L::kSlot + L::kHalf);
                        // NB = 64: a plane is one swizzle atom wide, the next one a plane behind;
                        // NB = 16: the planes share the 64 bytes of a key
                        const uint64_t dp = desc_sw64(p, L::kPlane, 512);
#pragma unroll
                        for (int ks = 0; ks < kTile / 32; ++ks)
                            mma_f8_warp(tO, dv + ((ks * 32 * D) >> 4), dp + ((ks * 2048) >> 4), id_pv, np > 0 || ks > 0);
                        if constexpr (NB == 64) {
                            const uint64_t d3 = desc_sw64(p + 2 * L::kPlane, 0, 512);
#pragma unroll
                            for (int ks = 0; ks < kTile / 32; ++ks)
                                mma_f8_warp(tO + NB, dv + ((ks * 32 * D) >> 4), d3 + ((ks * 2048) >> 4), id_p3, 1);
                        }
                    } else {
                        // D = 64: the second half of the lanes repeats the first
                        const uint64_t dv = desc_sw128(ring_a + ((slv + 1) % R) * L::kSlot, D == 128 ? kTile * 128 : 0, 1024);
                        const uint64_t dp = desc_sw128(p, 0, 1024);
#pragma unroll
                        for (int ks = 0; ks < kTile / 16; ++ks)
                            mma_bf16_warp(tO, dv + ((ks * 2048) >> 4), dp + ((ks * 2048) >> 4), id_pt, np > 0 || ks > 0);
                    }
                    commit_warp(pv_done);
                    commit_warp(empty0 + 8 * stage);
                    if (t >= n_pre) commit_warp(empty0 + 8 * ((slv + 1) % R));
                    ++np;
                    p_par ^= 1;
                    spins = 0;
                } else if ((++spins & 7) == 0) {
                    if (spins == 8) t_last = clock64();
                    fail = __any_sync(0xffffffffu, clock64() - t_last > lim);
                }
            }
            slot0 += n_pre + 2 * n_tree;
        }
        // Everything in flight completes before TMEM is freed, whoever gave up.
        commit_warp(drain + 8 * st);
        warp_wait(drain + 8 * st, 0, kDrainCycles);
    } else if (warp == kUTmaWarp) {
        // -------------------------------- TMA warp --------------------------------
        int slot = 0;
        bool fail = false;
        auto free_slot = [&](int sl) {
            if (sl >= R && !warp_wait(empty0 + 8 * (sl % R), (uint32_t)((sl / R - 1) & 1), lim)) fail = true;
            return !fail;
        };
        uint32_t g = g_begin;
        for (q8::Segment s; !fail && q8::next_segment(w, first, g, g_end, s); g = s.end) {
            int n_pre, n_tree;
            prefix_of(s, n_pre, n_tree);
            const int hk = s.unit / a.qblocks;
            const int32_t* table = a.page_table + (size_t)s.b * a.M;
            const int pg0 = s.t0 * ppt, pages = (s.L + a.P - 1) / a.P;
            // lane i holds page i of a group of 32: its number two groups ahead, its
            // scales one group ahead
            auto page_id = [&](int i) {
                const int pg = pg0 + i;
                if (n_pre == 0 || pg >= pages) return -1;
                const int p = __ldg(table + pg);
                return p >= 0 && p < a.n_pages ? p : -1;
            };
            auto scales = [&](int p) {
                if (p < 0) return make_float2(0.f, 0.f);
                const size_t u = (size_t)p * a.Hkv + hk;
                return make_float2(__ldg(a.k_scale + u), __ldg(a.v_scale + u));
            };
            int id = page_id(lane), id1 = page_id(32 + lane), id2 = -1;
            float2 sc = scales(id), sc1 = make_float2(0.f, 0.f);
            for (int u = 0; u < n_pre; ++u, ++slot) {
                const int li = (u * ppt) & 31;
                if (li == 0) {
                    if (u) { id = id1; sc = sc1; id1 = id2; }
                    sc1 = scales(id1);
                    id2 = page_id(u * ppt + 64 + lane);
                }
                if (!free_slot(slot)) break;
                const int st = slot % R, j = lane - li;
                const bool in = j >= 0 && j < ppt, there = in && id >= 0;
                if (there) {
                    const int y = (id * a.Hkv + hk) * a.P;
                    const uint32_t dst = ring_a + st * L::kSlot + j * a.P * D;
                    tma_load_2d(dst, &tmk, 0, y, full0 + 8 * st);
                    tma_load_2d(dst + L::kHalf, &tmv, 0, y, full0 + 8 * st);
                }
                const unsigned m = __ballot_sync(0xffffffffu, there);
                if (in)
                    s_info[st * 8 + j] = there && q8::scale_ok(sc.x) && q8::scale_ok(sc.y) ? make_float2(sc.x, log2f(sc.y))
                                                                                            : make_float2(0.f, -INFINITY);
                __syncwarp();
                if (lane == 0) mbar_expect_tx(full0 + 8 * st, (uint32_t)(__popc(m) * a.P * D * 2));
            }
            const int pt = w.prefix_tiles(s.L);
            for (int u = n_pre; u < n_pre + n_tree && !fail; ++u) {
                const int row = (s.t0 + u - pt) * kTile;
                // both slots are free before either is filled: when K is in, V's slot holds
                // no earlier tile on its way
                if (!free_slot(slot) || !free_slot(slot + 1)) break;
                for (int kv = 0; kv < 2; ++kv, ++slot) {
                    if (lane == 0) {
                        const int st = slot % R;
                        mbar_expect_tx(full0 + 8 * st, kTile * D * 2);
#pragma unroll
                        for (int x = 0; x < D / 64; ++x)
                            tma_load_4d(ring_a + st * L::kSlot + x * kTile * 128, kv ? &tmvt : &tmkt, x * 64, hk, row, s.b,
                                        full0 + 8 * st);
                    }
                }
            }
        }
        // Every slot that was asked for lands before the CTA leaves, whoever gave up.
        if (lane == 0)
            for (int sl = max(0, slot - R); sl < slot; ++sl)
                mbar_wait(full0 + 8 * (sl % R), (uint32_t)((sl / R) & 1), kDrainCycles);
        if (lane == 0) plan_share(a, first, L::kRowsBlock);
    } else if (warp < kUMmaWarp) {
        // ------------------------------ softmax warps ------------------------------
        constexpr int CW = NB;  // rows (columns of S^T) per thread
        const int st = warp >> 2, quarter = warp & 3;
        const int key = quarter * 32 + lane;  // TMEM lane: key of a tile, then output column
        const int stid = tid & (kUStream - 1);
        const int page_shift = 31 - __clz(a.P);
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tO = tmem + lane_off + kO + st * OP * NB;
        float* m_row = s_m + st * NB;  // negated
        float* corr_row = s_corr + st * NB;
        uint8_t* p_row = base + L::kOffP + st * L::kP;
        const float scale = a.scale_log2;
        int n_s = 0;             // steps of this stream before the segment
        int n_buf[2] = {0, 0};   // of them in each buffer of S
        int slot0 = 0;
        int n_checked = 0;  // tree tiles before the segment (shared streams)
        // Q rows of a segment's block, 16 bytes a load; rows behind its end are zero
        constexpr int CH = D / 8, QN = (L::kRowsBlock * CH + kUSoftmax - 1) / kUSoftmax;
        uint4 qv[QN];
        auto load_q = [&](const q8::Segment& s) {
            const int hk = s.unit / a.qblocks, row0 = s.unit % a.qblocks * L::kRowsBlock;
            const int nrows = min(L::kRowsBlock, rows_all - row0);
#pragma unroll
            for (int i = 0; i < QN; ++i) {
                const int c = tid + i * kUSoftmax, r = c / CH;
                qv[i] = make_uint4(0, 0, 0, 0);
                if (r < nrows) {
                    const int gr = row0 + r;
                    qv[i] = ld_stream16(static_cast<const uint16_t*>(a.q) +
                                        (((size_t)s.b * w.N + gr / a.G) * a.Hq + hk * a.G + gr % a.G) * D + c % CH * 8);
                }
            }
        };
        float kq = 0.f;  // scale / the factor of Q's planes
        // What a segment needs before its first step, in two parts around a barrier of
        // all softmax threads: largest |q| and rows' addresses; then Q into shared memory
        // (bf16 for the tree's tiles, two e4m3 planes for the pages'), which the MMA warp
        // waits for.
        auto begin_segment = [&](const q8::Segment& s, int seg) {
            const int hk = s.unit / a.qblocks, row0 = s.unit % a.qblocks * L::kRowsBlock;
            float qmax = 0.f;
#pragma unroll
            for (int i = 0; i < QN; ++i) {
                const uint32_t x[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float f0 = fabsf(bf16_lo(x[e])), f1 = fabsf(bf16_hi(x[e]));
                    if (f0 < INFINITY) qmax = fmaxf(qmax, f0);
                    if (f1 < INFINITY) qmax = fmaxf(qmax, f1);
                }
            }
            qmax = redux_max(qmax);
            if (lane == 0) s_qmax[(seg & 1) * (kUSoftmax / 32) + warp] = qmax;
            if (tid < L::kRowsBlock) {
                const int gr = row0 + tid;
                s_row[(seg & 1) * L::kRowsBlock + tid] = gr / a.G * a.Hq + hk * a.G + gr % a.G;
            }
        };
        auto take_q = [&](const q8::Segment& s, int seg) {
            const int row0 = s.unit % a.qblocks * L::kRowsBlock;
            const int nrows = min(L::kRowsBlock, rows_all - row0);
            const bool tree = s.t1 > w.prefix_tiles(s.L);
            float qmax = 0.f;
#pragma unroll
            for (int i = 0; i < kUSoftmax / 32; ++i) qmax = fmaxf(qmax, s_qmax[(seg & 1) * (kUSoftmax / 32) + i]);
            // factor 2^k with qmax * 2^k in [128, 256)
            const int qe = q8::clamp_int(254 + 7 - (int)(__float_as_uint(qmax) >> 23), 1, 253);
            const float qf = __uint_as_float((uint32_t)qe << 23);
            kq = scale * __uint_as_float((uint32_t)(254 - qe) << 23);
#pragma unroll
            for (int i = 0; i < QN; ++i) {
                const int c = tid + i * kUSoftmax, r = c / CH, ch = c % CH;
                if (r >= L::kRowsBlock) continue;
                const int blk = SHARED ? r / NB : 0, rb = SHARED ? r % NB : r;
                const uint32_t x[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
                uint16_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float f0 = bf16_lo(x[e]) * qf, f1 = bf16_hi(x[e]) * qf;
                    if (!(fabsf(f0) < INFINITY)) f0 = NAN;
                    if (!(fabsf(f1) < INFINITY)) f1 = NAN;
                    hi[e] = q8::float2_to_e4m3x2(f0, f1);
                    const float2 h = q8::e4m3x2_to_float2(hi[e]);
                    lo[e] = q8::float2_to_e4m3x2(f0 - h.x, f1 - h.y);
                }
                uint8_t* q8p = base + L::kOffQ8 + blk * L::kQ8;
                auto at8 = [&](int row) {  // 8 bytes of chunk ch of a row of D codes
                    const int c16 = ch >> 1;
                    return D == 128 ? row * 128 + ((c16 ^ (row & 7)) << 4) + (ch & 1) * 8
                                    : row * 64 + ((c16 ^ ((row >> 1) & 3)) << 4) + (ch & 1) * 8;
                };
                *reinterpret_cast<uint2*>(q8p + at8(rb)) = make_uint2(join16(hi[0], hi[1]), join16(hi[2], hi[3]));
                *reinterpret_cast<uint2*>(q8p + at8(NB + rb)) = make_uint2(join16(lo[0], lo[1]), join16(lo[2], lo[3]));
                if (tree)
                    *reinterpret_cast<uint4*>(base + L::kOffQB + blk * L::kQB + sw128_offset(rb, ch, NB)) = qv[i];
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(qfull);
            if (tree) {
                const uint32_t* mask = reinterpret_cast<const uint32_t*>(a.mask);
                for (int i = tid; i < L::kRowsBlock * 16; i += kUSoftmax) {
                    const int r = i >> 4, word = i & 15;
                    if (word < 2 * a.W) s_mask[i] = r < nrows ? __ldg(mask + (size_t)((row0 + r) / a.G) * (2 * a.W) + word) : 0u;
                }
            }
        };
        uint32_t g = g_begin;
        q8::Segment s;
        bool more = q8::next_segment(w, first, g, g_end, s);
        if (more) {
            load_q(s);
            begin_segment(s, 0);
            bar_sync(3, kUSoftmax);
            take_q(s, 0);
            bar_sync(3, kUSoftmax);
        } else if (g_begin == g_end && tid < L::kRowsBlock) {  // an empty share gives nothing to the units around it
            a.part_ml[(size_t)2 * blockIdx.x * L::kRowsBlock + tid] = make_float2(-INFINITY, 0.f);
        }
        for (int seg = 0; more; ++seg) {
            int n_pre, n_tree;
            prefix_of(s, n_pre, n_tree);
            const int n = n_pre + n_tree;
            const int steps = SHARED ? n : (n + 1 - st) >> 1;  // of this stream
            const int row0 = s.unit % a.qblocks * L::kRowsBlock;
            const int nrows = min(L::kRowsBlock, rows_all - row0);
            if (stid < NB) m_row[stid] = INFINITY;

            float l[CW];
#pragma unroll
            for (int c = 0; c < CW; ++c) l[c] = 0.f;
            bool fail = false;
            const int pt = w.prefix_tiles(s.L);
            const int i_tree = min(steps, SHARED ? n_pre : (n_pre + 1 - st) >> 1);  // first step of the tree's
            // Rows of this thread that see tree row m0 + lane.
            auto seen64 = [&](int m0) -> uint64_t {
                uint32_t lo = 0, hi = 0;
                if (m0 < w.N) {
                    const uint32_t* words = s_mask + (SHARED ? st * NB : 0) * 16 + (m0 >> 5);
#pragma unroll 16
                    for (int c = 0; c < (CW < 32 ? CW : 32); ++c) lo |= ((words[c * 16] >> lane) & 1u) << c;
#pragma unroll 16
                    for (int c = 32; c < CW; ++c) hi |= ((words[c * 16] >> lane) & 1u) << (c - 32);
                }
                return (uint64_t)hi << 32 | lo;
            };
            // One step; false: a wait gave up.  The tree's tiles have a body of their own,
            // which keeps their bookkeeping out of the prefix's registers.
            auto step = [&](auto is_tree, const int i) -> bool {
                constexpr bool tree = decltype(is_tree)::value;
                const int t = SHARED ? i : 2 * i + st;
                const int sl = slot0 + t + (tree ? t - n_pre : 0);
                const uint32_t tS = tmem + lane_off + (2 * st + (i & 1)) * NB;
                bool ok = warp_wait(s_full0 + 8 * (2 * st + (i & 1)), (uint32_t)((n_buf[i & 1] + (i >> 1)) & 1), lim);
                float kc = kq, lv = 0.f;  // lv: log2 of the V scale
                bool valid, bad_v = false;
                uint64_t sees = ~0ull;  // rows that see the key
                if constexpr (!tree) {
                    const float2 sc = s_info[(sl % R) * 8 + (key >> page_shift)];
                    valid = sc.y > -INFINITY && (s.t0 + t) * kTile + key < s.L;
                    kc = kq * sc.x;
                    lv = valid ? sc.y : 0.f;
                    sees = valid ? sees : 0;
                } else {
                    kc = scale;
                    ok = warp_wait(full0 + 8 * ((sl + 1) % R), (uint32_t)(((sl + 1) / R) & 1), lim) && ok;
                    const int m = (s.t0 + t - pt) * kTile + key;  // tree row
                    valid = m < w.N;
                    // A tree row whose V is not finite (or too large): 0 * inf of a query row that
                    // does not see it would spoil that one, so its V counts as zero and rows that
                    // see it are marked (s_hurt), which makes them NaN at the end.  Of two streams
                    // that share the tile stream 0 looks.
                    if (!SHARED || st == 0) {
                        const uint8_t* v = base + L::kOffRing + ((sl + 1) % R) * L::kSlot + key * 128;
#pragma unroll 4
                        for (int c = 0; c < D / 8; ++c)
                            bad_v = too_large(*reinterpret_cast<const uint4*>(v + (c >> 3) * kTile * 128 +
                                                                               (((c + lane) & 7) << 4))) || bad_v;
                        if constexpr (SHARED) {
                            const unsigned bad = __ballot_sync(0xffffffffu, bad_v);
                            if (lane == 0) {
                                s_bad[((n_checked + t - n_pre) & 1) * 4 + quarter] = bad;
                                mbar_arrive(checked0 + 8 * ((n_checked + t - n_pre) & 1));
                            }
                        }
                    } else {
                        // (stream 0 is at most a tile ahead: two answers are kept)
                        const int k = n_checked + t - n_pre;
                        ok = warp_wait(checked0 + 8 * (k & 1), (uint32_t)((k >> 1) & 1), lim) && ok;
                        bad_v = s_bad[(k & 1) * 4 + quarter] >> lane & 1;
                    }
                    sees = seen64(m - lane);
                    if (!valid) sees = 0;
                }
                fence_after_sync();
                const bool partial = !tree && __any_sync(0xffffffffu, !valid);
                const float lift = lv + kLift;
                const float unit = exp2_approx(-kUnit - lv);  // from w * 2^kLift to the row sums
                // log2 of w * 2^kLift, n columns of scores from c0 on.  They are read from TMEM
                // again wherever they are needed: held in between they would not fit next to the
                // sums, and what the compiler then spills does not fit L1 next to this much shared
                // memory.
                auto relative = [&](int c0, auto& x, int n) {
#pragma unroll
                    for (int e = 0; e < n; e += 4) {
                        const float4 m = *reinterpret_cast<const float4*>(m_row + c0 + e);
                        fma2(x[e], x[e + 1], x[e], x[e + 1], kc, lift, lift);
                        fma2(x[e + 2], x[e + 3], x[e + 2], x[e + 3], kc, lift, lift);
                        add2(x[e], x[e + 1], m.x, m.y);
                        add2(x[e + 2], x[e + 3], m.z, m.w);
                    }
                    if (partial) {
#pragma unroll
                        for (int e = 0; e < n; ++e) x[e] = valid ? x[e] : -INFINITY;
                    }
                    if constexpr (tree) {
#pragma unroll
                        for (int e = 0; e < n; ++e) x[e] = (sees >> (c0 + e)) & 1 ? x[e] : -INFINITY;
                    }
                };
                // The stream's last PV, behind which P and O are free.  Shared blocks form the
                // first columns' weights before this wait and write them after it (410 us
                // against 441 for 341 rows over 8192 keys); the others wait for tiles rather
                // than for products and keep the registers (113 us against 118).
                constexpr bool late = SHARED;
                auto wait_pv = [&]() {
                    if (i > 0) ok = warp_wait(pv_done0 + 8 * st, (uint32_t)((n_s + i - 1) & 1), lim) && ok;
                    if (!ok && lane == 0) s_fail[st] = 1;
                };
                if (!late || i == 0) wait_pv();
                // Weights, their sums and their planes; returns the largest score.  They are
                // written on the old references; where a score turns out to lie too far above
                // them they are taken back and written again.
                auto weights = [&](auto again) -> float {
                    constexpr bool wait_here = late && !decltype(again)::value;
                    float top = -INFINITY;
                    if constexpr (!tree) {
                        // Sixteen columns at a time.  Shared blocks load the next ones ahead (409 us
                        // against 423 for 341 rows over 8192 keys); the others gain more from the
                        // registers (119 us against 123 for eight sequences of 64 rows).
                        constexpr int W = 16, kAhead = SHARED ? 1 : 0;
                        float x[1 + kAhead][W];
                        if constexpr (kAhead) tmem_ld16(tS, x[0]);
#pragma unroll
                        for (int c0 = 0; c0 < CW; c0 += W) {
                            float(&y)[W] = x[(c0 / W) & kAhead];
                            if constexpr (!kAhead) tmem_ld16(tS + c0, y);
                            tmem_wait_ld();
                            if (kAhead && c0 + W < CW) tmem_ld16(tS + c0 + W, x[((c0 / W) & 1) ^ kAhead]);
                            relative(c0, y, W);
                            uint32_t pw[3][W / 4];
#pragma unroll
                            for (int e = 0; e < W / 4; ++e) {
                                uint32_t two[2][3];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const int c = 4 * e + 2 * k;
                                    top = max3(top, y[c], y[c + 1]);
                                    const float w0 = exp2_approx(y[c]), w1 = exp2_approx(y[c + 1]);
                                    fma2(l[c0 + c], l[c0 + c + 1], w0, w1, unit, l[c0 + c], l[c0 + c + 1]);
                                    split_weights(w0, w1, two[k]);
                                }
#pragma unroll
                                for (int p = 0; p < 3; ++p) pw[p][e] = __byte_perm(two[0][p], two[1][p], 0x7531);
                            }
                            if (wait_here && c0 == 0) wait_pv();
#pragma unroll
                            for (int p = 0; p < 3; ++p) {
                                // NB = 64: one plane of 64 bytes a key after the other; NB = 16:
                                // the planes are the key's 16-byte chunks 0, 1, 2
                                const int chunk = NB == 64 ? c0 >> 4 : p;
                                uint8_t* to = p_row + (NB == 64 ? p * L::kPlane : 0) + key * 64 +
                                              ((chunk ^ ((key >> 1) & 3)) << 4);
                                *reinterpret_cast<uint4*>(to) = make_uint4(pw[p][0], pw[p][1], pw[p][2], pw[p][3]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int c0 = 0; c0 < CW; c0 += 8) {
                            uint32_t h[4];
                            float x[8];
                            tmem_ld8(tS + c0, x);
                            tmem_wait_ld();
                            relative(c0, x, 8);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int c = 2 * e;
                                top = max3(top, x[c], x[c + 1]);
                                const float w0 = exp2_approx(x[c]), w1 = exp2_approx(x[c + 1]);
                                h[e] = pack_bf16x2(w0, w1);
                                fma2(l[c0 + c], l[c0 + c + 1], w0, w1, unit, l[c0 + c], l[c0 + c + 1]);
                            }
                            if (wait_here && c0 == 0) wait_pv();
                            *reinterpret_cast<uint4*>(p_row + key * 128 + (((c0 >> 3) ^ (key & 7)) << 4)) =
                                make_uint4(h[0], h[1], h[2], h[3]);
                        }
                    }
                    return top;
                };
                bool move = i == 0;
                for (;;) {
                    if (!move) {
                        const float top = weights(std::false_type{});
                        __syncwarp();
                        if (!named_barrier_or(1 + st, kUStream, !ok || top > (tree ? kTopTree : kTopPage))) break;
                        // Taken back: l + p - p is off by half a unit of l + p at most, and p falls
                        // to the key's own share of the sum on the new references, so the error is
                        // one rounding of the row's sum.
#pragma unroll
                        for (int c0 = 0; c0 < CW; c0 += 8) {
                            float y[8];
                            tmem_ld8(tS + c0, y);
                            tmem_wait_ld();
                            relative(c0, y, 8);
#pragma unroll
                            for (int e = 0; e < 8; e += 2)
                                fma2(l[c0 + e], l[c0 + e + 1], exp2_approx(y[e]), exp2_approx(y[e + 1]), -unit, l[c0 + e], l[c0 + e + 1]);
                        }
                    }
                    // The references move: largest score and scale per row over the tile's keys.
#pragma unroll 1
                    for (int c0 = 0; c0 < CW; c0 += 8) {
                        float y[8];
                        tmem_ld8(tS + c0, y);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; e += 2) fma2(y[e], y[e + 1], y[e], y[e + 1], kc, lv, lv);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float m = redux_max_nan((sees >> (c0 + e)) & 1 ? y[e] : -INFINITY);
                            if (lane == e) s_red[(st * 4 + quarter) * NB + c0 + e] = m;
                        }
                    }
                    bar_sync(1 + st, kUStream);
                    const bool fail = s_fail[st] != 0;
                    if (stid < NB) {
                        const float* r = s_red + st * 4 * NB + stid;
                        const float m0 = -m_row[stid];
                        // (a NaN score makes the reference, and with it the row, NaN)
                        const float m1 = max_nan(max_nan(max_nan(r[0], r[NB]), max_nan(r[2 * NB], r[3 * NB])), m0);
                        // (no w that a factor above 0 belongs to was infinite)
                        corr_row[stid] = m0 == -INFINITY || m0 - m1 < -kDrop ? 0.f : exp2f(m0 - m1);
                        m_row[stid] = -m1;
                    }
                    bar_sync(1 + st, kUStream);
                    if (fail) return false;
                    if (i > 0) {  // what was added up so far
#pragma unroll
                        for (int c = 0; c < CW; c += 4) {
                            const float4 r = *reinterpret_cast<const float4*>(corr_row + c);
                            // (0, not l * 0: where p was infinite l is NaN)
                            l[c] = r.x == 0.f ? 0.f : l[c] * r.x;
                            l[c + 1] = r.y == 0.f ? 0.f : l[c + 1] * r.y;
                            l[c + 2] = r.z == 0.f ? 0.f : l[c + 2] * r.z;
                            l[c + 3] = r.w == 0.f ? 0.f : l[c + 3] * r.w;
                        }
                        fence_after_sync();
#pragma unroll 1
                        for (int c = 0; c < CW; c += 8) {
                            float o[OP][8];
#pragma unroll
                            for (int p = 0; p < OP; ++p) tmem_ld8(tO + p * NB + c, o[p]);
                            tmem_wait_ld();
#pragma unroll
                            for (int p = 0; p < OP; ++p) {
                                uint32_t ow[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) ow[e] = __float_as_uint(o[p][e] * corr_row[c + e]);
                                tmem_st8(tO + p * NB + c, ow);
                            }
                        }
                        tmem_wait_st();
                    }
                    weights(std::true_type{});
                    break;
                }
                // A key that is not there has no V either: whatever the slot holds (stale
                // codes may be NaN) is cleared, by each stream that multiplies it.
                {
                    if (!tree && !valid) {
                        uint4* v = reinterpret_cast<uint4*>(base + L::kOffRing + (sl % R) * L::kSlot + L::kHalf + key * D);
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) v[c] = make_uint4(0, 0, 0, 0);
                    }
                    if (bad_v) {
                        // (a mark of its own: sums may be dropped when references move later)
                        atomicOr(s_hurt + 2 * st, (uint32_t)sees);
                        if constexpr (NB > 32) atomicOr(s_hurt + 2 * st + 1, (uint32_t)(sees >> 32));
                        uint8_t* v = base + L::kOffRing + ((sl + 1) % R) * L::kSlot + key * 128;
#pragma unroll 1
                        for (int c = 0; c < D / 8; ++c)
                            *reinterpret_cast<uint4*>(v + (c >> 3) * kTile * 128 + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
                    }
                }
                __syncwarp();
                fence_async_smem();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full0 + 8 * st);
                return true;
            };
            for (int i = 0; i < i_tree && !fail; ++i) fail = !step(std::false_type{}, i);
            for (int i = i_tree; i < steps && !fail; ++i) fail = !step(std::true_type{}, i);
            // row sums over the keys of this warp: halve the columns a lane holds while
            // adding the other half's
            if constexpr (CW >= 32) {
#pragma unroll
                for (int c0 = 0; c0 < CW; c0 += 32) {
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) {
                        const bool up = lane & o;
#pragma unroll
                        for (int c = c0; c < c0 + o; ++c) {
                            const float give = up ? l[c] : l[c + o], keep = up ? l[c + o] : l[c];
                            l[c] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                        }
                    }
                    s_red[(st * 4 + quarter) * NB + c0 + lane] = l[c0];
                }
            } else {
#pragma unroll
                for (int c = 0; c < CW; ++c) {
                    const float v = warp_sum(l[c]);
                    if (lane == c) s_red[(st * 4 + quarter) * NB + c] = v;
                }
            }
            // the next segment's Q, asked for now; its products start while this one's
            // results go out
            q8::Segment next = s;
            g = s.end;
            more = q8::next_segment(w, first, g, g_end, next);
            if (more) {
                load_q(next);
                begin_segment(next, seg + 1);
            }
            bool ok = !fail && warp_wait(seen, (uint32_t)(seg & 1), lim);
            if (ok && steps > 0) ok = warp_wait(pv_done0 + 8 * st, (uint32_t)((n_s + steps - 1) & 1), lim);
            __syncwarp();
            if (named_barrier_or(3, kUSoftmax, !ok)) {
                gave_up = true;
                g_failed = s.begin + w.V + s.t0;
                break;
            }
            fence_after_sync();
            n_s += steps;
            n_buf[0] += (steps + 1) >> 1;
            n_buf[1] += steps >> 1;
            slot0 += n_pre + 2 * n_tree;
            n_checked += n_tree;
            if (more) take_q(next, seg + 1);

            // Each row's coefficients.  Split streams: relative to the larger reference.
            const bool whole = s.whole();
            const size_t part = (size_t)s.slot(blockIdx.x) * L::kRowsBlock;
            if (tid < L::kRowsBlock) {
                auto sum_of = [&](int x, int c) {
                    const float* r = s_red + x * 4 * NB + c;
                    return (r[0] + r[NB]) + (r[2 * NB] + r[3 * NB]);
                };
                constexpr float kToSums = 1.f / (1ull << (int)kUnit);  // from O to the units of the sums
                float m, sum, c0, c1 = 0.f;
                if (SHARED) {
                    const int x = tid / NB, c = tid % NB;
                    m = -s_m[x * NB + c];
                    sum = sum_of(x, c);
                    c0 = kToSums;
                } else {
                    const float ma = -s_m[tid], mb = -s_m[NB + tid];
                    m = fmaxf(ma, mb);
                    const float ref = m == -INFINITY ? 0.f : m;
                    const float wa = exp2f(ma - ref), wb = exp2f(mb - ref);
                    sum = sum_of(0, tid) * wa + sum_of(1, tid) * wb;
                    c0 = wa * kToSums;
                    c1 = wb * kToSums;
                }
                const int hc = SHARED ? tid % NB : tid;
                const uint32_t hurt = SHARED ? s_hurt[2 * (tid / NB) + (hc >> 5)] : s_hurt[hc >> 5] | s_hurt[2 + (hc >> 5)];
                if (hurt >> (hc & 31) & 1) sum = NAN;
                if (whole) {
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    c0 *= inv;
                    c1 *= inv;
                } else {
                    a.part_ml[part + tid] = make_float2(m, sum);
                }
                s_corr[tid] = c0;
                if (!SHARED) s_corr[NB + tid] = c1;
            }
            bar_sync(3, kUSoftmax);
            if (tid < 4) s_hurt[tid] = 0;
            // O^T: this thread's output column of the stream's own rows (shared) or of half
            // of the block's
            constexpr int COLS = SHARED ? NB : NB / 2;
            const int first_row = st * COLS, o_col = SHARED ? 0 : first_row;
            const uint32_t oa = tmem + lane_off + kO + (SHARED ? st * OP * NB : 0) + o_col, ob = tmem + lane_off + kO + OP * NB + o_col;
            const int n_b = SHARED ? 0 : n >> 1;               // steps behind O_1
            const bool all_a = n_pre > 0, all_b = n_pre > 1;   // prefix tiles among a stream's: all planes are there
            const int* rows = s_row + (seg & 1) * L::kRowsBlock + first_row;
            uint16_t* out = static_cast<uint16_t*>(a.out) + (size_t)s.b * w.N * a.Hq * D + key;
            float* part_o = a.part_o + (part + first_row) * D + key;
            if (first_row < nrows && (D == 128 || quarter < 2)) {
#pragma unroll 1
                for (int c = 0; c < COLS; c += 8) {
                    float va[OP][8], vb[OP][8];
                    tmem_ld8(oa + c, va[0]);
                    if (all_a) {
#pragma unroll
                        for (int p = 1; p < OP; ++p) tmem_ld8(oa + p * NB + c, va[p]);
                    }
                    if (n_b > 0) tmem_ld8(ob + c, vb[0]);
                    if (!SHARED && all_b) {
#pragma unroll
                        for (int p = 1; p < OP; ++p) tmem_ld8(ob + p * NB + c, vb[p]);
                    }
                    const float4 ca[2] = {*reinterpret_cast<const float4*>(s_corr + first_row + c),
                                          *reinterpret_cast<const float4*>(s_corr + first_row + c + 4)};
                    const int4 rr[2] = {*reinterpret_cast<const int4*>(rows + c), *reinterpret_cast<const int4*>(rows + c + 4)};
                    tmem_wait_ld();
                    float o[8];
                    const float* cf = &ca[0].x;
                    const int* rf = &rr[0].x;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        o[e] = va[0][e];
                        if (all_a) {
#pragma unroll
                            for (int p = 1; p < OP; ++p) o[e] += va[p][e];
                        }
                        o[e] *= cf[e];
                    }
                    if (n_b > 0) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float y = vb[0][e];
                            if (all_b) {
#pragma unroll
                                for (int p = 1; p < OP; ++p) y += vb[p][e];
                            }
                            o[e] = fmaf(y, s_corr[NB + first_row + c + e], o[e]);
                        }
                    }
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (first_row + c + e < nrows) store1(out + (size_t)(uint32_t)rf[e] * D, o[e]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) part_o[(c + e) * D] = o[e];
                    }
                }
            }
            fence_before_sync();
            bar_sync(3, kUSoftmax);  // O is free for the next segment's products
            s = next;
        }
    }
    const bool bad = __syncthreads_or(gave_up);
    if (bad) {
        // what this CTA was to give from the segment on that it could not finish
        if (tid == 0) atomicExch(&g_wait_gave_up, 1);
        uint32_t g = g_failed;
        for (q8::Segment s; tid < kUSoftmax && q8::next_segment(w, first, g, g_end, s); g = s.end) {
            const int hk = s.unit / a.qblocks, row0 = s.unit % a.qblocks * L::kRowsBlock;
            const int nrows = min(L::kRowsBlock, rows_all - row0);
            if (!s.whole()) {
                if (tid < L::kRowsBlock)
                    a.part_ml[(size_t)s.slot(blockIdx.x) * L::kRowsBlock + tid] = make_float2(0.f, NAN);
                continue;
            }
            for (int i = tid; i < nrows * D; i += kUSoftmax) {
                const int gr = row0 + i / D;
                store1(static_cast<uint16_t*>(a.out) +
                           (((size_t)s.b * w.N + gr / a.G) * a.Hq + hk * a.G + gr % a.G) * D + i % D, NAN);
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, kCols);
}

// Joins the partial results.  Block (c, y): the unit that share c begins and others
// finish (plan_share); rows from y * kMergeThreads / (D / 4) on, four columns a
// thread.  All of a thread's loads are in flight at once (a loop of dependent loads
// took 16 rows x 10 round trips to memory, 80 us).  What a block joins is worked out
// by the shares themselves: each block doing it anew, with a scan over the sequences
// and divisions by the number of tiles, took 7 to 15 us.
constexpr int kMergeThreads = 256, kMergeBatch = 8;
template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) attn_q8_merge_kernel(const AttnQ8Args a, int rows_block) {
    pdl_wait();
    pdl_trigger();
    const int c0 = blockIdx.x;
    const int4 plan = a.plan[c0];
    const int c1 = plan.x;
    const int i = blockIdx.y * (kMergeThreads / (D / 4)) + threadIdx.x / (D / 4), d = threadIdx.x % (D / 4) * 4;
    if (c1 < 0 || i >= min(rows_block, a.work.N * a.G - plan.w)) return;
    auto slot = [&](int j) { return (size_t)(2 * j + (j == c0 ? 1 : 0)) * rows_block + i; };
    float top = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j0 = c0; j0 <= c1; j0 += kMergeBatch) {
        float2 ml[kMergeBatch];
        float4 v[kMergeBatch];
#pragma unroll
        for (int k = 0; k < kMergeBatch; ++k) {
            ml[k] = make_float2(-INFINITY, 0.f);
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j0 + k <= c1) {
                ml[k] = a.part_ml[slot(j0 + k)];
                v[k] = *reinterpret_cast<const float4*>(a.part_o + slot(j0 + k) * D + d);
            }
        }
        float m = top;
#pragma unroll
        for (int k = 0; k < kMergeBatch; ++k) m = fmaxf(m, ml[k].x);
        const float ref = m == -INFINITY ? 0.f : m;
        const float f0 = weight(top - ref);
        top = m;
        l *= f0;
        o.x *= f0; o.y *= f0; o.z *= f0; o.w *= f0;
#pragma unroll
        for (int k = 0; k < kMergeBatch; ++k) {
            // no key seen there, or an empty share, which writes no sums (a NaN row keeps its l)
            if (ml[k].x == -INFINITY && ml[k].y == 0.f) continue;
            const float f = weight(ml[k].x - ref);
            l += ml[k].y * f;
            o.x += v[k].x * f; o.y += v[k].y * f; o.z += v[k].z * f; o.w += v[k].w * f;
        }
    }
    const int r = plan.w + i;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    store4(static_cast<T*>(a.out) + (((size_t)plan.y * a.work.N + r / a.G) * a.Hq + plan.z * a.G + r % a.G) * D + d, o, inv);
}

struct Plan {
    int rows, keys, setup, ctas, whole;
};
// Rows per block, by the rows a KV head has: 16 (plain decoding), 64, or 128 in
// two streams.  Units that the table's width holds to `whole` tiles are not cut, which
// saves the merge.  bf16, cut against whole: at three tiles 17.1 / 13.8 us (one sequence, 32
// heads, 64 rows), 42 / 38 (eight, 40 heads), 9.4 / 8.0 (one of one token, 8 heads), 24.7 /
// 22.1 (one, 8 heads, 200 rows); at four and five 24.8 / 27.5 (the last), 19.0 / 19.5 (the
// first).  float32: at two tiles 12.5 / 12.3 us, at three 13.7 / 17.0.
Plan plan_q8(medusa_dtype dtype, int N, int G, int D) {
    const int rows = N * G, sms = sm_count();
    if (dtype == MEDUSA_F32) return rows <= 32 ? Plan{16, kKeys, 1, 2 * sms, 2} : Plan{64, kKeys, 1, D == 64 ? 2 * sms : sms, 2};
    if (rows <= 16) return Plan{16, kTile, kSetup16, sms, 3};
    if (rows <= 64) return Plan{64, kTile, kSetup, sms, 3};
    return Plan{128, kTile, kSetup, sms, 3};
}

int check_attn_q8(int B, int N, int Hq, int Hkv, int D, int P, int n_pages, int M) {
    if (B < 1 || N < 1 || Hq < 1 || Hkv < 1 || n_pages < 1 || M < 1)
        return fail(MEDUSA_ERR_INVALID_ARG, "tree_attention_q8: sizes must be positive");
    if (int rc = q8::check_pool("tree_attention_q8", B, Hkv, D, P, n_pages, M)) return rc;
    if (N > 512 || Hq % Hkv || (long long)N * (Hq / Hkv) > 4096)
        return fail(MEDUSA_ERR_UNSUPPORTED, "tree_attention_q8: unsupported shape (N=%d Hq=%d Hkv=%d)", N, Hq, Hkv);
    return MEDUSA_OK;
}

size_t ws_bytes_q8(const Plan& p, int D) { return (size_t)2 * p.ctas * p.rows * (D + 2) * sizeof(float) + p.ctas * sizeof(int4); }

template <typename T, int D>
cudaError_t launch_merge(const AttnQ8Args& a, const Plan& p, cudaStream_t st) {
    constexpr int rows = kMergeThreads / (D / 4);  // of a block
    const int all = a.work.N * a.G, most = all < p.rows ? all : p.rows;
    return launch(attn_q8_merge_kernel<T, D>, dim3(a.work.ctas, (most + rows - 1) / rows), dim3(kMergeThreads), 0, st, a, p.rows);
}

// The attribute is the kernel's, not the call's, so it is always what the largest batch
// takes: a call of few sequences on another thread must not lower it under this one.
template <typename Kern>
cudaError_t allow_smem(Kern kern, int most) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

template <int D, int ROWS, int THREADS>
cudaError_t launch_simple(AttnQ8Args& a, const Plan& p, cudaStream_t st) {
    auto kern = tree_attn_q8_simple_kernel<D, ROWS, THREADS>;
    constexpr int most = SimpleSmem<D, ROWS>::bytes(q8::kMaxBatch);
    static_assert(most + 1024 <= q8::kMaxSmem, "the largest batch does not fit (1024: static arrays)");
    const int smem = SimpleSmem<D, ROWS>::bytes(a.work.B);
    cudaError_t e = allow_smem(kern, most);
    if (e == cudaSuccess) e = launch(kern, dim3(a.work.ctas), dim3(THREADS), smem, st, a);
    if (e == cudaSuccess && !a.work.whole) e = launch_merge<float, D>(a, p, st);
    return e;
}

// codes [n_pages * Hkv * P][D] in boxes of one (page, head)
int pages_map(CUtensorMap* m, const void* pages, int D, int P, long long rows) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return fail(MEDUSA_ERR_CUDA, "tree_attention_q8: cuTensorMapEncodeTiled is unavailable");
    cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)D};
    cuuint32_t box[2] = {(cuuint32_t)D, (cuuint32_t)P};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(pages), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(MEDUSA_ERR_CUDA, "tree_attention_q8: tensor map encode failed (%d)", (int)r);
    return MEDUSA_OK;
}

// tree rows [B][N][Hkv][D] bf16 in boxes of 128 rows of one head x 64 elements;
// rows behind N read zero
int rows_map(CUtensorMap* m, const void* rows, int D, int Hkv, int N, int B) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)Hkv, (cuuint64_t)N, (cuuint64_t)B};
    cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)Hkv * D * 2, (cuuint64_t)N * Hkv * D * 2};
    cuuint32_t box[4] = {64, 1, (cuuint32_t)kTile, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(rows), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(MEDUSA_ERR_CUDA, "tree_attention_q8: tensor map encode failed (%d)", (int)r);
    return MEDUSA_OK;
}

template <int D, int NB, bool SHARED>
cudaError_t launch_umma(const CUtensorMap (&m)[4], AttnQ8Args& a, const Plan& p, cudaStream_t st) {
    auto kern = tree_attn_q8_umma_kernel<D, NB, SHARED>;
    constexpr int most = USmem<D, NB, SHARED>::bytes(q8::kMaxBatch);
    static_assert(most <= q8::kMaxSmem, "the largest batch does not fit");
    const int smem = USmem<D, NB, SHARED>::bytes(a.work.B);
    cudaError_t e = allow_smem(kern, most);
    if (e == cudaSuccess) e = launch(kern, dim3(a.work.ctas), dim3(kUThreads), smem, st, m[0], m[1], m[2], m[3], a);
    if (e == cudaSuccess && !a.work.whole) e = launch_merge<uint16_t, D>(a, p, st);
    return e;
}

}  // namespace
}  // namespace medusa

using namespace medusa;

extern "C" size_t medusa_tree_attention_q8_workspace(int B, int N, int Hq, int Hkv, int D, medusa_dtype dtype) {
    if (B < 1 || N < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || (D != 64 && D != 128)) return 0;
    return ws_bytes_q8(plan_q8(dtype, N, Hq / Hkv, D), D);
}

extern "C" int medusa_tree_attention_q8(const void* q, const void* k_tree, const void* v_tree, medusa_dtype dtype,
                                        const void* k_pages, const void* v_pages, const float* k_scale,
                                        const float* v_scale, const int32_t* page_table, const int32_t* kv_len,
                                        const uint64_t* mask, int B, int N, int Hq, int Hkv, int D, int P,
                                        int n_pages, int M, float scale, void* out, void* ws, size_t ws_bytes,
                                        void* stream) {
    if (int rc = check_attn_q8(B, N, Hq, Hkv, D, P, n_pages, M)) return rc;
    if (dtype != MEDUSA_F32 && dtype != MEDUSA_BF16)
        return fail(MEDUSA_ERR_UNSUPPORTED, "tree_attention_q8: unknown dtype %d", (int)dtype);
    if (!q || !k_tree || !v_tree || !k_pages || !v_pages || !k_scale || !v_scale || !page_table || !kv_len || !mask || !out)
        return fail(MEDUSA_ERR_INVALID_ARG, "tree_attention_q8: null pointer");
    if (!aligned16(q) || !aligned16(k_tree) || !aligned16(v_tree) || !aligned16(k_pages) || !aligned16(v_pages) ||
        !aligned16(out))
        return fail(MEDUSA_ERR_INVALID_ARG, "tree_attention_q8: q, tree rows, pages and out must be 16-byte aligned");
    if (!(scale > 0.f) || !(scale * kLog2e <= FLT_MAX))
        return fail(MEDUSA_ERR_INVALID_ARG, "tree_attention_q8: scale must be positive, scale * log2(e) finite");
    const Plan p = plan_q8(dtype, N, Hq / Hkv, D);
    const size_t need = ws_bytes_q8(p, D);
    if (!ws || ws_bytes < need)
        return fail(MEDUSA_ERR_WORKSPACE, "tree_attention_q8: workspace of %zu bytes needed", need);
    if (!aligned16(ws)) return fail(MEDUSA_ERR_INVALID_ARG, "tree_attention_q8: ws must be 16-byte aligned");
    AttnQ8Args a{};
    a.q = q; a.k_tree = k_tree; a.v_tree = v_tree;
    a.k_pages = (const uint8_t*)k_pages; a.v_pages = (const uint8_t*)v_pages;
    a.k_scale = k_scale; a.v_scale = v_scale;
    a.page_table = page_table; a.kv_len = kv_len; a.mask = mask; a.out = out;
    a.part_o = (float*)ws;
    a.part_ml = (float2*)((float*)ws + (size_t)2 * p.ctas * p.rows * D);
    a.plan = (int4*)(a.part_ml + (size_t)2 * p.ctas * p.rows);
    a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv; a.P = P; a.M = M; a.n_pages = n_pages; a.W = (N + 63) / 64;
    a.qblocks = (N * a.G + p.rows - 1) / p.rows;
    const long long tiles = ((long long)M * P + p.keys - 1) / p.keys + (N + p.keys - 1) / p.keys;  // of the longest unit
    const long long units = (long long)B * Hkv * a.qblocks;
    const bool whole = tiles <= p.whole && units <= 1 << 20;  // (share_begin counts in 32 bits)
    a.work = q8::Work{B, N, Hkv * a.qblocks, p.keys, p.setup, M * P, whole && units < p.ctas ? (int)units : p.ctas, whole};
    if ((long long)B * a.work.U * (((long long)M * P + p.keys - 1) / p.keys + (N + p.keys - 1) / p.keys + p.setup) > 0x7fffffffll)
        return fail(MEDUSA_ERR_UNSUPPORTED, "tree_attention_q8: %d sequences of up to %lld tokens are too many tiles", B,
                    (long long)M * P);
    a.scale_log2 = scale * kLog2e;
    cudaStream_t st = as_stream(stream);
    cudaError_t e;
    if (dtype == MEDUSA_F32) {
        e = p.rows == 16 ? (D == 64 ? launch_simple<64, 16, 256>(a, p, st) : launch_simple<128, 16, 256>(a, p, st))
                         : (D == 64 ? launch_simple<64, 64, 256>(a, p, st) : launch_simple<128, 64, 512>(a, p, st));
    } else {
        CUtensorMap m[4];
        const long long rows = (long long)n_pages * Hkv * P;
        int rc = pages_map(&m[0], k_pages, D, P, rows);
        if (!rc) rc = pages_map(&m[1], v_pages, D, P, rows);
        if (!rc) rc = rows_map(&m[2], k_tree, D, Hkv, N, B);
        if (!rc) rc = rows_map(&m[3], v_tree, D, Hkv, N, B);
        if (rc) return rc;
        if (D == 64)
            e = p.rows == 16   ? launch_umma<64, 16, false>(m, a, p, st)
                : p.rows == 64 ? launch_umma<64, 64, false>(m, a, p, st)
                               : launch_umma<64, 64, true>(m, a, p, st);
        else
            e = p.rows == 16   ? launch_umma<128, 16, false>(m, a, p, st)
                : p.rows == 64 ? launch_umma<128, 64, false>(m, a, p, st)
                               : launch_umma<128, 64, true>(m, a, p, st);
    }
    if (e != cudaSuccess)
        return fail(MEDUSA_ERR_CUDA, "tree_attention_q8: launch failed: %s", cudaGetErrorString(e));
    return MEDUSA_OK;
}
