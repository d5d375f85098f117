// attention_chunk_q8.cu -- attention of a chunk of new tokens over the 8-bit paged cache: a
// prompt, a later piece of one, or one decoded token per sequence ("Medusa Heads" glossary
// page, "Tree attention and acceptance": the prefix that the tree's pass attends to has to be
// computed first).
//
// The chunk's n = last + 1 rows are the last n of the L slots that the sequence holds, keys
// and values in the pages like those before them.  Row i sees the slots [0, L - n + i]:
//   out = softmax(scale * q.k) v,   k = code * K scale, v = code * V scale
//
//   chunk_attn_q8_umma_kernel : bf16, on the tensor cores (single rows go to the kernel of attention_q8.cu:
//                               single_row)
//   chunk_attn_q8_f32_kernel  : float32, on the CUDA cores
//   chunk_merge_kernel        : joins the partial results of units that several CTAs share
//                               (chunks.cuh)
#include <float.h>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "chunks.cuh"
#include "common.cuh"
#include "q8.cuh"
#include "tmap.cuh"
#include "umma.cuh"

namespace medusa {
namespace {

MEDUSA_WAIT_CONTROL()

constexpr float kLog2e = 1.4426950408889634f;

struct ChunkArgs {
    const void* q;
    const uint8_t *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    const int32_t *page_table, *kv_len, *last;
    void* out;
    float* part_o;    // ws [2 * ctas][rows][D]: sums relative to the row's reference
    float2* part_ml;  // ws [2 * ctas][rows]: (reference in log2 units, sum)
    int4* plan;       // ws [ctas]: chunks::plan_share
    chunks::Work work;
    int Hq, Hkv, G, P, M, n_pages, rows;  // rows: query rows of a unit
    float scale_log2;
};

__device__ __forceinline__ void store4(float* p, float4 v, float f) {
    *reinterpret_cast<float4*>(p) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void store4(uint16_t* p, float4 v, float f) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v.x * f, v.y * f), pack_bf16(v.z * f, v.w * f));
}

// ---------------------------------------------------------------------------
// tcgen05 kernel (bf16 queries).
//
// Queries in the TMEM lanes, a softmax thread per query row.
//   scores  K's codes enter the product as they are.  A bf16 value has eight significant bits:
//           q = q_hi + q_lo, an e4m3 and an e5m2 plane under one power of two per row.  What
//           q_hi leaves of a value has three bits, which e5m2 holds down to 2^-16: the sum is
//           exact for values down to 2^-13 of the row's largest, and off by 2^-21 of it below.
//   output  a page's V scale (vs) enters the weights, w = 2^(x + log2 vs - m), x the score in
//           log2 units and m the row's reference, the largest x + log2 vs when it was set (to a
//           whole number above it, so that what moves with it keeps its bits): a page's scale then
//           counts only as far as its weight does.  Weights are rounded to f16, 11 bits where the
//           model's bf16 has 8; 2^kLift times w stays below 2^15 until references move and keeps
//           its bits down to 2^-22 of the row's largest.  V's codes are converted to f16, exactly,
//           by warps of their own: the tensor core multiplies types of one kind only, and three
//           8-bit planes of the weights would cost the softmax warps more than the conversion.
//   sums    of w / vs, in float32, unrounded.
//
// Scales are those of a page: 16 neighbouring keys share theirs, so they cost a thread one
// load and two instructions per 16 scores.
//
// Two streams per CTA (a softmax warpgroup and an MMA warp each), each with its own S and O in
// TMEM, so that one stream's softmax runs while the tensor core works for the other:
//   PAIR = true   blocks of 256 rows, 128 a stream; both use every tile
//   PAIR = false  blocks of up to 128 rows (short chunks): the streams take
//                 alternate tiles, each an online softmax of its own, joined at the end
// A tile: S = q K^T into TMEM; the softmax warps write the weights of its first 64 keys over S, then
// those of the others; the MMA warp adds each half's PV to O, and forms the next S behind the second.
// So a stream's scores being in says that its PV before are done.
//
// Warps 0-3, 4-7 softmax of stream 0, 1, 8-11 queries to planes and V codes to f16, 12, 13 MMA of
// stream 0, 1, 14 pages, scales and TMA, 15 rows of units that see nothing.
//
// V codes that are NaN would spoil rows that do not see them (0 * NaN), and the slots behind a
// sequence's length hold anything: the conversion writes zero for them and notes the first such
// slot.  A row that sees it, and so all rows that see any, is made NaN when its results go out.
//
// Every wait is bounded; a CTA that gives up marks its results NaN.
//
// Measured, merge included: 486 us for four prompts of 2048 to 4096 rows, 32 heads (329 GFLOP
// counted, 677 TFLOP/s); 168 us for one of 4096 rows, 32 / 8 heads (816 TFLOP/s); 88 us for 512 rows
// on 8192 (808).  A
// tile takes about 4200 cycles where its products take 2300: per stream two halves of 1300 to 1500
// cycles (scores out of TMEM 200, their maximum 200, weights 600, handing over 150) and 1300 from
// the last weights to the next scores, of which the other stream hides a part.  One MMA warp for
// both streams 10% slower; scores of 64 keys, two buffers a stream, cost as many cycles an instruction
// as those of 128 (75) and took 40% longer; two threads a row (four softmax warpgroups) 30%.
// ---------------------------------------------------------------------------
constexpr int kTile = 128, kRows = 128;  // keys of a tile, rows of a stream
constexpr int kHalf = kTile / 2;           // keys whose weights are handed over together
constexpr int kThreads = 512, kConvWarp = 8, kConvWarps = 4, kMmaWarp = 12, kTmaWarp = 14, kZeroWarp = 15;  // an MMA warp per stream
constexpr int kGroups = kTile / 16;  // keys that share a scale
constexpr float kLift = 8.f, kMove = 7.f;
// Tiles that a unit counts more for its queries, first references and results.  Measured with 1 / 2 /
// 4 / 6 / 8: one prompt of 4096 rows 264 / 204 / 166 / 168 / 175 us, 512 rows on 8192 91 / 90 / 87 / 87
// / 89.
constexpr int kSetup = 4;
constexpr uint32_t kDrainCycles = (uint32_t)kDefaultWaitCycles;

template <int D, bool PAIR>
struct USmem {
    static constexpr int KR = (PAIR ? 3 : 4) * (128 / D), VR = (PAIR ? 2 : 3) * (128 / D);
    static constexpr int kScaleRing = 1024 / D;  // tiles whose scales are held
    static constexpr int kCodes = kTile * D;  // K or V of a tile, or a plane of q
    static constexpr int kOffK = (PAIR ? 4 : 2) * kCodes;
    static constexpr int kOffV = kOffK + KR * kCodes;
    static constexpr int kOffV16 = kOffV + VR * kCodes;
    static constexpr int kOffScale = kOffV16 + 2 * kCodes * 2;  // float4 [kScaleRing][kGroups]
    static constexpr int kOffNan = kOffScale + kScaleRing * kGroups * 16;  // int [4][kConvWarps]: first slot with a NaN code of V
    static constexpr int kOffQf = kOffNan + 64;  // float [2][256]: the rows' factors
    static constexpr int kOffX = kOffQf + 2 * 2 * kRows * 4;  // float2 [2][128]: the streams' references and sums (split)
    static constexpr int kOffCursor = kOffX + (PAIR ? 0 : 2 * kRows * 8);
    static constexpr int kOffBar = kOffCursor + 32;
    // kfull kempty [KR], vfull vempty [VR], wfull wempty [2], sfull [2], pfull odone [2][2], qfull qfree [2], xfull xdone turn [2] drain [2], qseen [2][4], scfull
    static constexpr int kBars = 2 * KR + 2 * VR + 4 + 10 + 18 + kScaleRing;
    static constexpr int kOffMisc = kOffBar + kBars * 8;  // TMEM slot, flag
    static constexpr int kOffTables = kOffMisc + 8;
    static constexpr int bytes(int B) { return kOffTables + chunks::table_bytes(B) + 1024; }  // + alignment
    static_assert(kOffCursor % 16 == 0 && kOffTables % 8 == 0, "alignment");
    // scales of a tile are written once those kScaleRing before it are done with
    static_assert(kScaleRing >= VR + 3, "V of a tile requested means that the products VR + 2 before it are done");
};

__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b, float c) {
    asm("{\n.reg .b64 ra, rb, rc, rd;\nmov.b64 ra, {%2, %3};\nmov.b64 rb, {%4, %4};\nmov.b64 rc, {%5, %5};\n"
        "fma.rn.f32x2 rd, ra, rb, rc;\nmov.b64 {%0, %1}, rd;\n}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1) {
    asm("{\n.reg .b64 ra, rd;\nmov.b64 rd, {%0, %1};\nmov.b64 ra, {%2, %3};\nadd.rn.f32x2 rd, rd, ra;\nmov.b64 {%0, %1}, rd;\n}"
        : "+f"(d0), "+f"(d1) : "f"(a0), "f"(a1));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// four e4m3 codes -> two pairs of f16
__device__ __forceinline__ void codes_to_f16(uint32_t c, uint32_t& lo, uint32_t& hi) {
    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(lo), "=r"(hi) : "r"(c));
}
// kind::f16 with f16 A and B, float32 D; A K-major, B MN-major
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
    return (1u << 4) | (1u << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// D(tmem) (+)= A(tmem) * B(smem), issued by a whole warp in step
__device__ __forceinline__ void mma_f16_ta_warp(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n.reg .pred p, e;\nsetp.ne.b32 p, %4, 0;\nelect.sync _|e, 0xffffffff;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// A wait by a whole warp: true if the phase completed for every lane.  (A suspended try comes back
// late: limits that are shorter than that, set to make waits run out, are kept by polling.)
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint32_t lim) {
    bool done = umma::mbar_test(bar, parity);
    if (!done) {
        const uint32_t t0 = (uint32_t)clock64();
        do done = lim < 65536 ? umma::mbar_test(bar, parity) : umma::mbar_try(bar, parity);
        while (!done && (uint32_t)clock64() - t0 <= lim);
    }
    return __all_sync(0xffffffffu, done);
}

// Offset of 16-byte chunk c of row r of a tile of D-byte rows as TMA and the tensor core lay it
// out: 128-byte swizzle (D = 128) or 64-byte swizzle (D = 64).
template <int D>
__device__ __forceinline__ uint32_t code_offset(int r, int c) {
    if constexpr (D == 128) return (uint32_t)((r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4));
    else return (uint32_t)((r >> 3) * 512 + (r & 7) * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}
template <int D>
__device__ __forceinline__ uint64_t code_desc(uint32_t addr) {
    if constexpr (D == 128) return umma::desc_sw128(addr, 16, 1024);
    else return umma::desc_sw64(addr, 16, 512);
}

// Eight values of a query row as two planes; f: the row's power of two, which brings them to
// where f16 holds all of their bits that the planes do.
__device__ __forceinline__ void split_planes(const uint4& x, float f, uint2& hi, uint2& lo) {
    const uint32_t v[4] = {x.x, x.y, x.z, x.w};
    uint16_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t q = pack_f16(bf16_lo(v[i]) * f, bf16_hi(v[i]) * f);
        asm("{\n.reg .b32 g, r;\ncvt.rn.satfinite.e4m3x2.f16x2 %0, %2;\ncvt.rn.f16x2.e4m3x2 g, %0;\nsub.f16x2 r, %2, g;\n"
            "cvt.rn.satfinite.e5m2x2.f16x2 %1, r;\n}"
            : "=&h"(h[i]), "=h"(l[i]) : "r"(q));
    }
    hi = make_uint2((uint32_t)h[0] | (uint32_t)h[1] << 16, (uint32_t)h[2] | (uint32_t)h[3] << 16);
    lo = make_uint2((uint32_t)l[0] | (uint32_t)l[1] << 16, (uint32_t)l[2] | (uint32_t)l[3] << 16);
}

// 32 bytes, both 16-byte halves at once where the address allows
__device__ __forceinline__ void store32(uint16_t* p, const uint32_t (&w)[8], bool aligned) {
    if (aligned) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
                     "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(p + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// What a score is multiplied with; never 0, so that a masked one stays -inf.
__device__ __forceinline__ float factor(float k, float qf) { return fmaxf(k * qf, FLT_MIN); }

__device__ __forceinline__ float max16(const float (&v)[16]) {
    float m0 = v[0], m1 = v[1];
#pragma unroll
    for (int e = 2; e < 14; e += 4) {
        m0 = max3(m0, v[e], v[e + 1]);
        m1 = max3(m1, v[e + 2], v[e + 3]);
    }
    return max3(m0, m1, fmaxf(v[14], v[15]));
}

// Weights of 16 scores of one page, 2^(v * kc + off), as f16; their sum / vs added to l.
__device__ __forceinline__ void row_weights(const float (&v)[16], float kc, float off, float per_vs, uint32_t* p, float& l) {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
        float x0, x1;
        fma2(x0, x1, v[e], v[e + 1], kc, off);
        x0 = umma::exp2_approx(x0);
        x1 = umma::exp2_approx(x1);
        add2(s0, s1, x0, x1);
        p[e / 2] = pack_f16(x0, x1);
    }
    l = fmaf(s0 + s1, per_vs, l);
}

template <int D, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) chunk_attn_q8_umma_kernel(const __grid_constant__ CUtensorMap tmk,
                                                                         const __grid_constant__ CUtensorMap tmv,
                                                                         const ChunkArgs a) {
    using namespace umma;
    using L = USmem<D, PAIR>;
    constexpr int KR = L::KR, VR = L::VR, kScaleRing = L::kScaleRing;
    constexpr uint32_t kOCol = 128, kSCol = 256, kCols = 512;  // O_s at 128 s, S_s at 256 + 128 s
    extern __shared__ uint8_t smem_raw[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t* base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t base_a = smem_addr(base);
    const uint32_t bar = base_a + L::kOffBar;
    const uint32_t kfull = bar, kempty = kfull + 8 * KR, vfull = kempty + 8 * KR, vempty = vfull + 8 * VR, wfull = vempty + 8 * VR,
                   wempty = wfull + 16, sfull = wempty + 16, pfull = sfull + 16, odone = pfull + 32, qfull = odone + 32, qfree = qfull + 16,
                   xfull = qfree + 16, xdone = xfull + 8, turn = xdone + 8, drain = turn + 16, qseen = drain + 16, scfull = qseen + 64;
    float4* s_scale = reinterpret_cast<float4*>(base + L::kOffScale);
    volatile int* s_nan = reinterpret_cast<volatile int*>(base + L::kOffNan);
    float* s_qf = reinterpret_cast<float*>(base + L::kOffQf);
    int* s_cursor = reinterpret_cast<int*>(base + L::kOffCursor);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + L::kOffMisc);
    volatile int* flag = reinterpret_cast<volatile int*>(base + L::kOffMisc + 4);
    const chunks::Work& w = a.work;
    const chunks::Tables tab(base + L::kOffTables, w.B);
    const uint32_t lim = (uint32_t)min(g_wait_limit, kDefaultWaitCycles);

    if (warp == kTmaWarp && lane == 0) {
        for (int i = 0; i < L::kBars; ++i) mbar_init(bar + 8 * i, 1);
        for (int i = 0; i < VR; ++i) mbar_init(vempty + 8 * i, kConvWarps);
        for (int i = 0; i < 2; ++i) mbar_init(wfull + 8 * i, kConvWarps);
        if (PAIR) {  // both streams' products are done with a tile
            for (int i = 0; i < KR; ++i) mbar_init(kempty + 8 * i, 2);
            for (int i = 0; i < 2; ++i) mbar_init(wempty + 8 * i, 2);
        }
        if (!PAIR) mbar_init(qfree, 2);  // (both streams are done with the one block of queries)
        for (int i = 0; i < 4; ++i) mbar_init(pfull + 8 * i, 4);
        for (int i = 0; i < 2; ++i) mbar_init(qfull + 8 * i, kConvWarps);
        for (int i = 0; i < 8; ++i) mbar_init(qseen + 8 * i, kConvWarps);
        mbar_init(xfull, 8);
        mbar_init(xdone, 8);
        mbar_init_fence();
        *flag = 0;
        prefetch_tmap(&tmk);
        prefetch_tmap(&tmv);
    }
    if (warp == 0) tmem_alloc(tmem_slot, kCols);
    pdl_wait();
    pdl_trigger();
    chunks::fill_tables(w, a.kv_len, a.last, tab);
    const uint32_t total = tab.first[w.B];
    const uint32_t g0 = w.share(total, blockIdx.x), g1 = w.share(total, blockIdx.x + 1);
    if (warp == 0 && g0 < g1) {
        const chunks::Cursor c = chunks::cursor_at(w, tab, g0);
        if (lane == 0) {
            s_cursor[0] = c.b; s_cursor[1] = c.j; s_cursor[2] = c.h; s_cursor[3] = (int)c.begin;
        }
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    auto first_unit = [&] {
        chunks::Cursor c;
        c.b = c.j = c.h = c.L = c.n = c.tiles = 0;
        c.begin = g1;
        if (g0 < g1) {
            c.b = s_cursor[0]; c.j = s_cursor[1]; c.h = s_cursor[2];
            c.begin = (uint32_t)s_cursor[3];
            c.set(w, tab);
        }
        return c;
    };
    chunks::Cursor at = first_unit();
    const uint32_t g_magic = (65536u + a.G - 1) / a.G;  // r / G for r < 256, G <= 64
    auto token_of = [&](int r) { return (int)((uint32_t)r * g_magic >> 16); };
    int issued_k = 0, issued_v = 0;  // tiles requested
    bool ok = true;

    if (warp >= kMmaWarp && warp < kTmaWarp) {
        // -------------------------------- MMA --------------------------------
        constexpr uint32_t idesc_hi = idesc_f8(kRows, kTile, 0, 0, 0, 0), idesc_lo = idesc_f8(kRows, kTile, 1, 0, 0, 0);
        constexpr uint32_t idesc_pv = idesc_f16(kRows, D);
        const int s = warp - kMmaWarp;
        const uint64_t dq = code_desc<D>(base_a + (PAIR ? 2 * s : 0) * L::kCodes), dk = code_desc<D>(base_a + L::kOffK);
        const uint64_t dv = desc_sw128(base_a + L::kOffV16, kTile * 128, 1024);
        const uint32_t tO = tmem + s * kOCol, tS = tmem + kSCol + s * 128;
        uint32_t first = 0, segments = 0, had = 0;  // tiles before the segment, the stream's among them
        for (; ok && at.begin < g1; at.next(w, tab)) {
            const int nt = at.end_tile(w, g1) - at.first_tile(w, g0);
            if (nt <= 0) continue;
            const int ns = PAIR ? nt : (nt + 1 - s) / 2;  // tiles of the stream
            auto tile_of = [&](int i) { return first + (PAIR ? i : 2 * i + s); };
            auto issue_s = [&](int i) {
                const uint32_t tile = tile_of(i), slot = tile % KR;
                if (!warp_wait(kfull + 8 * slot, (tile / KR) & 1, lim)) return false;
                const uint64_t k = dk + (uint64_t)((slot * L::kCodes) >> 4);
#pragma unroll
                for (int c = 0; c < D / 32; ++c) mma_f8_warp(tS, dq + 2 * c, k + 2 * c, idesc_hi, c > 0);
#pragma unroll
                for (int c = 0; c < D / 32; ++c) mma_f8_warp(tS, dq + (L::kCodes >> 4) + 2 * c, k + 2 * c, idesc_lo, 1);
                commit_warp(sfull + 8 * s);
                commit_warp(kempty + 8 * slot);
                if (i + 1 == ns) commit_warp(qfree + (PAIR ? 8 * s : 0));
                return true;
            };
            ok = warp_wait(qfull + (PAIR ? 8 * s : 0), segments & 1, lim);
            fence_after_sync();
            if (ns) ok = ok && issue_s(0);
            else if (lane == 0) mbar_arrive(qfree);
            for (int i = 0; i < ns && ok; ++i) {
                const uint32_t tile = tile_of(i), slot = tile & 1;
                const uint64_t v = dv + (uint64_t)((slot * L::kCodes * 2) >> 4);
                ok = warp_wait(wfull + 8 * slot, (tile >> 1) & 1, lim);
                for (int h = 0; h < 2 && ok; ++h) {
                    ok = warp_wait(pfull + 8 * (2 * s + h), (had + i) & 1, lim);
                    // The streams take turns with a tile's second PV and the next scores: issued side by
                    // side both take twice as long, and both streams wait at the same time.
                    if (PAIR && h && ok && (s || had + i)) ok = warp_wait(turn + 8 * s, (had + i - (s ? 0 : 1)) & 1, lim);
                    if (!ok) break;
                    fence_after_sync();
#pragma unroll
                    for (int k = 0; k < kHalf / 16; ++k)
                        mma_f16_ta_warp(tO, tS + 32 * h + 8 * k, v + (((4 * h + k) * 2048) >> 4), idesc_pv, (i > 0 || h > 0 || k > 0) ? 1u : 0u);
                    commit_warp(odone + 8 * (2 * s + h));
                }
                if (!ok) break;
                commit_warp(wempty + 8 * slot);
                if (i + 1 < ns) ok = issue_s(i + 1);
                if (PAIR && lane == 0) mbar_arrive(turn + 8 * (s ^ 1));
            }
            first += nt;
            had += ns;
            ++segments;
        }
        if (!ok) *flag = 1;
    } else if (warp == kTmaWarp) {
        // ------------------------- pages, scales, TMA -------------------------
        const int ppt = kTile / a.P;  // pages of a tile
        const int nowhere = a.n_pages * a.Hkv * a.P;  // rows behind the pool read zero
        for (; ok && at.begin < g1; at.next(w, tab)) {
            const int t0 = at.first_tile(w, g0), t1 = at.end_tile(w, g1);
            if (t1 <= t0) continue;
            const int32_t* table = a.page_table + (size_t)at.b * a.M;
            const int pages = (at.L + a.P - 1) / a.P, p0 = t0 * ppt;
            auto page_of = [&](int i) { return i < pages ? table[i] : -1; };
            auto scales_of = [&](int page, float& ks, float& vs) {
                ks = vs = 0.f;  // not readable
                if (page < 0 || page >= a.n_pages) return;
                ks = a.k_scale[(size_t)page * a.Hkv + at.h];
                vs = a.v_scale[(size_t)page * a.Hkv + at.h];
            };
            // 32 pages at a time, one a lane: the next ones' scales and the page numbers behind
            // those are on their way
            int page = page_of(p0 + lane), page1 = page_of(p0 + 32 + lane);
            float ks, vs, ks1, vs1;
            scales_of(page, ks, vs);
            int at_page = 0;
            float4 sc;
            int row;
            auto take = [&] {
                const bool there = q8::scale_ok(ks) && q8::scale_ok(vs);
                const uint32_t u = __float_as_uint(vs);
                const float lg = (u & 0x7fffffu) ? log2f(vs) : (float)((int)(u >> 23) - 127);
                sc = there ? make_float4(ks * a.scale_log2, lg, 1.f / vs, 0.f) : make_float4(1.f, -INFINITY, 0.f, 0.f);
                row = there ? (page * a.Hkv + at.h) * a.P : nowhere;
            };
            scales_of(page1, ks1, vs1);
            int page2 = page_of(p0 + 64 + lane);
            take();
            for (int t = t0; t < t1 && ok; ++t) {
                const uint32_t kslot = (uint32_t)issued_k % KR, vslot = (uint32_t)issued_v % VR;
                const int i = lane - at_page;  // page of the tile
                const bool mine = i >= 0 && i < ppt;
                if (issued_k >= KR) ok = warp_wait(kempty + 8 * kslot, (uint32_t)(issued_k / KR - 1) & 1, lim);
                if (!ok) break;
                if (lane == 0) mbar_expect_tx(kfull + 8 * kslot, L::kCodes);
                __syncwarp();
                if (mine) tma_load_2d(base_a + L::kOffK + kslot * L::kCodes + i * a.P * D, &tmk, 0, row, kfull + 8 * kslot);
                const uint32_t sslot = (uint32_t)issued_k % kScaleRing;
                ++issued_k;
                if (mine)
                    for (int g = 0; g < a.P / 16; ++g) s_scale[sslot * kGroups + i * (a.P / 16) + g] = sc;
                __syncwarp();
                if (lane == 0) mbar_arrive(scfull + 8 * sslot);
                if (issued_v >= VR) ok = warp_wait(vempty + 8 * vslot, (uint32_t)(issued_v / VR - 1) & 1, lim);
                if (!ok) break;
                if (lane == 0) mbar_expect_tx(vfull + 8 * vslot, L::kCodes);
                __syncwarp();
                if (mine) tma_load_2d(base_a + L::kOffV + vslot * L::kCodes + i * a.P * D, &tmv, 0, row, vfull + 8 * vslot);
                ++issued_v;
                at_page += ppt;
                if (at_page == 32 && t + 1 < t1) {
                    at_page = 0;
                    const int next = p0 + (t + 1 - t0) * ppt;
                    page = page1; ks = ks1; vs = vs1;
                    page1 = page2;
                    scales_of(page1, ks1, vs1);
                    page2 = page_of(next + 64 + lane);
                    take();
                }
            }
        }
        if (!ok) *flag = 1;
    } else if (warp == kZeroWarp) {
        // Units that see nothing, by the share that they begin in: rows of zeros.  A warp of its own,
        // 32 values of 16 bytes side by side (row by row in the softmax warps, such a unit cost as
        // much as five tiles).
        for (; at.begin < g1; at.next(w, tab)) {
            if (at.tiles || at.begin < g0) continue;
            const int tokens = min(w.tb, w.T - at.j * w.tb);
            uint16_t* out = static_cast<uint16_t*>(a.out) + (((size_t)at.b * w.T + at.j * w.tb) * a.Hq + at.h * a.G) * D;
            for (int i = lane; i < tokens * a.G * (D / 8); i += 32) {
                const int r = i / (D / 8), t = token_of(r);
                *reinterpret_cast<uint4*>(out + ((size_t)t * a.Hq + r - t * a.G) * D + i % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
            }
        }
    } else if (warp >= kConvWarp) {
        // ---------------- queries to planes, V codes to f16 ----------------
        const int cw = warp - kConvWarp;
        uint32_t tile = 0, segments = 0;
        for (; ok && at.begin < g1; at.next(w, tab)) {
            const int t0 = at.first_tile(w, g0), nt = at.end_tile(w, g1) - t0;
            if (nt <= 0) continue;
            {
                // Rows two by two (D = 128) or four by four, sixteen bytes a lane: a row's largest value
                // by shuffles; the next eight loads are on their way meanwhile.
                // (PAIR: stream 0's rows first, so that it can go on while stream 1 still works)
                constexpr int W = D / 8, PER = 32 / W, ROWS = kRows / kConvWarps, PASSES = ROWS / PER, B = PASSES < 8 ? PASSES : 8;
                const uint16_t* q = static_cast<const uint16_t*>(a.q) + (((size_t)at.b * w.T + at.j * w.tb) * a.Hq + at.h * a.G) * D + lane % W * 8;
                const int see0 = at.L - at.n + at.j * w.tb, left = min(w.tb, at.n - at.j * w.tb);
                auto row_of = [&](int p) { return p / PASSES * kRows + cw * ROWS + p % PASSES * PER + lane / W; };
                auto load = [&](int p, uint4 (&x)[B]) {
#pragma unroll
                    for (int k = 0; k < B; ++k) {
                        const int r = row_of(p + k), t = token_of(r);
                        x[k] = make_uint4(0, 0, 0, 0);
                        if (t < left && see0 + t >= 0) x[k] = *reinterpret_cast<const uint4*>(q + ((size_t)t * a.Hq + (r - t * a.G)) * D);
                    }
                };
                uint4 x[B];
                load(0, x);
#pragma unroll 1
                for (int p = 0; p < (PAIR ? 2 : 1) * PASSES; p += B) {
                    uint4 ahead[B];
                    if (p + B < (PAIR ? 2 : 1) * PASSES) load(p + B, ahead);
                    if (segments && p % PASSES == 0) ok = warp_wait(qfree + 8 * (p / PASSES), (segments - 1) & 1, lim);
                    if (!ok) break;
#pragma unroll
                    for (int k = 0; k < B; ++k) {
                        const int r = row_of(p + k);
                        const uint32_t v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
                        uint32_t m = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) m = max(m, max(v[e] & 0x7fffu, v[e] >> 16 & 0x7fffu));
#pragma unroll
                        for (int o = W / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                        const bool finite = m < 0x7f80u;  // otherwise the row's results are NaN
                        // largest |q| in [2^e, 2^(e + 1)) goes to [2^7, 2^8)
                        const int e = max((int)(m >> 7) - 127, -119);
                        uint2 hi, lo;
                        split_planes(finite ? x[k] : make_uint4(0, 0, 0, 0), __uint_as_float((uint32_t)(7 - e + 127) << 23), hi, lo);
                        uint8_t* to = base + 2 * (r >> 7) * L::kCodes + code_offset<D>(r & 127, lane % W >> 1) + (lane & 1) * 8;
                        *reinterpret_cast<uint2*>(to) = hi;
                        *reinterpret_cast<uint2*>(to + L::kCodes) = lo;
                        if (lane % W == 0) s_qf[(segments & 1) * 2 * kRows + r] = finite ? __uint_as_float((uint32_t)(e - 7 + 127) << 23) : -1.f;
                    }
                    if ((p + B) % PASSES == 0) {
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(qfull + 8 * (p / PASSES));
                            mbar_arrive(qseen + 8 * (4 * (p / PASSES) + segments % 4));
                        }
                    }
#pragma unroll
                    for (int k = 0; k < B; ++k) x[k] = ahead[k];
                }
                if (!ok) break;
                ++segments;
                // the next unit's queries into L2: 128 bytes a lane
                chunks::Cursor n = at;
                n.next(w, tab);
                if (n.begin < g1) {
                    const int rows = (PAIR ? 2 : 1) * kRows, tokens = min(w.tb, n.n - n.j * w.tb);
                    for (int i = cw * 32 + lane; i < rows * D / 64; i += kConvWarps * 32) {
                        const int r = i / (D / 64), t = token_of(r);
                        if (t < tokens)
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint16_t*>(a.q) +
                                (((size_t)n.b * w.T + n.j * w.tb + t) * a.Hq + n.h * a.G + r - t * a.G) * D + i % (D / 64) * 64));
                    }
                }
            }
            const int first_nan = (segments - 1) % 4 * kConvWarps + cw;
            if (lane == 0) s_nan[first_nan] = 0x7fffffff;
            for (int t = 0; t < nt; ++t, ++tile) {
                const uint32_t vslot = tile % VR, slot = tile & 1;
                ok = warp_wait(vfull + 8 * vslot, (tile / VR) & 1, lim);
                if (ok && tile >= 2) ok = warp_wait(wempty + 8 * slot, ((tile >> 1) - 1) & 1, lim);
                if (!ok) break;
                const uint8_t* from = base + L::kOffV + vslot * L::kCodes;
                uint8_t* to = base + L::kOffV16 + slot * L::kCodes * 2;
                constexpr int C = D / 16;  // 16-code chunks of a key
                // each warp has 32 keys
                uint32_t bad = 0;
                auto place = [&](int key, int c, const uint32_t (&o)[8]) {
                    // (the two halves in an order that spreads a quarter warp over all banks)
                    const uint4 h0 = make_uint4(o[0], o[1], o[2], o[3]), h1 = make_uint4(o[4], o[5], o[6], o[7]);
                    const int swap = (c >> 2) & 1;
                    *reinterpret_cast<uint4*>(to + sw128_offset(key, 2 * c + swap, kTile)) = swap ? h1 : h0;
                    *reinterpret_cast<uint4*>(to + sw128_offset(key, 2 * c + 1 - swap, kTile)) = swap ? h0 : h1;
                };
#pragma unroll 4
                for (int i = 0; i < C; ++i) {
                    const int x = i * 32 + lane, key = cw * 32 + x / C, c = x % C;
                    const uint4 v = *reinterpret_cast<const uint4*>(from + key * D + c * 16);
                    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
                    uint32_t o[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        bad |= (in[e] & 0x7f7f7f7fu) + 0x01010101u;
                        codes_to_f16(in[e], o[2 * e], o[2 * e + 1]);
                    }
                    place(key, c, o);
                }
                if (__any_sync(0xffffffffu, bad & 0x80808080u)) {  // once more, with zeros for NaN codes
                    int nan_slot = 0x7fffffff;
#pragma unroll 1
                    for (int i = 0; i < C; ++i) {
                        const int x = i * 32 + lane, key = cw * 32 + x / C, c = x % C;
                        const uint4 v = *reinterpret_cast<const uint4*>(from + key * D + c * 16);
                        const uint32_t in[4] = {v.x, v.y, v.z, v.w};
                        uint32_t o[8], any = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t n = ((in[e] & 0x7f7f7f7fu) + 0x01010101u) >> 7 & 0x01010101u;
                            any |= n;
                            codes_to_f16(in[e] & ~(n * 0xffu), o[2 * e], o[2 * e + 1]);
                        }
                        if (any) nan_slot = min(nan_slot, (t0 + t) * kTile + key);
                        place(key, c, o);
                    }
                    nan_slot = __reduce_min_sync(0xffffffffu, nan_slot);
                    if (lane == 0) s_nan[first_nan] = min(s_nan[first_nan], nan_slot);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(vempty + 8 * vslot);
                    mbar_arrive(wfull + 8 * slot);
                }
            }
            if (!ok) break;
        }
        if (!ok) *flag = 1;
    } else {
        // ------------------------------ softmax ------------------------------
        const int s = warp >> 2, r = tid & 127, row = PAIR ? tid : r;  // row of the unit
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + kSCol + s * 128, tO = tmem + lane_off + s * kOCol;
        const int token_in = token_of(row), head_in = row - token_in * a.G;
        uint32_t tile = 0, segments = 0, had[2] = {0, 0};  // tiles before the segment: all, the streams'
        for (; ok && at.begin < g1; at.next(w, tab)) {
            const int t0 = at.first_tile(w, g0), nt = at.end_tile(w, g1) - t0;
            const int token = at.j * w.tb + token_in;
            const bool real = token_in < w.tb && token < w.T;
            uint16_t* out = static_cast<uint16_t*>(a.out) + (((size_t)at.b * w.T + token) * a.Hq + at.h * a.G + head_in) * D;
            if (nt <= 0) continue;
            const int limit = real && token < at.n ? at.L - at.n + token : -1;  // the last slot that the row sees
            const bool any = __any_sync(0xffffffffu, limit >= 0);
            // ---- tiles ----
            float ref = -INFINITY, l = 0.f, qf = 0.f;  // qf < 0: the row's query is not finite
            const int ns = PAIR ? nt : (nt + 1 - s) / 2;
            if (ns) {
                // The rows' factors.  (Where segments have one tile, the queries of the next segment, and in time
                // those behind them, can be ready before this warp has handed out the results of the last
                // one: a barrier of two phases would be misread, so there are four, used in turn.)
                ok = warp_wait(qseen + 8 * ((PAIR ? 4 * s : 0) + segments % 4), segments / 4 & 1, lim);
                if (!ok) break;
                qf = s_qf[(segments & 1) * 2 * kRows + row];
            }
            for (int i = 0; i < ns && ok; ++i) {
                const int x = PAIR ? i : 2 * i + s;  // tile of the segment
                const uint32_t n_tile = tile + x, n_mine = had[s] + i;
                ok = warp_wait(scfull + 8 * (n_tile % kScaleRing), (n_tile / kScaleRing) & 1, lim);
                if (!ok) break;
                const float4* sc = s_scale + (n_tile % kScaleRing) * kGroups;
                float kc[4], off[4], per_vs[4];
                auto scales = [&](int h) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const float4 f = sc[4 * h + g];
                        kc[g] = factor(f.x, fabsf(qf));
                        off[g] = f.y;
                        per_vs[g] = f.z;
                    }
                };
                scales(0);
                ok = warp_wait(sfull + 8 * s, n_mine & 1, lim);
                if (!ok) break;
                if (!any) {
                    if (lane == 0) {
                        mbar_arrive(pfull + 16 * s);
                        mbar_arrive(pfull + 16 * s + 8);
                    }
                    continue;
                }
                fence_after_sync();
                // the last key of the tile that the row sees (rows that see nothing: what they sum up is not used)
                const int seen = limit < 0 ? kTile : limit - (t0 + x) * kTile;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    float v[4][16];
#pragma unroll
                    for (int g = 0; g < 4; ++g) tmem_ld16(tS + kHalf * h + 16 * g, v[g]);
                    const int see = seen - kHalf * h;
                    const bool plain = __all_sync(0xffffffffu, see >= kHalf - 1);
                    tmem_wait_ld();
                    if (!plain) {
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            if (!__all_sync(0xffffffffu, see >= 16 * g + 15)) {
#pragma unroll
                                for (int e = 0; e < 16; ++e) v[g][e] = 16 * g + e <= see ? v[g][e] : -INFINITY;
                            }
                    }
                    // Weights on the reference so far; formed anew where it turns out that it has to move.
                    float sum = 0.f;
                    float top = -INFINITY;
#pragma unroll
                    for (int g = 0; g < 4; ++g) top = fmaxf(top, fmaf(max16(v[g]), kc[g], off[g]));
                    const bool up = top > -INFINITY && !(top <= ref + kMove);
                    if (__any_sync(0xffffffffu, up)) {
                        // The reference moves to a whole number, so that what is scaled keeps its bits.
                        const float to = up ? ceilf(top) : ref;
                        const float corr = up && ref > -INFINITY ? exp2_approx(ref - to) : 1.f;
                        ref = to;
                        l *= corr;
                        if (__any_sync(0xffffffffu, corr != 1.f) && (i || h)) {  // (else there is no O yet)
                            if (h) ok = warp_wait(odone + 16 * s, n_mine & 1, lim);  // the products of the half before
                            if (!ok) break;
                            fence_after_sync();
#pragma unroll 1
                            for (int k = 0; k < D / 16; ++k) {
                                float o[16];
                                tmem_ld16(tO + 16 * k, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] *= corr;
                                tmem_st16(tO + 16 * k, o);
                            }
                        }
                    }
                    {
                        const float shift = kLift - (ref == -INFINITY ? 0.f : ref);
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t p[16];
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int g = 2 * c + k;
                                row_weights(v[g], kc[g], off[g] + shift, per_vs[g], p + 8 * k, sum);
                            }
                            tmem_st16u(tS + 32 * h + 16 * c, p);
                        }
                    }
                    l += sum;
                    tmem_wait_st();
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(pfull + 8 * (2 * s + h));
                    if (!h) scales(1);
                }
            }
            if (!ok) break;
            tile += nt;
            had[0] += PAIR ? nt : (nt + 1) / 2;
            had[1] += PAIR ? nt : nt / 2;
            // ---- results ----
            const bool whole = nt == at.tiles;
            const bool split = !PAIR && nt > 1;  // both streams have an O
            if (limit < 0) { ref = -INFINITY; l = 0.f; }
            if (qf < 0.f && l != 0.f) l = NAN;  // (its planes are zero, so that l says whether it sees a key)
            float m_out = ref, l_out = l, f0 = 1.f, f1 = 0.f;  // f: factors of this stream's O, or of both streams'
            if constexpr (!PAIR) {
                float2* s_x = reinterpret_cast<float2*>(base + L::kOffX);
                s_x[s * kRows + r] = make_float2(ref, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(xfull);
                ok = warp_wait(xfull, segments & 1, lim);
                if (!ok) break;
                const float2 A = s_x[r], B = s_x[kRows + r];
                m_out = fmaxf(A.x, B.x);
                const float z = m_out == -INFINITY ? 0.f : m_out;
                f0 = exp2f(A.x - z);
                f1 = exp2f(B.x - z);
                l_out = A.y * f0 + B.y * f1;
            }
            // (a commit comes with all products before it)
            if (PAIR || s == 0 || split) ok = warp_wait(odone + 8 * (2 * s + 1), (had[s] - 1) & 1, lim);
            if (!PAIR && ok && (s == 1 || split)) ok = warp_wait(odone + 8 * (2 * (s ^ 1) + 1), (had[s ^ 1] - 1) & 1, lim);
            if (!ok) break;
            fence_after_sync();
            {
                int nan_slot = 0x7fffffff;
                for (int k = 0; k < kConvWarps; ++k) nan_slot = min(nan_slot, s_nan[segments % 4 * kConvWarps + k]);
                if (limit >= nan_slot) l_out = NAN;
            }
            const size_t part = (size_t)(2 * blockIdx.x + (t0 > 0 ? 0 : 1)) * a.rows + row;
            const bool zero = whole && l_out == 0.f;
            if (whole) {
                const float inv = zero ? 0.f : 1.f / l_out;
                f0 *= inv;
                f1 *= inv;
            } else if (real && (PAIR || s == 0)) {
                a.part_ml[part] = make_float2(m_out, l_out);
            }
            constexpr int WC = D / (PAIR ? 1 : 2);  // columns of a warpgroup
            const int col0 = PAIR ? 0 : s * WC;
            const uint32_t from = tmem + lane_off + (PAIR ? s * kOCol : 0) + col0;
            const bool aligned = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
            if (any) {
#pragma unroll 1
                for (int c = 0; c < WC; c += 32) {
                    float o[32];
                    tmem_ld32(from + c, o);
                    if (split) {
                        float o1[32];
                        tmem_ld32(from + kOCol + c, o1);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = o[e] * f0 + o1[e] * f1;
                    } else {
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= f0;
                    }
                    if (!real) continue;
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 16) {
                            uint32_t b[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) b[k] = zero ? 0u : pack_bf16(o[e + 2 * k], o[e + 2 * k + 1]);
                            store32(out + col0 + c + e, b, aligned);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4*>(a.part_o + part * D + col0 + c + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
            } else if (real && whole) {  // a warp without rows that see anything
                for (int c = 0; c < WC; c += 8) *reinterpret_cast<uint4*>(out + col0 + c) = make_uint4(0, 0, 0, 0);
            }
            if constexpr (!PAIR) {
                // the other stream has read both O and the exchanged sums
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(xdone);
                ok = warp_wait(xdone, segments & 1, lim);
            }
            ++segments;
        }
        if (!ok) *flag = 1;
    }
    __syncthreads();
    const bool bad = *flag != 0;  // every write to the flag precedes the barrier
    if (bad) {
        // Gave up: let everything this CTA started complete before its tensor memory is freed
        // and it leaves (default-limit waits), and mark what it owns.
        if (warp >= kMmaWarp && warp < kTmaWarp) {
            commit_warp(drain + 8 * (warp - kMmaWarp));
            warp_wait(drain + 8 * (warp - kMmaWarp), 0, kDrainCycles);
        }
        if (warp == kTmaWarp) {
            for (int u = max(0, issued_k - KR); u < issued_k; ++u) warp_wait(kfull + 8 * (u % KR), (uint32_t)(u / KR) & 1, kDrainCycles);
            for (int u = max(0, issued_v - VR); u < issued_v; ++u) warp_wait(vfull + 8 * (u % VR), (uint32_t)(u / VR) & 1, kDrainCycles);
        }
        if (tid == 0) atomicExch(&g_wait_gave_up, 1);
        for (chunks::Cursor c = first_unit(); c.begin < g1; c.next(w, tab)) {
            const int t0 = c.first_tile(w, g0), nt = c.end_tile(w, g1) - t0;
            if (nt <= 0) continue;
            for (int i = tid; i < a.rows; i += kThreads) {
                const int token = c.j * w.tb + i / a.G;
                if (nt < c.tiles) {
                    a.part_ml[(size_t)(2 * blockIdx.x + (t0 > 0 ? 0 : 1)) * a.rows + i] = make_float2(0.f, NAN);
                } else if (i / a.G < w.tb && token < w.T) {
                    uint16_t* o = static_cast<uint16_t*>(a.out) + (((size_t)c.b * w.T + token) * a.Hq + c.h * a.G + i % a.G) * D;
                    for (int e = 0; e < D; e += 8) *reinterpret_cast<uint4*>(o + e) = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
                }
            }
        }
    }
    // an empty share gives nothing to the units around it
    if (!w.whole) {
        if (g0 >= g1 && tid < a.rows) a.part_ml[(size_t)2 * blockIdx.x * a.rows + tid] = make_float2(-INFINITY, 0.f);
        if (warp == 1) {
            const int4 p = chunks::plan_share(w, tab, g0, g1);
            if (lane == 0) a.plan[blockIdx.x] = p;
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, kCols);
}

// Joins the partial results.  Block (c, y): the unit that share c begins and others finish;
// rows from y * kMergeThreads / (D / 4) on, four columns a thread, eight shares' loads in
// flight at once.
constexpr int kMergeThreads = 256, kMergeBatch = 8;
template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) chunk_merge_kernel(const ChunkArgs a) {
    pdl_wait();
    pdl_trigger();
    const int c0 = blockIdx.x;
    const int4 plan = a.plan[c0];
    const int c1 = plan.x, i = blockIdx.y * (kMergeThreads / (D / 4)) + threadIdx.x / (D / 4), d = threadIdx.x % (D / 4) * 4;
    const int token = plan.z * a.work.tb + i / a.G;
    if (c1 < 0 || i / a.G >= a.work.tb || token >= a.work.T) return;
    auto slot = [&](int j) { return (size_t)(2 * j + (j == c0 ? 1 : 0)) * a.rows + i; };
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
        const float f0 = exp2f(top - ref);
        top = m;
        l *= f0;
        o.x *= f0; o.y *= f0; o.z *= f0; o.w *= f0;
#pragma unroll
        for (int k = 0; k < kMergeBatch; ++k) {
            // no key seen there: no sums are written (a NaN row keeps its l)
            if (ml[k].x == -INFINITY && ml[k].y == 0.f) continue;
            const float f = exp2f(ml[k].x - ref);
            l += ml[k].y * f;
            o.x += v[k].x * f; o.y += v[k].y * f; o.z += v[k].z * f; o.w += v[k].w * f;
        }
    }
    T* out = static_cast<T*>(a.out) + (((size_t)plan.y * a.work.T + token) * a.Hq + plan.w * a.G + i % a.G) * D + d;
    if (l == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
    store4(out, o, l == 0.f ? 0.f : 1.f / l);
}

// ---------------------------------------------------------------------------
// float32 kernel.  A CTA works through its share of (unit, tile) pairs; a unit has ROWS query
// rows, 16 or 64, a tile 64 keys, dequantised into shared memory once for all rows; scores,
// softmax and sums are float32.  A thread has four rows and KT keys (then CP columns) of each
// product.  Bound by shared memory and issue (147 us for two chunks of 300 rows on 500, 16 / 4 heads, 22
// TFLOP/s), small calls by latency (14 us for nine rows, four heads of 64 and 137 keys).  One token goes
// through a block of 16 rows: 540 us for sixteen sequences of 777 to 16384 keys, 8 heads of 4 rows.
// ---------------------------------------------------------------------------
constexpr int kKeys = 64, kSetupF32 = 1;

template <int D, int ROWS>
struct FSmem {
    static constexpr int kStride = D + 4, kStrideP = kKeys + 4;  // rows 16 bytes apart in the banks
    static constexpr int kOffV = kKeys * kStride * 4;
    static constexpr int kOffQ = kOffV + kKeys * D * 4;
    static constexpr int kOffP = kOffQ + ROWS * kStride * 4;
    static constexpr int kOffStat = kOffP + ROWS * kStrideP * 4;  // corr, m, l, limit
    static constexpr int kOffTables = kOffStat + 4 * ROWS * 4;
    static constexpr int bytes(int B) { return kOffTables + chunks::table_bytes(B); }
    static_assert(kOffTables % 8 == 0, "alignment");
};

template <int D, int ROWS, int THREADS>
__global__ void __launch_bounds__(THREADS) chunk_attn_q8_f32_kernel(const ChunkArgs a) {
    using L = FSmem<D, ROWS>;
    extern __shared__ __align__(16) uint8_t smem[];
    float* sk = reinterpret_cast<float*>(smem);
    float* sv = reinterpret_cast<float*>(smem + L::kOffV);
    float* sq = reinterpret_cast<float*>(smem + L::kOffQ);
    float* sp = reinterpret_cast<float*>(smem + L::kOffP);
    float* s_corr = reinterpret_cast<float*>(smem + L::kOffStat);
    float* s_m = s_corr + ROWS;
    float* s_l = s_m + ROWS;
    int* s_limit = reinterpret_cast<int*>(s_l + ROWS);  // last slot that a row sees
    const chunks::Work& w = a.work;
    const chunks::Tables tab(smem + L::kOffTables, w.B);
    __shared__ int s_there[kKeys], s_bad[kKeys], s_cursor[4];  // key is held; its V has a NaN code
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    chunks::fill_tables(w, a.kv_len, a.last, tab);
    const uint32_t total = tab.first[w.B];
    const uint32_t g0 = w.share(total, blockIdx.x), g1 = w.share(total, blockIdx.x + 1);
    if (warp == 0 && g0 < g1) {
        const chunks::Cursor c = chunks::cursor_at(w, tab, g0);
        if (lane == 0) {
            s_cursor[0] = c.b; s_cursor[1] = c.j; s_cursor[2] = c.h; s_cursor[3] = (int)c.begin;
        }
    }
    __syncthreads();
    chunks::Cursor at;
    at.b = at.j = at.h = at.L = at.n = at.tiles = 0;
    at.begin = g1;
    if (g0 < g1) {
        at.b = s_cursor[0]; at.j = s_cursor[1]; at.h = s_cursor[2];
        at.begin = (uint32_t)s_cursor[3];
        at.set(w, tab);
    }
    // this thread's four rows; its KT keys, KL apart; its CP columns, CW side by side
    constexpr int KT = ROWS * kKeys / (4 * THREADS), KL = kKeys / KT, CP = D * ROWS / (4 * THREADS), CW = CP < 4 ? CP : 4;
    const int r0 = tid / KL * 4, kl = tid % KL;
    auto column = [&](int j) { return (j / CW * KL + kl) * CW + j % CW; };
    for (; at.begin < g1; at.next(w, tab)) {
        const int t0 = at.first_tile(w, g0), t1 = at.end_tile(w, g1);
        if (t1 <= t0 && !(at.tiles == 0 && g0 <= at.begin)) continue;
        auto real = [&](int r) { return r / a.G < w.tb && at.j * w.tb + r / a.G < w.T; };
        auto place = [&](int r) { return (((size_t)at.b * w.T + at.j * w.tb + r / a.G) * a.Hq + at.h * a.G + r % a.G) * D; };
        for (int i = tid; i < ROWS * D; i += THREADS) {
            const int r = i / D;
            const float x = real(r) && at.j * w.tb + r / a.G < at.n ? static_cast<const float*>(a.q)[place(r) + i % D] : 0.f;
            // (an infinity as NaN: scores that are all -inf would look like keys that are not there)
            sq[r * L::kStride + i % D] = fabsf(x) < INFINITY ? x : NAN;
        }
        if (tid < ROWS) {
            s_m[tid] = -INFINITY;
            s_l[tid] = 0.f;
            const int token = at.j * w.tb + tid / a.G;
            s_limit[tid] = real(tid) && token < at.n ? at.L - at.n + token : -1;
        }
        float acc[4][CP];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < CP; ++j) acc[i][j] = 0.f;
        for (int t = t0; t < t1; ++t) {
            __syncthreads();
            if (tid < kKeys) s_bad[tid] = 0;
            __syncthreads();
            const int k0 = t * kKeys;
            // keys of the tile, 8 elements a step; absent ones read zero
            for (int i = tid; i < kKeys * (D / 8); i += THREADS) {
                const int key = i / (D / 8), c = i % (D / 8) * 8, slot = k0 + key;
                float kx[8], vx[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) kx[e] = vx[e] = 0.f;
                bool there = slot < at.L;
                if (there) {
                    const int page = a.page_table[(size_t)at.b * a.M + slot / a.P];
                    there = page >= 0 && page < a.n_pages;
                    if (there) {
                        const size_t unit = (size_t)page * a.Hkv + at.h;
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
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (isnan(vx[e])) { vx[e] = 0.f; s_bad[key] = 1; }
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    *reinterpret_cast<float4*>(sk + key * L::kStride + c + e) = make_float4(kx[e], kx[e + 1], kx[e + 2], kx[e + 3]);
                    *reinterpret_cast<float4*>(sv + key * D + c + e) = make_float4(vx[e], vx[e + 1], vx[e + 2], vx[e + 3]);
                }
                if (c == 0) s_there[key] = there;
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
                    const int key = kl + j * KL;
                    const bool there = s_there[key];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sp[(r0 + i) * L::kStrideP + key] = there && k0 + key <= s_limit[r0 + i] ? z[i][j] * a.scale_log2 : -INFINITY;
                }
            }
            __syncthreads();
            // running maximum and sum, several rows per warp
            constexpr int RW = ROWS * 32 / THREADS;
#pragma unroll 4
            for (int r = RW * warp; r < RW * (warp + 1); ++r) {
                const float x0 = sp[r * L::kStrideP + lane], x1 = sp[r * L::kStrideP + lane + 32];
                float mx = fmaxf(x0, x1);  // (a NaN score makes the row NaN: the sum below carries it)
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float m0 = s_m[r], m1 = fmaxf(m0, mx);
                const float ref = m1 == -INFINITY ? 0.f : m1;
                const float p0 = exp2f(x0 - ref), p1 = exp2f(x1 - ref);
                float sum = warp_sum(p0 + p1);
                const int limit = s_limit[r] - k0;
                if (__any_sync(0xffffffffu, (s_bad[lane] && lane <= limit) || (s_bad[lane + 32] && lane + 32 <= limit))) sum = NAN;
                sp[r * L::kStrideP + lane] = p0;
                sp[r * L::kStrideP + lane + 32] = p1;
                if (lane == 0) {
                    const float c = exp2f(m0 - ref);  // 0 where nothing was seen before
                    s_corr[r] = c;
                    s_m[r] = m1;
                    s_l[r] = s_l[r] * c + sum;
                }
            }
            __syncthreads();
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
        __syncthreads();
        const bool whole = t1 - t0 == at.tiles;
        const size_t part = (size_t)(2 * blockIdx.x + (t0 > 0 ? 0 : 1)) * ROWS;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float l = s_l[r0 + i];
            if (!real(r0 + i)) continue;
            float* out = static_cast<float*>(a.out) + place(r0 + i);
#pragma unroll
            for (int j = 0; j < CP; ++j) {
                if (whole) out[column(j)] = l == 0.f ? 0.f : acc[i][j] / l;
                else a.part_o[(part + r0 + i) * D + column(j)] = acc[i][j];
            }
        }
        if (!whole && tid < ROWS) a.part_ml[part + tid] = make_float2(s_m[tid], s_l[tid]);
        __syncthreads();  // q, statistics free again
    }
    if (!w.whole) {
        // an empty share gives nothing to the units around it
        if (g0 >= g1 && tid < ROWS) a.part_ml[(size_t)2 * blockIdx.x * ROWS + tid] = make_float2(-INFINITY, 0.f);
        if (warp == 0) {
            const int4 p = chunks::plan_share(w, tab, g0, g1);
            if (lane == 0) a.plan[blockIdx.x] = p;
        }
    }
}

// Rows of a unit, keys of a tile, tiles that a unit counts more, CTAs, and the tiles up to
// which units are not cut.
struct Plan {
    int rows, keys, setup, ctas, whole;
};
Plan plan_chunk(medusa_dtype dtype, int T, int G, int D) {
    const long long rows = (long long)T * G;
    const int sms = sm_count();
    if (dtype == MEDUSA_F32) return rows <= 32 && G <= 16 ? Plan{16, kKeys, kSetupF32, 2 * sms, 2} : Plan{64, kKeys, kSetupF32, D == 64 ? 2 * sms : sms, 2};
    return rows <= kRows ? Plan{kRows, kTile, kSetup, sms, 3} : Plan{2 * kRows, kTile, kSetup, sms, 3};
}

// One row a sequence and at most 16 query heads a KV head: the kernel that has the keys in the TMEM
// lanes and the rows in the columns, whose work is in proportion to 16 rows instead of 128.  One token of
// sixteen sequences of 777 to 16384, 32 / 8 heads (282 MB): 74 us here, 54 there; of one sequence of 2048, 32 heads,
// 18 and 13.  Its weights have 9 bits where this kernel's have 11, its q is exact to 2^-17 of its block's largest: for
// those sixteen an output is off by 0.172% (rms) there, 0.167% here, of which rounding to bf16 alone is 0.165%.  A NaN
// code of V makes its own column NaN there, the row here.
bool single_row(medusa_dtype dtype, int T, int G) { return dtype == MEDUSA_BF16 && T == 1 && G <= 16; }

size_t ws_bytes_chunk(const Plan& p, int D) { return (size_t)2 * p.ctas * p.rows * (D + 2) * sizeof(float) + p.ctas * sizeof(int4); }

template <typename T, int D>
cudaError_t launch_merge(const ChunkArgs& a, cudaStream_t st) {
    constexpr int rows = kMergeThreads / (D / 4);  // of a block
    const long long all = (long long)a.work.T * a.G;
    const int most = all < a.rows ? (int)all : a.rows;
    return launch(chunk_merge_kernel<T, D>, dim3(a.work.ctas, (most + rows - 1) / rows), dim3(kMergeThreads), 0, st, a);
}

// (the shared memory limit is the kernel's, not the call's, so it is always what the largest
// batch takes: a call of few sequences on another thread must not lower it under this one)
template <int D, int ROWS, int THREADS>
cudaError_t launch_f32(const ChunkArgs& a, cudaStream_t st) {
    auto kern = chunk_attn_q8_f32_kernel<D, ROWS, THREADS>;
    constexpr int most = FSmem<D, ROWS>::bytes(q8::kMaxBatch);
    static_assert(most + 1024 <= q8::kMaxSmem, "the largest batch does not fit (1024: static arrays)");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess) e = launch(kern, dim3(a.work.ctas), dim3(THREADS), FSmem<D, ROWS>::bytes(a.work.B), st, a);
    if (e == cudaSuccess && !a.work.whole) e = launch_merge<float, D>(a, st);
    return e;
}
template <int D, bool PAIR>
cudaError_t launch_umma(const CUtensorMap& mk, const CUtensorMap& mv, const ChunkArgs& a, cudaStream_t st) {
    auto kern = chunk_attn_q8_umma_kernel<D, PAIR>;
    constexpr int most = USmem<D, PAIR>::bytes(q8::kMaxBatch);
    static_assert(most <= q8::kMaxSmem, "the largest batch does not fit");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess) e = launch(kern, dim3(a.work.ctas), dim3(kThreads), USmem<D, PAIR>::bytes(a.work.B), st, mk, mv, a);
    if (e == cudaSuccess && !a.work.whole) e = launch_merge<uint16_t, D>(a, st);
    return e;
}

// codes [n_pages * Hkv * P][D] in boxes of one (page, head); V is read by threads, K by the
// tensor core
int pages_map(CUtensorMap* m, const void* pages, int D, int P, long long rows, bool swizzled) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return fail(MEDUSA_ERR_CUDA, "chunk_attention_q8: cuTensorMapEncodeTiled is unavailable");
    cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)D};
    cuuint32_t box[2] = {(cuuint32_t)D, (cuuint32_t)P};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(pages), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     !swizzled ? CU_TENSOR_MAP_SWIZZLE_NONE : D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(MEDUSA_ERR_CUDA, "chunk_attention_q8: tensor map encode failed (%d)", (int)r);
    return MEDUSA_OK;
}

}  // namespace
}  // namespace medusa

using namespace medusa;

extern "C" size_t medusa_chunk_attention_q8_workspace(int B, int T, int Hq, int Hkv, int D, medusa_dtype dtype) {
    if (B < 1 || T < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || (D != 64 && D != 128)) return 0;
    return single_row(dtype, T, Hq / Hkv) ? row_attention_q8_workspace(Hq / Hkv, D) : ws_bytes_chunk(plan_chunk(dtype, T, Hq / Hkv, D), D);
}

extern "C" int medusa_chunk_attention_q8(const void* q, medusa_dtype dtype, const void* k_pages, const void* v_pages,
                                         const float* k_scale, const float* v_scale, const int32_t* page_table,
                                         const int32_t* kv_len, const int32_t* last, int B, int T, int Hq, int Hkv, int D,
                                         int P, int n_pages, int M, float scale, void* out, void* ws, size_t ws_bytes,
                                         void* stream) {
    const char* who = "chunk_attention_q8";
    if (B < 1 || T < 1 || Hq < 1 || Hkv < 1 || n_pages < 1 || M < 1)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: sizes must be positive", who);
    if (int rc = q8::check_pool(who, B, Hkv, D, P, n_pages, M)) return rc;
    if (Hq % Hkv || Hq / Hkv > 64 || T > 1 << 20)
        return fail(MEDUSA_ERR_UNSUPPORTED, "%s: unsupported shape (T=%d Hq=%d Hkv=%d)", who, T, Hq, Hkv);
    if (dtype != MEDUSA_F32 && dtype != MEDUSA_BF16) return fail(MEDUSA_ERR_UNSUPPORTED, "%s: unknown dtype %d", who, (int)dtype);
    if (!q || !k_pages || !v_pages || !k_scale || !v_scale || !page_table || !kv_len || !out)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: null pointer", who);
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: q, pages and out must be 16-byte aligned", who);
    if (q == out) return fail(MEDUSA_ERR_INVALID_ARG, "%s: out must not be q", who);
    if (!(scale > 0.f) || !(scale * kLog2e <= FLT_MAX))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: scale must be positive, scale * log2(e) finite", who);
    const int G = Hq / Hkv;
    const Plan p = plan_chunk(dtype, T, G, D);
    const size_t need = medusa_chunk_attention_q8_workspace(B, T, Hq, Hkv, D, dtype);
    if (!ws || ws_bytes < need) return fail(MEDUSA_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", who, need);
    if (!aligned16(ws)) return fail(MEDUSA_ERR_INVALID_ARG, "%s: ws must be 16-byte aligned", who);
    if (single_row(dtype, T, G))
        return row_attention_q8(who, q, k_pages, v_pages, k_scale, v_scale, page_table, kv_len, last, B, Hq, Hkv, D, P, n_pages, M, scale, out,
                                ws, stream);
    ChunkArgs a{};
    a.q = q;
    a.k_pages = (const uint8_t*)k_pages; a.v_pages = (const uint8_t*)v_pages;
    a.k_scale = k_scale; a.v_scale = v_scale;
    a.page_table = page_table; a.kv_len = kv_len; a.last = last; a.out = out;
    a.part_o = (float*)ws;
    a.part_ml = (float2*)((float*)ws + (size_t)2 * p.ctas * p.rows * D);
    a.plan = (int4*)(a.part_ml + (size_t)2 * p.ctas * p.rows);
    a.Hq = Hq; a.Hkv = Hkv; a.G = G; a.P = P; a.M = M; a.n_pages = n_pages; a.rows = p.rows;
    const int tb = p.rows / G, blocks = (T + tb - 1) / tb;
    const long long tiles = ((long long)M * P + p.keys - 1) / p.keys;  // of the longest unit
    const long long units = (long long)B * Hkv * blocks;
    const bool whole = tiles <= p.whole;
    if (units * (whole ? 1 : tiles + p.setup) > 0x7fffffffll)
        return fail(MEDUSA_ERR_UNSUPPORTED, "%s: %d sequences of %d rows and up to %lld tokens are too many tiles", who, B, T, (long long)M * P);
    a.work = chunks::Work{B, T, Hkv, blocks, tb, p.keys, p.setup, M * P, whole && units < p.ctas ? (int)units : p.ctas, whole};
    a.scale_log2 = scale * kLog2e;
    cudaStream_t st = as_stream(stream);
    cudaError_t e;
    if (dtype == MEDUSA_F32) {
        e = p.rows == 16 ? (D == 64 ? launch_f32<64, 16, 256>(a, st) : launch_f32<128, 16, 256>(a, st))
                         : (D == 64 ? launch_f32<64, 64, 256>(a, st) : launch_f32<128, 64, 512>(a, st));
    } else {
        CUtensorMap mk, mv;
        const long long rows = (long long)n_pages * Hkv * P;
        int rc = pages_map(&mk, k_pages, D, P, rows, true);
        if (!rc) rc = pages_map(&mv, v_pages, D, P, rows, false);
        if (rc) return rc;
        if (p.rows == kRows) e = D == 64 ? launch_umma<64, false>(mk, mv, a, st) : launch_umma<128, false>(mk, mv, a, st);
        else e = D == 64 ? launch_umma<64, true>(mk, mv, a, st) : launch_umma<128, true>(mk, mv, a, st);
    }
    if (e != cudaSuccess) return fail(MEDUSA_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    return MEDUSA_OK;
}
