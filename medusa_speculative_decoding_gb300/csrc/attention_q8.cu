// attention_q8.cu -- tree attention over the 8-bit paged cache ("Medusa Heads"
// glossary page, "Tree attention and acceptance").
//
// Query i attends to the prefix keys in the pages (code * scale) and to the
// tree rows m whose bit m of mask row i is set:
//   out = softmax(scale * q.k) v
// The tree's own K and V rows are given in the model's type, next to the cache:
// rejected candidates never reach a page.
//
//   tree_attn_q8_simple_kernel : float32 arithmetic on the CUDA cores
//   attn_q8_merge_kernel       : joins the partial results of units that several
//                                CTAs share (q8.cuh, Work)
#include <float.h>

#include "common.cuh"
#include "q8.cuh"

namespace medusa {
namespace {

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
    q8::Work work;
    int Hq, Hkv, G, P, M, n_pages, W, qblocks;
    float scale_log2;
};

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) {
    uint16_t r;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(v));
    *p = r;
}

// 2^x with x <= 0 or -inf; exp2f is within 2 units in the last place
__device__ __forceinline__ float weight(float x) { return exp2f(x); }

// ---------------------------------------------------------------------------
// One CTA works through its share of (unit, tile) pairs; a unit's block has
// kRows query rows.  Each tile of kKeys keys is dequantised into shared memory
// once for all rows; scores, softmax and sums are float32.
// ---------------------------------------------------------------------------
constexpr int kRows = 16, kKeys = 64, kSimpleThreads = 256;

template <int D>
struct SimpleSmem {
    static constexpr int kStrideK = D + 4;  // rows 16 bytes apart in the banks
    static constexpr int kOffV = kKeys * kStrideK * 4;
    static constexpr int kOffQ = kOffV + kKeys * D * 4;
    static constexpr int kOffP = kOffQ + kRows * D * 4;
    static constexpr int kOffStat = kOffP + kRows * kKeys * 4;  // corr, m, l
    static constexpr int kOffFirst = kOffStat + 3 * kRows * 4;  // tile offsets
    static int bytes(int B) { return kOffFirst + (B + 1) * 8; }
};

template <typename T, int D>
__global__ void __launch_bounds__(kSimpleThreads) tree_attn_q8_simple_kernel(const AttnQ8Args a) {
    using L = SimpleSmem<D>;
    extern __shared__ __align__(16) uint8_t smem[];
    float* sk = reinterpret_cast<float*>(smem);
    float* sv = reinterpret_cast<float*>(smem + L::kOffV);
    float* sq = reinterpret_cast<float*>(smem + L::kOffQ);
    float* sp = reinterpret_cast<float*>(smem + L::kOffP);
    float* s_corr = reinterpret_cast<float*>(smem + L::kOffStat);
    float* s_m = s_corr + kRows;
    float* s_l = s_m + kRows;
    long long* first = reinterpret_cast<long long*>(smem + L::kOffFirst);
    __shared__ uint32_t s_seen[kKeys];  // rows that see the key, one bit each
    __shared__ int s_bad[kKeys];        // tree key whose V row holds an infinity or NaN
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const q8::Work w = a.work;
    pdl_wait();
    pdl_trigger();
    q8::tile_offsets(w, a.kv_len, first);
    const long long total = first[w.B];
    long long g = w.cta_begin(total, blockIdx.x);
    const long long g_end = w.cta_begin(total, blockIdx.x + 1);
    const int rows_all = w.N * a.G;
    constexpr int ACC = kRows * D / kSimpleThreads;  // output rows per thread (one column)
    const int d = tid % D, r0 = tid / D * ACC;
    while (g < g_end) {
        const q8::Segment s = q8::segment_at(w, first, a.kv_len, g, g_end);
        g += s.t1 - s.t0;
        const int hk = s.unit / a.qblocks, row0 = s.unit % a.qblocks * kRows;
        const int nrows = min(kRows, rows_all - row0);
        for (int i = tid; i < kRows * D; i += kSimpleThreads) {
            const int r = row0 + i / D;
            float v = 0.f;
            if (i / D < nrows)
                v = load1(static_cast<const T*>(a.q) +
                          (((size_t)s.b * w.N + r / a.G) * a.Hq + hk * a.G + r % a.G) * D + i % D);
            sq[i] = v;
        }
        if (tid < kRows) { s_m[tid] = -INFINITY; s_l[tid] = 0.f; }
        if (tid < kKeys) s_bad[tid] = 0;
        float acc[ACC];
#pragma unroll
        for (int i = 0; i < ACC; ++i) acc[i] = 0.f;
        const int pt = w.prefix_tiles(s.L);
        for (int t = s.t0; t < s.t1; ++t) {
            __syncthreads();
            const bool tree = t >= pt;
            const int k0 = tree ? (t - pt) * kKeys : t * kKeys;
            const int nk = min(kKeys, (tree ? w.N : s.L) - k0);
            // keys of the tile, 8 elements a step; absent ones read zero
            for (int i = tid; i < kKeys * (D / 8); i += kSimpleThreads) {
                const int key = i / (D / 8), c = i % (D / 8) * 8;
                float kx[8], vx[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) kx[e] = vx[e] = 0.f;
                bool there = key < nk;
                if (there && tree) {
                    const size_t o = (((size_t)s.b * w.N + k0 + key) * a.Hkv + hk) * D + c;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        kx[e] = load1(static_cast<const T*>(a.k_tree) + o + e);
                        vx[e] = load1(static_cast<const T*>(a.v_tree) + o + e);
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
                    *reinterpret_cast<float4*>(sk + key * L::kStrideK + c + e) = make_float4(kx[e], kx[e + 1], kx[e + 2], kx[e + 3]);
                    *reinterpret_cast<float4*>(sv + key * D + c + e) = make_float4(vx[e], vx[e + 1], vx[e + 2], vx[e + 3]);
                }
                if (c == 0) {
                    uint32_t seen = there ? 0xffffu : 0u;
                    if (there && tree) {
                        seen = 0;
                        const int m = k0 + key;
                        for (int r = 0; r < nrows; ++r)
                            seen |= (uint32_t)((a.mask[(size_t)((row0 + r) / a.G) * a.W + (m >> 6)] >> (m & 63)) & 1) << r;
                    }
                    s_seen[key] = seen;
                }
            }
            __syncthreads();
            {   // scores: thread = (key, four rows)
                const int key = tid % kKeys, rq = tid / kKeys * 4;
                float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
                for (int c = 0; c < D; c += 4) {
                    const float4 kx = *reinterpret_cast<const float4*>(sk + key * L::kStrideK + c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 qx = *reinterpret_cast<const float4*>(sq + (rq + i) * D + c);
                        z[i] = fmaf(qx.x, kx.x, fmaf(qx.y, kx.y, fmaf(qx.z, kx.z, fmaf(qx.w, kx.w, z[i]))));
                    }
                }
                const uint32_t seen = s_seen[key];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sp[(rq + i) * kKeys + key] = (seen >> (rq + i)) & 1 ? z[i] * a.scale_log2 : -INFINITY;
            }
            __syncthreads();
            // running maximum and sum: two rows per warp
            for (int r = 2 * warp; r < 2 * warp + 2; ++r) {
                const float x0 = sp[r * kKeys + lane], x1 = sp[r * kKeys + lane + 32];
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
                sp[r * kKeys + lane] = p0;
                sp[r * kKeys + lane + 32] = p1;
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
            for (int i = 0; i < ACC; ++i) acc[i] *= s_corr[r0 + i];
#pragma unroll 4
            for (int k = 0; k < kKeys; k += 4) {
                const float v0 = sv[k * D + d], v1 = sv[(k + 1) * D + d], v2 = sv[(k + 2) * D + d], v3 = sv[(k + 3) * D + d];
#pragma unroll
                for (int i = 0; i < ACC; ++i) {
                    const float4 p = *reinterpret_cast<const float4*>(sp + (r0 + i) * kKeys + k);
                    acc[i] = fmaf(p.x, v0, fmaf(p.y, v1, fmaf(p.z, v2, fmaf(p.w, v3, acc[i]))));
                }
            }
        }
        if (s.whole()) {
#pragma unroll
            for (int i = 0; i < ACC; ++i) {
                const int r = row0 + r0 + i;
                if (r0 + i < nrows) {
                    const float l = s_l[r0 + i];
                    store1(static_cast<T*>(a.out) + (((size_t)s.b * w.N + r / a.G) * a.Hq + hk * a.G + r % a.G) * D + d,
                           l == 0.f ? 0.f : acc[i] / l);
                }
            }
        } else {
            const size_t base = (size_t)s.slot(blockIdx.x) * kRows;
#pragma unroll
            for (int i = 0; i < ACC; ++i) a.part_o[(base + r0 + i) * D + d] = acc[i];
            if (tid < kRows) a.part_ml[base + tid] = make_float2(s_m[tid], s_l[tid]);
        }
        __syncthreads();  // q, statistics free again
    }
}

// Joins the partial results.  Block (c, y): the unit that share c - 1 leaves
// unfinished, if that is the first share boundary inside it; rows y, y + gridDim.y, ...
template <typename T, int D>
__global__ void __launch_bounds__(D) attn_q8_merge_kernel(const AttnQ8Args a, int rows_block) {
    extern __shared__ long long first[];
    const q8::Work w = a.work;
    pdl_wait();
    pdl_trigger();
    q8::tile_offsets(w, a.kv_len, first);
    const long long total = first[w.B];
    const int c = blockIdx.x + 1;
    const long long g = w.cta_begin(total, c);
    if (g >= total || w.cta_begin(total, c + 1) == g) return;  // an empty share
    const q8::Segment s = q8::segment_at(w, first, a.kv_len, g, g);
    if (s.t0 == 0) return;                         // the boundary falls between units
    const long long u0 = g - s.t0, u1 = u0 + s.tiles;
    const int c0 = w.cta_of(total, u0);            // share that begins the unit
    if (c0 != w.cta_of(total, g - 1)) return;      // an earlier boundary is the first
    const int c1 = w.cta_of(total, u1 - 1);
    const int hk = s.unit / a.qblocks, row0 = s.unit % a.qblocks * rows_block;
    const int nrows = min(rows_block, w.N * a.G - row0);
    const int d = threadIdx.x;
    for (int i = blockIdx.y; i < nrows; i += gridDim.y) {
        float top = -INFINITY;
        for (int j = c0; j <= c1; ++j) {
            if (w.cta_begin(total, j) == w.cta_begin(total, j + 1)) continue;  // an empty share
            const float2 ml = a.part_ml[(size_t)(2 * j + (j == c0 ? 1 : 0)) * rows_block + i];
            top = fmaxf(top, ml.x);
        }
        const float ref = top == -INFINITY ? 0.f : top;
        float o = 0.f, l = 0.f;
        for (int j = c0; j <= c1; ++j) {
            if (w.cta_begin(total, j) == w.cta_begin(total, j + 1)) continue;
            const size_t at = (size_t)(2 * j + (j == c0 ? 1 : 0)) * rows_block + i;
            const float2 ml = a.part_ml[at];
            const float f = weight(ml.x - ref);
            l += ml.y * f;
            o += a.part_o[at * D + d] * f;
        }
        const int r = row0 + i;
        store1(static_cast<T*>(a.out) + (((size_t)s.b * w.N + r / a.G) * a.Hq + hk * a.G + r % a.G) * D + d,
               l == 0.f ? 0.f : o / l);
    }
}

struct Plan {
    int rows, keys, ctas;
};
Plan plan_q8(medusa_dtype dtype) {
    (void)dtype;
    return Plan{kRows, kKeys, 2 * sm_count()};
}

int check_attn_q8(int B, int N, int Hq, int Hkv, int D, int P, int n_pages, int M) {
    if (B < 1 || N < 1 || Hq < 1 || Hkv < 1 || n_pages < 1 || M < 1)
        return fail(MEDUSA_ERR_INVALID_ARG, "tree_attention_q8: sizes must be positive");
    if (int rc = q8::check_pool("tree_attention_q8", B, Hkv, D, P, n_pages, M)) return rc;
    if (N > 512 || Hq % Hkv || (long long)N * (Hq / Hkv) > 4096)
        return fail(MEDUSA_ERR_UNSUPPORTED, "tree_attention_q8: unsupported shape (N=%d Hq=%d Hkv=%d)", N, Hq, Hkv);
    return MEDUSA_OK;
}

size_t ws_bytes_q8(const Plan& p, int D) { return (size_t)2 * p.ctas * p.rows * (D + 2) * sizeof(float); }

template <typename T, int D>
cudaError_t launch_simple(AttnQ8Args& a, const Plan& p, cudaStream_t st) {
    auto kern = tree_attn_q8_simple_kernel<T, D>;
    const int smem = SimpleSmem<D>::bytes(a.work.B);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = launch(kern, dim3(p.ctas), dim3(kSimpleThreads), smem, st, a);
    if (e == cudaSuccess)
        e = launch(attn_q8_merge_kernel<T, D>, dim3(p.ctas - 1, 4), dim3(D), (a.work.B + 1) * 8, st, a, p.rows);
    return e;
}

}  // namespace
}  // namespace medusa

using namespace medusa;

extern "C" size_t medusa_tree_attention_q8_workspace(int B, int N, int Hq, int Hkv, int D, medusa_dtype dtype) {
    if (B < 1 || N < 1 || Hq < 1 || Hkv < 1 || (D != 64 && D != 128)) return 0;
    return ws_bytes_q8(plan_q8(dtype), D);
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
    if (!(scale > 0.f) || scale > 3.0e38f)
        return fail(MEDUSA_ERR_INVALID_ARG, "tree_attention_q8: scale must be positive and finite");
    const Plan p = plan_q8(dtype);
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
    a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv; a.P = P; a.M = M; a.n_pages = n_pages; a.W = (N + 63) / 64;
    a.qblocks = (N * a.G + p.rows - 1) / p.rows;
    a.work = q8::Work{B, N, Hkv * a.qblocks, p.keys, M * P, p.ctas};
    a.scale_log2 = scale * kLog2e;
    cudaStream_t st = as_stream(stream);
    cudaError_t e;
    if (dtype == MEDUSA_F32)
        e = D == 64 ? launch_simple<float, 64>(a, p, st) : launch_simple<float, 128>(a, p, st);
    else
        e = D == 64 ? launch_simple<uint16_t, 64>(a, p, st) : launch_simple<uint16_t, 128>(a, p, st);
    if (e != cudaSuccess)
        return fail(MEDUSA_ERR_CUDA, "tree_attention_q8: launch failed: %s", cudaGetErrorString(e));
    return MEDUSA_OK;
}
