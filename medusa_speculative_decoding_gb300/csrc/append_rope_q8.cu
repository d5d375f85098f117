// append_rope_q8.cu -- unrotated K rows and V rows into the 8-bit paged cache, the rotary
// positions applied on the way, and the same rows' queries rotated beside them: what stands
// between a layer's projections and its attention over the pages, in one launch ("Medusa
// Heads" glossary page, "Tree attention and acceptance": the accepted branch is kept).
//
// Row i goes to slot kv_len + i and turns by the angles of that position.  K is rotated in
// float32 and rounded once, to its code.  A rotated pair is at most sqrt(2) larger than the
// larger of its two values, so K's scale is the smallest 2^e with |x| <= 316 * 2^e over the
// rows as they are given (316 sqrt(2) = 446.9): it depends on the values and not on their
// positions nor on how sines are rounded, and nothing is clipped.  e4m3 is a floating type, so
// the half bit of range that this can leave unused costs no precision but in its subnormals.
//
// One CTA per (page that receives rows, up to four heads of K, of V or of the queries,
// sequence).  The page's sines and cosines are formed once into shared memory, while the first
// head's rows are on their way; a thread has pieces of sixteen values, both halves of eight
// pairs, so that no value crosses threads.  130 us for four prompts of 2048 to 4096 rows, 32 heads
// (503 MB, 3.9 TB/s; without the queries 88, of which kv_append_q8 takes 63): a CTA's steps follow one
// another, lengths, rows, turns, the largest value, codes; 5 us for a token of sixteen sequences.
// With 2 / 4 / 8 / 16 / 32 heads a CTA: 141 / 129 / 130 / 141 / 170 us.
#include <algorithm>

#include "append.cuh"
#include "common.cuh"
#include "q8.cuh"
#include "rope.cuh"

namespace medusa {
using namespace append;
namespace {

constexpr int kMostK = 316, kMostV = 448;

struct AppendRopeArgs {
    const void* rows[2];  // K, V rows [B][T][Hkv][D]
    const void* q;        // [B][T][Hq][D] or NULL
    void* q_out;
    uint8_t* pages[2];
    float* scale[2];
    const int32_t* page_table;
    const int32_t* kv_len;
    const int32_t* index;  // [B][R] or NULL
    const int32_t* last;   // [B] or NULL
    const int32_t* best_node;
    const uint4* hidden;
    uint4* h_next;
    int32_t* kv_len_out;
    int32_t* appended;
    rope::Freqs f;
    int B, T, R, Hq, Hkv, P, M, n_pages, h16, per_cta, groups, q_groups;
};

// Blocks along x: `groups` of K heads, as many of V heads, one for the sequence's
// bookkeeping, `q_groups` of query heads.
template <typename T, int D, int THREADS, int ITEMS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) append_rope_q8_kernel(const AppendRopeArgs a) {
    constexpr int C16 = D / 16;  // items of a row
    using Raw = typename Raw8<T>::type;
    extern __shared__ __align__(16) float2 s_cs[];  // [P][n]
    __shared__ float s_top[2][THREADS / 32];
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.z, tid = threadIdx.x;
    const int L = a.kv_len[b], last = a.last ? a.last[b] : a.R - 1;
    const int n = last + 1, P = a.P;
    const int x_block = blockIdx.x;
    const rope::Item at = rope::item_at(a.f, tid % C16, D);  // THREADS is a multiple of C16: the same for all items of a thread

    if (x_block > 2 * a.groups) {  // queries: rows blockIdx.y * P on, zero behind `last`
        const int t0 = blockIdx.y * P, rows = min(P, a.T - t0), real = min(rows, (last >= a.T ? a.T : max(last, -1) + 1) - t0);
        if (rows <= 0) return;
        const int h0 = (x_block - 2 * a.groups - 1) * a.per_cta, h1 = min(h0 + a.per_cta, a.Hq);
        const size_t o = (((size_t)b * a.T + t0) * a.Hq) * D;
        const T* in = static_cast<const T*>(a.q) + o;
        T* out = static_cast<T*>(a.q_out) + o;
        auto load = [&](int h, Raw (&x)[ITEMS][2]) {
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                const int r = (tid + k * THREADS) / C16;
                if (r >= real) continue;
                const T* from = in + ((size_t)r * a.Hq + h) * D;
                x[k][0].load_plain(from + at.first);
                x[k][1].load_plain(from + at.second);
            }
        };
        Raw x[ITEMS][2];
        load(h0, x);
        rope::fill_table(a.f, s_cs, 0, real, [&](int r) { return (int)((uint32_t)L + (uint32_t)(t0 + r)); });
        __syncthreads();
#pragma unroll 1
        for (int h = h0; h < h1; ++h) {
            Raw ahead[ITEMS][2];
            if (h + 1 < h1) load(h + 1, ahead);
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                const int r = (tid + k * THREADS) / C16;
                if (r >= rows) continue;
                float u[8], v[8];
                if (r < real) {
                    x[k][0].unpack(u);
                    x[k][1].unpack(v);
                    if (at.turns >= 0) rope::rotate(a.f, u, v, reinterpret_cast<const float4*>(s_cs + r * a.f.n) + at.turns);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) u[e] = v[e] = 0.f;
                }
                T* to = out + ((size_t)r * a.Hq + h) * D;
                rope::store8(to + at.first, u);
                rope::store8(to + at.second, v);
            }
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) { x[k][0] = ahead[k][0]; x[k][1] = ahead[k][1]; }
        }
        return;
    }

    // The whole sequence is checked by every CTA, so that either all of its rows
    // are written or none is.
    bool ok = last >= -1 && last < a.R && L >= 0 && L <= a.M * P && n <= a.M * P - L;
    const int w0 = ok ? L / P : 0;  // first page that receives a row
    const int windows = ok && n > 0 ? (L + n - 1) / P - w0 + 1 : 0;
    const int32_t* table = a.page_table + (size_t)b * a.M;

    const bool rows_cta = x_block < 2 * a.groups && (int)blockIdx.y < windows;
    const int kv = x_block >= a.groups;
    const int first = (w0 + (int)blockIdx.y) * P - L;  // new row that the page's slot 0 takes
    const size_t row_stride = (size_t)a.Hkv * D;
    const int e0 = kv ? tid % C16 * 8 : at.first, e1 = kv ? D / 2 + e0 : at.second;
    int row[ITEMS];  // the row that each of this thread's items comes from, -1: none
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int slot = (tid + k * THREADS) / C16, i = first + slot;
        row[k] = -1;
        if (rows_cta && slot < P && i >= 0 && i < n) {
            const int r = a.index ? a.index[(size_t)b * a.R + i] : i;
            if (r < a.T) row[k] = r;
        }
    }
    auto load_rows = [&](int h, Raw (&x)[ITEMS][2]) {
        const T* rows = static_cast<const T*>(a.rows[kv]) + ((size_t)b * a.T * a.Hkv + h) * D;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            x[k][0] = x[k][1] = {};
            if (row[k] >= 0) {
                x[k][0].load(rows + row[k] * row_stride + e0);
                x[k][1].load(rows + row[k] * row_stride + e1);
            }
        }
    };
    int h = (x_block - kv * a.groups) * a.per_cta;
    const int h_end = min(h + a.per_cta, a.Hkv);
    Raw x[ITEMS][2];
    if (rows_cta) load_rows(h, x);

    bool mine = true;
    for (int i = tid; i < windows; i += THREADS) {
        const int p = table[w0 + i];
        mine = mine && p >= 0 && p < a.n_pages;
    }
    if (a.index && ok)
        for (int i = tid; i < n; i += THREADS) {
            const int r = a.index[(size_t)b * a.R + i];
            mine = mine && r >= 0 && r < a.T;
        }
    if (a.best_node && tid == 0) mine = mine && a.best_node[b] >= 0 && a.best_node[b] < a.T;
    ok = __syncthreads_and(ok && mine);

    if (x_block == 2 * a.groups) {  // the sequence's bookkeeping
        if (blockIdx.y) return;
        if (tid == 0) {
            a.kv_len_out[b] = ok ? L + n : L;
            if (a.appended) a.appended[b] = ok ? n : -2;
        }
        if (a.hidden) {  // zero where the sequence is rejected: never what memory held before
            const uint4* src = a.hidden + ((size_t)b * a.T + (ok ? a.best_node[b] : 0)) * a.h16;
            for (int i = tid; i < a.h16; i += THREADS)
                a.h_next[(size_t)b * a.h16 + i] = ok ? src[i] : make_uint4(0, 0, 0, 0);
        }
        return;
    }
    if (!ok || !rows_cta) return;
    if (!kv) {
        const int from = max(0, -first);
        rope::fill_table(a.f, s_cs, from, min(P, n - first) - from, [&](int slot) { return L + first + slot; });
    }

    const size_t page = table[w0 + blockIdx.y];
    const bool had = first < 0;  // the page holds earlier rows
#pragma unroll 1
    for (; h < h_end; ++h) {
        const size_t unit = page * a.Hkv + h;
        uint8_t* codes = a.pages[kv] + unit * P * D;
        const float s0 = had ? a.scale[kv][unit] : 0.f;
        Raw ahead[ITEMS][2];
        if (h + 1 < h_end) load_rows(h + 1, ahead);
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) top = fmaxf(top, fmaxf(x[k][0].top(), x[k][1].top()));
        if (top == INFINITY) {  // the scale is set by finite values
            top = 0.f;
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) top = fmaxf(top, fmaxf(finite_top(x[k][0]), finite_top(x[k][1])));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if ((tid & 31) == 0) s_top[h & 1][tid >> 5] = top;
        __syncthreads();  // every thread has read the page's scale, too, and the table is filled
#pragma unroll
        for (int i = 0; i < THREADS / 32; ++i) top = fmaxf(top, s_top[h & 1][i]);

        const bool readable = !had || q8::scale_ok(s0);  // an unreadable page stays one
        const bool keep = had && (!readable || (kv ? fits<kMostV>(top, s0) : fits<kMostK>(top, s0)));
        const float s1 = keep ? s0 : kv ? page_scale<kMostV>(top) : page_scale<kMostK>(top);
        if (tid == 0 && !keep) a.scale[kv][unit] = s1;
        if (readable) {
            // 1 / s1 is exact for the powers of two written here; a caller's own scale is divided by
            const bool pow2 = (__float_as_uint(s1) & 0x7fffffu) == 0;
            const float inv = 1.f / s1;
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                const int slot = (tid + k * THREADS) / C16, i = first + slot;
                if (slot >= P || i >= n) continue;
                uint2* dst[2] = {reinterpret_cast<uint2*>(codes + slot * D + e0), reinterpret_cast<uint2*>(codes + slot * D + e1)};
                float y[2][8];
                if (i < 0) {
                    if (keep) continue;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint2 w = *dst[j];
                        const uint16_t old[4] = {(uint16_t)w.x, (uint16_t)(w.x >> 16), (uint16_t)w.y, (uint16_t)(w.y >> 16)};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = q8::e4m3x2_to_float2(old[e]);
                            y[j][2 * e] = multiply_to_odd(f.x, s0);
                            y[j][2 * e + 1] = multiply_to_odd(f.y, s0);
                        }
                    }
                } else {
                    x[k][0].unpack(y[0]);
                    x[k][1].unpack(y[1]);
                    if (!kv && at.turns >= 0) rope::rotate(a.f, y[0], y[1], reinterpret_cast<const float4*>(s_cs + slot * a.f.n) + at.turns);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint16_t q[4];
                    if (pow2) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            q8::mul2(y[j][2 * e], y[j][2 * e + 1], y[j][2 * e], y[j][2 * e + 1], inv);
                            q[e] = q8::float2_to_e4m3x2(y[j][2 * e], y[j][2 * e + 1]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            q[e] = q8::float2_to_e4m3x2(divide_to_odd(y[j][2 * e], s1), divide_to_odd(y[j][2 * e + 1], s1));
                    }
                    *dst[j] = make_uint2((uint32_t)q[0] | (uint32_t)q[1] << 16, (uint32_t)q[2] | (uint32_t)q[3] << 16);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) { x[k][0] = ahead[k][0]; x[k][1] = ahead[k][1]; }
    }
}

template <typename T, int D, int THREADS, int ITEMS>
cudaError_t launch_append(const AppendRopeArgs& a, int windows, cudaStream_t st) {
    auto kern = append_rope_q8_kernel<T, D, THREADS, ITEMS>;
    // (the attribute is the kernel's, not the call's: always what the largest page takes)
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * (D / 2) * (int)sizeof(float2));
    if (e != cudaSuccess) return e;
    const dim3 grid(2 * a.groups + 1 + a.q_groups, windows, a.B);
    return launch(kern, grid, dim3(THREADS), (size_t)a.P * a.f.n * sizeof(float2), st, a);
}

// 64 bytes of rows per thread, twice over, as in append_q8_kernel.
template <typename T, int D>
cudaError_t pick_append(const AppendRopeArgs& a, int windows, cudaStream_t st) {
    const int items = a.P * D / 16;
    if (items <= 256) return launch_append<T, D, 256, 1>(a, windows, st);
    if constexpr (sizeof(T) == 2) {
        if (items <= 512) return launch_append<T, D, 256, 2>(a, windows, st);
        return launch_append<T, D, 512, 2>(a, windows, st);
    } else {
        if (items <= 512) return launch_append<T, D, 512, 1>(a, windows, st);
        return launch_append<T, D, 1024, 1>(a, windows, st);
    }
}

}  // namespace
}  // namespace medusa

using namespace medusa;

extern "C" int medusa_kv_append_rope_q8(const void* k_rows, const void* v_rows, medusa_dtype dtype, void* k_pages,
                                        void* v_pages, float* k_scale, float* v_scale, const int32_t* page_table,
                                        const int32_t* kv_len, const int32_t* rows, const int32_t* last,
                                        const float* inv_freq, int n_freq, int interleaved, const void* q, void* q_out,
                                        int B, int T, int R, int Hq, int Hkv, int D, int P, int n_pages, int M,
                                        const int32_t* best_node, const void* hidden_rows, void* h_next, int H,
                                        int32_t* kv_len_out, int32_t* appended, void* stream) {
    const char* who = "kv_append_rope_q8";
    if (B < 1 || T < 1 || R < 1 || Hkv < 1 || n_pages < 1 || M < 1 || Hq < 0)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: sizes must be positive", who);
    if (int rc = q8::check_pool(who, B, Hkv, D, P, n_pages, M)) return rc;
    if (Hq > 1024) return fail(MEDUSA_ERR_UNSUPPORTED, "%s: %d query heads above 1024", who, Hq);
    if (dtype != MEDUSA_F32 && dtype != MEDUSA_BF16)
        return fail(MEDUSA_ERR_UNSUPPORTED, "%s: unknown dtype %d", who, (int)dtype);
    if (int rc = rope::check_freqs(who, inv_freq, n_freq, D)) return rc;
    if (!k_rows || !v_rows || !k_pages || !v_pages || !k_scale || !v_scale || !page_table || !kv_len || !kv_len_out)
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: null pointer", who);
    if (!rows && R > T) return fail(MEDUSA_ERR_INVALID_ARG, "%s: R %d above T %d without row indices", who, R, T);
    if ((q != nullptr) != (Hq > 0) || (q != nullptr) != (q_out != nullptr))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: q, q_out and Hq go together", who);
    if (q && rows) return fail(MEDUSA_ERR_INVALID_ARG, "%s: queries stand at the positions of rows in order, not of picked rows", who);
    if (q && R < T) return fail(MEDUSA_ERR_INVALID_ARG, "%s: with queries R must be T", who);
    const bool hid = hidden_rows != nullptr;
    if (hid != (h_next != nullptr) || hid != (best_node != nullptr))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: best_node, hidden_rows and h_next go together", who);
    const int elem = dtype == MEDUSA_F32 ? 4 : 2;
    if (hid && (H < 1 || ((long long)H * elem) % 16))
        return fail(MEDUSA_ERR_UNSUPPORTED, "%s: hidden rows must be multiples of 16 bytes", who);
    if (!aligned16(k_rows) || !aligned16(v_rows) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(q) ||
        !aligned16(q_out) || (hid && (!aligned16(hidden_rows) || !aligned16(h_next))))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: rows, pages and hidden states must be 16-byte aligned", who);
    if (q_out && (q_out == k_rows || q_out == v_rows || (hid && q_out == hidden_rows)))
        return fail(MEDUSA_ERR_INVALID_ARG, "%s: q_out may be q, but no other array that is read", who);
    for (const int32_t* read : {kv_len, last, best_node, rows, page_table})
        if (read && (read == kv_len_out || read == appended))
            return fail(MEDUSA_ERR_INVALID_ARG, "%s: kv_len_out and appended must not be what is read", who);
    if (appended == kv_len_out) return fail(MEDUSA_ERR_INVALID_ARG, "%s: kv_len_out and appended must differ", who);
    const int windows = (int)(((long long)R + P - 2) / P + 1);  // pages that R rows can touch
    if (windows > 65535) return fail(MEDUSA_ERR_UNSUPPORTED, "%s: %d rows span too many pages", who, R);
    AppendRopeArgs a{};
    a.rows[0] = k_rows; a.rows[1] = v_rows;
    a.q = q; a.q_out = q_out;
    a.pages[0] = (uint8_t*)k_pages; a.pages[1] = (uint8_t*)v_pages;
    a.scale[0] = k_scale; a.scale[1] = v_scale;
    a.page_table = page_table; a.kv_len = kv_len; a.index = rows; a.last = last;
    a.best_node = best_node;
    a.hidden = (const uint4*)hidden_rows; a.h_next = (uint4*)h_next;
    a.kv_len_out = kv_len_out; a.appended = appended;
    a.f = rope::Freqs{inv_freq, n_freq, interleaved != 0};
    a.B = B; a.T = T; a.R = R; a.Hq = Hq; a.Hkv = Hkv; a.P = P; a.M = M; a.n_pages = n_pages;
    a.h16 = hid ? (int)((long long)H * elem / 16) : 0;
    // A CTA takes up to four heads one after the other, the next one's rows on their way, as
    // long as that leaves four CTAs for every SM.
    a.per_cta = (int)std::min(4ll, std::max(1ll, (2ll * Hkv + Hq) * windows * B / (4 * sm_count())));
    a.groups = (Hkv + a.per_cta - 1) / a.per_cta;
    a.q_groups = (Hq + a.per_cta - 1) / a.per_cta;
    cudaStream_t st = as_stream(stream);
    cudaError_t e;
    if (dtype == MEDUSA_F32)
        e = D == 64 ? pick_append<float, 64>(a, windows, st) : pick_append<float, 128>(a, windows, st);
    else
        e = D == 64 ? pick_append<uint16_t, 64>(a, windows, st) : pick_append<uint16_t, 128>(a, windows, st);
    if (e != cudaSuccess) return fail(MEDUSA_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    return MEDUSA_OK;
}
