// append_q8.cu -- new K and V rows into the 8-bit paged cache.
//
// Rows go to the slots behind kv_len: a prompt's rows in order, a decoded token's,
// or the rows of a tree's accepted branch picked by index ("Medusa Heads"
// glossary page, "Tree attention and acceptance": the longest accepted branch is
// kept) -- the tree's other rows never reach the cache, so nothing is moved or
// undone later.
//
// A page's scale for one head is the smallest power of two 2^e with max|x| <=
// 448 * 2^e over the rows it holds.  e4m3 is a floating type: a power-of-two
// scale costs no precision, and when a later row needs a larger one the earlier
// codes move to the new grid exactly, except those that fall into e4m3's
// subnormal range, which round to its step.
//
// append_q8_kernel: one CTA per (page that receives rows, up to eight (head, K or
// V) of it, sequence).  The rows of one head's page are read once, 16 bytes a load,
// and held as loaded through the maximum and the conversion; the codes leave as one
// contiguous span.  The next head's rows are on their way meanwhile: with a CTA per
// head, 79 us for four prompts of 4096 rows x 32 heads x 128 bf16, since each waited
// for the lengths, the rows and a reduction in turn; now 59 us, 5.1 TB/s of rows read
// and codes written.
#include <algorithm>

#include "append.cuh"
#include "common.cuh"
#include "q8.cuh"

namespace medusa {
using namespace append;
namespace {

struct AppendArgs {
    const void* rows[2];  // K, V rows [B][T][Hkv][D]
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
    int B, T, R, Hkv, P, M, n_pages, h16, per_cta;
};

// THREADS * CHUNKS pieces of eight elements make a page of one head.
template <typename T, int D, int THREADS, int CHUNKS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) append_q8_kernel(const AppendArgs a) {
    constexpr int C8 = D / 8;  // 8-element chunks per row
    __shared__ float s_top[2][THREADS / 32];
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.z, tid = threadIdx.x;
    const int L = a.kv_len[b], last = a.last ? a.last[b] : a.R - 1;
    const int n = last + 1, P = a.P;
    // The whole sequence is checked by every CTA, so that either all of its rows
    // are written or none is.
    bool ok = last >= -1 && last < a.R && L >= 0 && L <= a.M * P && n <= a.M * P - L;
    const int w0 = ok ? L / P : 0;  // first page that receives a row
    const int windows = ok && n > 0 ? (L + n - 1) / P - w0 + 1 : 0;
    const int32_t* table = a.page_table + (size_t)b * a.M;

    // The first rows, asked for before the check's own loads have come back.
    const bool rows_cta = blockIdx.x + 1 < gridDim.x && (int)blockIdx.y < windows;
    const int first = (w0 + (int)blockIdx.y) * P - L;  // new row that the page's slot 0 takes
    const int chunks = P * C8;
    const size_t row_stride = (size_t)a.Hkv * D;
    using Raw = typename Raw8<T>::type;
    int row[CHUNKS];  // the row that each of this thread's chunks comes from, -1: none
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k) {
        const int c = tid + k * THREADS;
        const int i = first + c / C8;
        row[k] = -1;
        if (rows_cta && c < chunks && i >= 0 && i < n) {
            const int r = a.index ? a.index[(size_t)b * a.R + i] : i;
            if (r < a.T) row[k] = r;
        }
    }
    auto load_rows = [&](int id, Raw (&x)[CHUNKS]) {  // id = (head, K or V)
        const T* rows = static_cast<const T*>(a.rows[id & 1]) + ((size_t)b * a.T * a.Hkv + (id >> 1)) * D + tid % C8 * 8;
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            x[k] = {};
            if (row[k] >= 0) x[k].load(rows + row[k] * row_stride);
        }
    };
    int id = blockIdx.x * a.per_cta;
    const int id_end = min(id + a.per_cta, 2 * a.Hkv);
    Raw x[CHUNKS];
    if (rows_cta) load_rows(id, x);

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

    if (blockIdx.x + 1 == gridDim.x) {  // the sequence's bookkeeping
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

    const size_t page = table[w0 + blockIdx.y];
#pragma unroll 1
    for (; id < id_end; ++id) {
        const int h = id >> 1, kv = id & 1;
        const size_t unit = page * a.Hkv + h;
        uint8_t* codes = a.pages[kv] + unit * P * D;
        const bool had = first < 0;  // the page holds earlier rows
        const float s0 = had ? a.scale[kv][unit] : 0.f;
        Raw ahead[CHUNKS];
        if (id + 1 < id_end) load_rows(id + 1, ahead);
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) top = fmaxf(top, x[k].top());
        if (top == INFINITY) {  // the scale is set by finite values
            top = 0.f;
#pragma unroll
            for (int k = 0; k < CHUNKS; ++k) {
                float y[8];
                x[k].unpack(y);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (fabsf(y[e]) < INFINITY) top = fmaxf(top, fabsf(y[e]));
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if ((tid & 31) == 0) s_top[id & 1][tid >> 5] = top;
        __syncthreads();  // every thread has read the page's scale, too
#pragma unroll
        for (int i = 0; i < THREADS / 32; ++i) top = fmaxf(top, s_top[id & 1][i]);

        const bool readable = !had || q8::scale_ok(s0);  // an unreadable page stays one
        const bool keep = had && (!readable || fits<448>(top, s0));
        const float s1 = keep ? s0 : page_scale<448>(top);
        if (tid == 0 && !keep) a.scale[kv][unit] = s1;
        if (readable) {
            // 1 / s1 is exact for the powers of two written here; a caller's own scale is divided by
            const bool pow2 = (__float_as_uint(s1) & 0x7fffffu) == 0;
            const float inv = 1.f / s1;
#pragma unroll
            for (int k = 0; k < CHUNKS; ++k) {
                const int c = tid + k * THREADS;
                const int i = first + c / C8;
                if (c >= chunks || i >= n) continue;
                uint2* dst = reinterpret_cast<uint2*>(codes + (size_t)c * 8);
                float y[8];
                if (i < 0) {
                    if (keep) continue;
                    const uint2 w = *dst;
                    const uint16_t old[4] = {(uint16_t)w.x, (uint16_t)(w.x >> 16), (uint16_t)w.y, (uint16_t)(w.y >> 16)};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = q8::e4m3x2_to_float2(old[e]);
                        y[2 * e] = multiply_to_odd(f.x, s0);
                        y[2 * e + 1] = multiply_to_odd(f.y, s0);
                    }
                } else {
                    x[k].unpack(y);
                }
                uint16_t q[4];
                if (pow2) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        q8::mul2(y[2 * e], y[2 * e + 1], y[2 * e], y[2 * e + 1], inv);
                        q[e] = q8::float2_to_e4m3x2(y[2 * e], y[2 * e + 1]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) q[e] = q8::float2_to_e4m3x2(divide_to_odd(y[2 * e], s1), divide_to_odd(y[2 * e + 1], s1));
                }
                *dst = make_uint2((uint32_t)q[0] | (uint32_t)q[1] << 16, (uint32_t)q[2] | (uint32_t)q[3] << 16);
            }
        }
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) x[k] = ahead[k];
    }
}

template <typename T, int D, int THREADS, int CHUNKS>
cudaError_t launch_append(const AppendArgs& a, int windows, cudaStream_t st) {
    const dim3 grid((2 * a.Hkv + a.per_cta - 1) / a.per_cta + 1, windows, a.B);
    return launch(append_q8_kernel<T, D, THREADS, CHUNKS>, grid, dim3(THREADS), 0, st, a);
}

// 64 bytes of rows per thread, twice over, leave 64 registers for 1024 threads on an SM.
template <typename T, int D>
cudaError_t pick_append(const AppendArgs& a, int windows, cudaStream_t st) {
    const int pieces = a.P * D / 8;
    if (pieces <= 256) return launch_append<T, D, 256, 1>(a, windows, st);
    if (pieces <= 512) return launch_append<T, D, 256, 2>(a, windows, st);
    if constexpr (sizeof(T) == 2) {
        if (pieces <= 1024) return launch_append<T, D, 256, 4>(a, windows, st);
        return launch_append<T, D, 512, 4>(a, windows, st);
    } else {
        if (pieces <= 1024) return launch_append<T, D, 512, 2>(a, windows, st);
        return launch_append<T, D, 1024, 2>(a, windows, st);
    }
}

}  // namespace
}  // namespace medusa

using namespace medusa;

extern "C" int medusa_kv_append_q8(const void* k_rows, const void* v_rows, medusa_dtype dtype, void* k_pages,
                                   void* v_pages, float* k_scale, float* v_scale, const int32_t* page_table,
                                   const int32_t* kv_len, const int32_t* rows, const int32_t* last, int B, int T,
                                   int R, int Hkv, int D, int P, int n_pages, int M, const int32_t* best_node,
                                   const void* hidden_rows, void* h_next, int H, int32_t* kv_len_out,
                                   int32_t* appended, void* stream) {
    if (B < 1 || T < 1 || R < 1 || Hkv < 1 || n_pages < 1 || M < 1)
        return fail(MEDUSA_ERR_INVALID_ARG, "kv_append_q8: sizes must be positive");
    if (int rc = q8::check_pool("kv_append_q8", B, Hkv, D, P, n_pages, M)) return rc;
    if (dtype != MEDUSA_F32 && dtype != MEDUSA_BF16)
        return fail(MEDUSA_ERR_UNSUPPORTED, "kv_append_q8: unknown dtype %d", (int)dtype);
    if (!k_rows || !v_rows || !k_pages || !v_pages || !k_scale || !v_scale || !page_table || !kv_len || !kv_len_out)
        return fail(MEDUSA_ERR_INVALID_ARG, "kv_append_q8: null pointer");
    if (!rows && R > T) return fail(MEDUSA_ERR_INVALID_ARG, "kv_append_q8: R %d above T %d without row indices", R, T);
    const bool hid = hidden_rows != nullptr;
    if (hid != (h_next != nullptr) || hid != (best_node != nullptr))
        return fail(MEDUSA_ERR_INVALID_ARG, "kv_append_q8: best_node, hidden_rows and h_next go together");
    const int elem = dtype == MEDUSA_F32 ? 4 : 2;
    if (hid && (H < 1 || ((long long)H * elem) % 16))
        return fail(MEDUSA_ERR_UNSUPPORTED, "kv_append_q8: hidden rows must be multiples of 16 bytes");
    if (!aligned16(k_rows) || !aligned16(v_rows) || !aligned16(k_pages) || !aligned16(v_pages) ||
        (hid && (!aligned16(hidden_rows) || !aligned16(h_next))))
        return fail(MEDUSA_ERR_INVALID_ARG, "kv_append_q8: rows, pages and hidden states must be 16-byte aligned");
    for (const int32_t* read : {kv_len, last, best_node, rows, page_table})
        if (read && (read == kv_len_out || read == appended))
            return fail(MEDUSA_ERR_INVALID_ARG, "kv_append_q8: kv_len_out and appended must not be what is read");
    if (appended == kv_len_out)
        return fail(MEDUSA_ERR_INVALID_ARG, "kv_append_q8: kv_len_out and appended must differ");
    const int windows = (int)(((long long)R + P - 2) / P + 1);  // pages that R rows can touch
    if (windows > 65535) return fail(MEDUSA_ERR_UNSUPPORTED, "kv_append_q8: %d rows span too many pages", R);
    AppendArgs a{};
    a.rows[0] = k_rows; a.rows[1] = v_rows;
    a.pages[0] = (uint8_t*)k_pages; a.pages[1] = (uint8_t*)v_pages;
    a.scale[0] = k_scale; a.scale[1] = v_scale;
    a.page_table = page_table; a.kv_len = kv_len; a.index = rows; a.last = last;
    a.best_node = best_node;
    a.hidden = (const uint4*)hidden_rows; a.h_next = (uint4*)h_next;
    a.kv_len_out = kv_len_out; a.appended = appended;
    a.B = B; a.T = T; a.R = R; a.Hkv = Hkv; a.P = P; a.M = M; a.n_pages = n_pages;
    // A CTA takes up to eight (head, K or V) of its page one after the other, the next
    // one's rows on their way, as long as that leaves four CTAs for every SM.
    a.per_cta = (int)std::min(8ll, std::max(1ll, 2ll * Hkv * windows * B / (4 * sm_count())));
    a.h16 = hid ? (int)((long long)H * elem / 16) : 0;
    cudaStream_t st = as_stream(stream);
    cudaError_t e;
    if (dtype == MEDUSA_F32)
        e = D == 64 ? pick_append<float, 64>(a, windows, st) : pick_append<float, 128>(a, windows, st);
    else
        e = D == 64 ? pick_append<uint16_t, 64>(a, windows, st) : pick_append<uint16_t, 128>(a, windows, st);
    if (e != cudaSuccess) return fail(MEDUSA_ERR_CUDA, "kv_append_q8: launch failed: %s", cudaGetErrorString(e));
    return MEDUSA_OK;
}
