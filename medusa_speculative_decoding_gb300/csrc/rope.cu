// rope.cu -- rotary positions of new queries and keys ("Medusa Heads" glossary page, "Tree
// attention and acceptance": a tree's candidates are appended at once; those of one depth
// stand at the same position).
//
// Row i of sequence b turns by the angles of position kv_len[b] + depth[i] (kv_len[b] + i
// without depths).  Bound by HBM where the rows are many: every value is read and written
// once, 16 bytes a load.  A block takes some rows of one sequence and all or some of their
// heads, so that a row's sines and cosines are formed once for 16 heads or more, while the first
// values are on their way.  44 us for sixteen trees of 341 nodes, 48 heads of 128, float32 (6.1
// TB/s); 47 us for 16384 rows, 32 heads of 128, bf16 (5.7 TB/s; a copy 41); 3 us for one tree.
#include <algorithm>

#include "append.cuh"
#include "common.cuh"
#include "rope.cuh"

namespace medusa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 16;  // rows of a block

// items of a thread with their loads in flight: 128 bytes
template <typename T> constexpr int kBatch = 8 / sizeof(T);

struct RopeArgs {
    const void* in[2];  // q, k
    void* out[2];
    const int32_t *kv_len, *depth;
    rope::Freqs f;
    int T, D, heads[2], rows, per_block;  // rows, heads of a block
    uint32_t items_magic, heads_magic;    // 2^32 / items of a head, / heads of a block, rounded up
};

// i / d with d's magic, for i * d < 2^32
__device__ __forceinline__ int divide(int i, uint32_t magic) { return magic ? (int)__umulhi((uint32_t)i, magic) : i; }

template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 2 : 3) rope_rows_kernel(const RopeArgs a) {
    extern __shared__ __align__(16) float2 s_cs[];  // [rows][n]
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.z, t0 = blockIdx.x * a.rows, rows = min(a.rows, a.T - t0);
    const int base = a.kv_len[b];
    const int all = a.heads[0] + a.heads[1], items = a.D / 16;
    const int h0 = blockIdx.y * a.per_block, nh = min(a.per_block, all - h0);
    const int count = rows * a.per_block * items;  // (heads behind the last are left out below)
    using Raw = typename append::Raw8<T>::type;
    Raw x[kBatch<T>], y[kBatch<T>];
    T* out[kBatch<T>];
    int row[kBatch<T>];
    rope::Item at[kBatch<T>];
    auto load = [&](int first) {
#pragma unroll
        for (int k = 0; k < kBatch<T>; ++k) {
            const int i = first + k * kThreads;
            row[k] = -1;
            const int j = divide(i, a.items_magic), r = divide(j, a.heads_magic), h = h0 + j - r * a.per_block;
            if (i >= count || h >= h0 + nh) continue;
            row[k] = r;
            at[k] = rope::item_at(a.f, i - j * items, a.D);
            const bool key = h >= a.heads[0];
            const size_t o = (((size_t)b * a.T + t0 + r) * (key ? a.heads[1] : a.heads[0]) + (key ? h - a.heads[0] : h)) * a.D;
            const T* in = static_cast<const T*>(key ? a.in[1] : a.in[0]) + o;
            out[k] = static_cast<T*>(key ? a.out[1] : a.out[0]) + o;
            x[k].load_plain(in + at[k].first);
            y[k].load_plain(in + at[k].second);
        }
    };
    load(threadIdx.x);  // on their way while the table is filled
    rope::fill_table(a.f, s_cs, 0, rows, [&](int r) { return (int)((uint32_t)base + (uint32_t)(a.depth ? a.depth[t0 + r] : t0 + r)); });
    __syncthreads();
    for (int first = threadIdx.x; first < count; first += kBatch<T> * kThreads) {
        if (first != (int)threadIdx.x) load(first);
#pragma unroll
        for (int k = 0; k < kBatch<T>; ++k) {
            if (row[k] < 0) continue;
            float u[8], v[8];
            x[k].unpack(u);
            y[k].unpack(v);
            if (at[k].turns >= 0) rope::rotate(a.f, u, v, reinterpret_cast<const float4*>(s_cs + row[k] * a.f.n) + at[k].turns);
            rope::store8(out[k] + at[k].first, u);
            rope::store8(out[k] + at[k].second, v);
        }
    }
}

}  // namespace
}  // namespace medusa

using namespace medusa;

extern "C" int medusa_rope_rows(const void* q, const void* k, medusa_dtype dtype, const int32_t* kv_len,
                                const int32_t* depth, const float* inv_freq, int B, int T, int Hq, int Hkv, int D,
                                int n_freq, int interleaved, void* q_out, void* k_out, void* stream) {
    if (B < 1 || T < 1 || Hq < 1 || Hkv < 0 || D < 1)
        return fail(MEDUSA_ERR_INVALID_ARG, "rope_rows: sizes must be positive");
    if (dtype != MEDUSA_F32 && dtype != MEDUSA_BF16)
        return fail(MEDUSA_ERR_UNSUPPORTED, "rope_rows: unknown dtype %d", (int)dtype);
    if (D % 16 || D > 512 || B > 65535 || T > 1 << 24 || Hq > 1024 || Hkv > 1024)
        return fail(MEDUSA_ERR_UNSUPPORTED, "rope_rows: head dim %d must be a multiple of 16 up to 512, at most 65535 sequences, 2^24 rows and 1024 heads", D);
    if (int rc = rope::check_freqs("rope_rows", inv_freq, n_freq, D)) return rc;
    if (!q || !q_out || !kv_len || (Hkv > 0) != (k != nullptr) || (k != nullptr) != (k_out != nullptr))
        return fail(MEDUSA_ERR_INVALID_ARG, "rope_rows: null pointer");
    if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(k_out))
        return fail(MEDUSA_ERR_INVALID_ARG, "rope_rows: rows must be 16-byte aligned");
    if (q_out == k_out || (const void*)q_out == k || (const void*)k_out == q)
        return fail(MEDUSA_ERR_INVALID_ARG, "rope_rows: q_out and k_out must differ, and each may only be its own input");
    RopeArgs a{};
    a.in[0] = q; a.in[1] = k;
    a.out[0] = q_out; a.out[1] = k_out;
    a.kv_len = kv_len; a.depth = depth;
    a.f = rope::Freqs{inv_freq, n_freq, interleaved != 0};
    a.T = T; a.D = D; a.heads[0] = Hq; a.heads[1] = Hkv;
    // Blocks of about sixteen items a thread; where that leaves SMs without a block, of fewer
    // rows, then of fewer heads.
    const int all = Hq + Hkv, items = D / 16, sms = sm_count();
    a.rows = std::clamp(16 * kThreads / (all * items), 1, kMaxRows);
    while (a.rows > 1 && (long long)B * ((T + a.rows - 1) / a.rows) < 2 * sms) a.rows /= 2;
    a.per_block = all;
    while (a.per_block > 16 && (long long)B * ((T + a.rows - 1) / a.rows) * ((all + a.per_block - 1) / a.per_block) < sms)
        a.per_block = (a.per_block + 1) / 2;
    auto magic = [](int d) { return d == 1 ? 0u : (uint32_t)(((1ull << 32) + d - 1) / d); };
    a.items_magic = magic(items);
    a.heads_magic = magic(a.per_block);
    const dim3 grid((T + a.rows - 1) / a.rows, (all + a.per_block - 1) / a.per_block, B);
    const size_t smem = (size_t)a.rows * n_freq * sizeof(float2);  // at most 16 * 256 * 8 bytes
    cudaStream_t st = as_stream(stream);
    const cudaError_t e = dtype == MEDUSA_F32 ? launch(rope_rows_kernel<float>, grid, dim3(kThreads), smem, st, a)
                                              : launch(rope_rows_kernel<uint16_t>, grid, dim3(kThreads), smem, st, a);
    if (e != cudaSuccess) return fail(MEDUSA_ERR_CUDA, "rope_rows: launch failed: %s", cudaGetErrorString(e));
    return MEDUSA_OK;
}
