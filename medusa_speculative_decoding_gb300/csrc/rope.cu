// rope.cu -- rotary positions of new queries and keys ("Medusa Heads" glossary page, "Tree
// attention and acceptance": a tree's candidates are appended at once; those of one depth
// stand at the same position).
//
// Row i of sequence b turns by the angles of position kv_len[b] + depth[i] (kv_len[b] + i
// without depths).  Bound by HBM where the rows are many: every value is read and written
// once, 16 bytes a load.  A block takes some rows of one sequence and all or some of their
// heads, so that a row's sines and cosines are formed once for 16 heads or more.
#include <algorithm>

#include "append.cuh"
#include "common.cuh"
#include "rope.cuh"

namespace medusa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 16;  // rows of a block
constexpr int kBatch = 4;     // items of a thread with their loads in flight

struct RopeArgs {
    const void* in[2];  // q, k
    void* out[2];
    const int32_t *kv_len, *depth;
    rope::Freqs f;
    int T, D, heads[2], rows, per_block;  // rows, heads of a block
};

template <typename T>
__global__ void __launch_bounds__(kThreads) rope_rows_kernel(const RopeArgs a) {
    extern __shared__ __align__(16) float2 s_cs[];  // [rows][n]
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.z, t0 = blockIdx.x * a.rows, rows = min(a.rows, a.T - t0);
    const int base = a.kv_len[b];
    for (int i = threadIdx.x; i < a.f.n; i += kThreads) {
        const uint64_t turn = rope::turn(a.f.inv_freq[i]);
        for (int r = 0; r < rows; ++r)
            s_cs[r * a.f.n + i] = rope::cos_sin(turn, (int)((uint32_t)base + (uint32_t)(a.depth ? a.depth[t0 + r] : t0 + r)));
    }
    __syncthreads();
    const int all = a.heads[0] + a.heads[1], items = a.D / 16;
    const int h0 = blockIdx.y * a.per_block, nh = min(a.per_block, all - h0);
    const int count = rows * nh * items;
    using Raw = typename append::Raw8<T>::type;
    for (int first = threadIdx.x; first < count; first += kBatch * kThreads) {
        Raw x[kBatch], y[kBatch];
        T* out[kBatch];
        int row[kBatch];
        rope::Item at[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int i = first + k * kThreads;
            row[k] = -1;
            if (i >= count) continue;
            const int h = h0 + i / items % nh;
            row[k] = i / items / nh;
            at[k] = rope::item_at(a.f, i % items);
            const int which = h >= a.heads[0];
            const size_t o = (((size_t)b * a.T + t0 + row[k]) * a.heads[which] + (which ? h - a.heads[0] : h)) * a.D;
            const T* in = static_cast<const T*>(a.in[which]) + o;
            out[k] = static_cast<T*>(a.out[which]) + o;
            x[k].load_plain(in + at[k].first);
            y[k].load_plain(in + at[k].second);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (row[k] < 0) continue;
            float u[8], v[8];
            x[k].unpack(u);
            y[k].unpack(v);
            if (at[k].freq >= 0) rope::rotate(u, v, s_cs + row[k] * a.f.n + at[k].freq, a.f.interleaved);
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
    if (D % 16 || D > 512 || B > 65535 || Hq > 1024 || Hkv > 1024)
        return fail(MEDUSA_ERR_UNSUPPORTED, "rope_rows: head dim %d must be a multiple of 16 up to 512, at most 65535 sequences and 1024 heads", D);
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
    // Blocks of about four batches a thread; where that leaves SMs without a block, of fewer
    // rows, then of fewer heads.
    const int all = Hq + Hkv, items = D / 16, sms = sm_count();
    a.rows = std::clamp(4 * kBatch * kThreads / (all * items), 1, kMaxRows);
    while (a.rows > 1 && (long long)B * ((T + a.rows - 1) / a.rows) < 2 * sms) a.rows /= 2;
    a.per_block = all;
    while (a.per_block > 16 && (long long)B * ((T + a.rows - 1) / a.rows) * ((all + a.per_block - 1) / a.per_block) < sms)
        a.per_block = (a.per_block + 1) / 2;
    const dim3 grid((T + a.rows - 1) / a.rows, (all + a.per_block - 1) / a.per_block, B);
    const size_t smem = (size_t)a.rows * n_freq * sizeof(float2);  // at most 16 * 256 * 8 bytes
    cudaStream_t st = as_stream(stream);
    const cudaError_t e = dtype == MEDUSA_F32 ? launch(rope_rows_kernel<float>, grid, dim3(kThreads), smem, st, a)
                                              : launch(rope_rows_kernel<uint16_t>, grid, dim3(kThreads), smem, st, a);
    if (e != cudaSuccess) return fail(MEDUSA_ERR_CUDA, "rope_rows: launch failed: %s", cudaGetErrorString(e));
    return MEDUSA_OK;
}
