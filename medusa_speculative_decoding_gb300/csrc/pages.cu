// pages.cu -- who holds which page of the 8-bit cache: fork, free and reserve
// pages of sequences in one call, and compact a pool.
//
// Several continuations of one text (the branches a sampler keeps, a prompt that
// many requests begin with) share its full pages; only the page a sequence still
// writes to has to be its own.  Which pages are free follows from the tables
// alone, so no allocator state exists that could disagree with them: every call
// counts the references anew (a table of 64 x 512 entries is 128 KB).
//
//   pages_fork_kernel    : one cluster of CTAs.  Sequence tables, reference
//                          counts and the list of free pages are each spread
//                          over the cluster's threads; cluster barriers stand
//                          between the steps.  One launch does what a chain of
//                          dependent small launches would.
//   pages_copy_open_kernel : the open pages that forks take a copy of
//   pages_compact_kernel : one cluster; live pages are ranked by a scan, those
//                          behind the last hole move down, the tables follow
//   pages_move_kernel    : their contents
//
// The planning kernels are bound by the latency of six dependent steps (14 us for 64
// rows of 8192 tokens in pages of 16, 16 us to compact a pool of 8192 pages); a cluster
// barrier costs less than a launch between two of them would.  The move is bound by
// HBM: 2048 pages of 128 KB in 82 to 86 us, 6.2 to 6.5 TB/s read and written.
#include "common.cuh"
#include "q8.cuh"
#include "umma.cuh"

namespace medusa {
namespace {

constexpr int kPlanCtas = 8;  // one portable cluster
constexpr int kPlanThreads = 1024;

// Exclusive scan of one int per thread over the block; returns the thread's
// offset and the block's sum.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += u;
    }
    __syncthreads();  // s_warp free again
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int y = lane < kPlanThreads / 32 ? s_warp[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += u;
        }
        s_warp[lane] = y;
    }
    __syncthreads();
    *sum = s_warp[kPlanThreads / 32 - 1];
    return (warp ? s_warp[warp - 1] : 0) + x - v;
}

struct ForkArgs {
    const int32_t *table, *kv_len, *src, *need, *held;
    int32_t *table_out, *kv_len_out, *refs, *taken;
    int32_t* run;      // ws [B]: leading pages of each source row
    int32_t* counts;   // ws [kPlanCtas]
    int2* copies;      // ws [B]: open page to copy and its copy, x = -1: none
    int32_t* copy_rows;  // ws [B]: rows of it in use
    int32_t* free_list;  // ws [n_pages]
    int B, M, P, n_pages;
};

__global__ void __launch_bounds__(kPlanThreads) pages_fork_kernel(const ForkArgs a) {
    __shared__ int s_lead[q8::kMaxBatch];  // the row that keeps source s's open page
    __shared__ int s_have[q8::kMaxBatch];  // pages that row b has before it takes any
    __shared__ int s_src[q8::kMaxBatch];   // source of row b, -1: none
    __shared__ int s_warp[32];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, rank = blockIdx.x;
    const int gtid = rank * kPlanThreads + tid, gthreads = kPlanCtas * kPlanThreads;
    const int B = a.B, M = a.M, P = a.P, n = a.n_pages;
    const long long entries = (long long)B * M;
    auto page_ok = [&](int p) { return p >= 0 && p < n; };

    for (int b = gtid; b < B; b += gthreads) a.run[b] = M;
    for (int p = gtid; p < n; p += gthreads) a.refs[p] = a.held ? max(a.held[p], 0) : 0;
    umma::cluster_sync();

    // 1. leading pages of every row: where the first entry without a page stands
    for (long long x = gtid; x < entries; x += gthreads) {
        const int j = (int)(x % M);
        if (!page_ok(a.table[x]) && (j == 0 || page_ok(a.table[x - 1]))) atomicMin(&a.run[x / M], j);
    }
    umma::cluster_sync();

    // 2. what each row goes on from; every CTA works this out for all rows
    const int b_own = tid;  // B <= kPlanThreads
    int src = -1, status = 0, len = 0, whole = 0, used = 0, have = 0, takes = 0;
    bool copies = false, fits = true;
    if (b_own < B) {
        s_lead[b_own] = B;
        src = a.src ? a.src[b_own] : b_own;
        if (src < -1 || src >= B) { src = -1; status = -2; }
        if (src >= 0) {
            len = a.kv_len[src];
            if (len < 0 || len > M * P || (len + P - 1) / P > __ldcg(&a.run[src])) { src = -1; status = -2; len = 0; }
        }
        s_src[b_own] = src;
    }
    __syncthreads();
    if (src >= 0) atomicMin(&s_lead[src], src == b_own ? -1 : b_own);
    __syncthreads();
    if (src >= 0) {
        const int lead = s_lead[src] < 0 ? src : s_lead[src];
        whole = len / P;
        used = (len + P - 1) / P;
        have = lead == b_own ? __ldcg(&a.run[src]) : whole;
        copies = lead != b_own && used > whole;
        const long long want = ((long long)len + (a.need ? max(a.need[b_own], 0) : 0) + P - 1) / P;
        fits = want <= M;
        takes = fits ? max((int)want - have, copies ? 1 : 0) : 0;
    }
    if (b_own < B) s_have[b_own] = have;
    int total;
    const int first = block_scan(takes, s_warp, &total);  // its barriers publish s_have too

    // 3. the rows' own tables and the references they hold
    for (long long x = gtid; x < entries; x += gthreads) {
        const int b = (int)(x / M), j = (int)(x - (long long)b * M);
        const int p = j < s_have[b] ? a.table[(long long)s_src[b] * M + j] : -1;
        a.table_out[x] = p;
        if (p >= 0) atomicAdd(&a.refs[p], 1);
    }
    umma::cluster_sync();

    // 4. free pages in rising order: each CTA counts its slice, then ranks it
    const int per = (n + kPlanCtas - 1) / kPlanCtas;
    const int p0 = min(rank * per, n), p1 = min(p0 + per, n);
    int mine = 0;
    for (int p = p0 + tid; p < p1; p += kPlanThreads) mine += __ldcg(&a.refs[p]) == 0;
    int slice;
    block_scan(mine, s_warp, &slice);
    if (tid == 0) a.counts[rank] = slice;
    umma::cluster_sync();
    int base = 0, free_pages = 0;
    for (int r = 0; r < kPlanCtas; ++r) {
        const int c = __ldcg(&a.counts[r]);
        base += r < rank ? c : 0;
        free_pages += c;
    }
    for (int q = p0; q < p1 && base < total; q += kPlanThreads) {
        const int p = q + tid;
        const int is_free = p < p1 && __ldcg(&a.refs[p]) == 0;
        int sum;
        const int at = base + block_scan(is_free, s_warp, &sum);
        if (is_free && at < total) a.free_list[at] = p;
        base += sum;
    }
    umma::cluster_sync();

    // 5. rows take their pages; a row's share begins at its offset, so a row that
    // finds too few leaves them to no one.  A row that needs none lacks none.
    const bool served = fits && (takes == 0 || (long long)first + takes <= free_pages);
    if (b_own < B && rank == 0) {
        int2 c = make_int2(-1, -1);
        if (copies && served) c = make_int2(a.table[(long long)src * M + whole], __ldcg(&a.free_list[first]));
        a.copies[b_own] = c;
        a.copy_rows[b_own] = len - whole * P;
        a.kv_len_out[b_own] = copies && !served ? whole * P : len;
        a.taken[b_own] = status ? status : (src < 0 ? 0 : (served ? takes : -1));
    }
    __syncthreads();
    if (b_own < B) {  // s_lead: first page taken, s_src: how many
        s_lead[b_own] = first;
        s_src[b_own] = served ? takes : 0;
    }
    __syncthreads();
    const int lane = tid & 31;
    for (int b = gtid >> 5; b < B; b += gthreads >> 5)
        for (int k = lane; k < s_src[b]; k += 32) {
            const int p = __ldcg(&a.free_list[s_lead[b] + k]);
            a.table_out[(long long)b * M + s_have[b] + k] = p;
            a.refs[p] = 1;
        }
}

// Copies of the open pages: the rows in use of one head's K or V per CTA.
__global__ void __launch_bounds__(256) pages_copy_open_kernel(uint4* __restrict__ kp, uint4* __restrict__ vp,
                                                              float* __restrict__ ks, float* __restrict__ vs,
                                                              const int2* __restrict__ copies,
                                                              const int32_t* __restrict__ copy_rows, int Hkv, int P,
                                                              int row16) {
    pdl_wait();
    pdl_trigger();
    const int2 c = copies[blockIdx.y];
    if (c.x < 0) return;
    const int h = blockIdx.x >> 1, kv = blockIdx.x & 1;
    const int n = copy_rows[blockIdx.y] * row16;
    uint4* pages = kv ? vp : kp;
    const uint4* src = pages + ((size_t)c.x * Hkv + h) * P * row16;
    uint4* dst = pages + ((size_t)c.y * Hkv + h) * P * row16;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += 256) dst[i] = src[i];
    if (threadIdx.x == 0) {
        float* s = kv ? vs : ks;
        s[(size_t)c.y * Hkv + h] = s[(size_t)c.x * Hkv + h];
    }
}

struct CompactArgs {
    const int32_t *table, *held;
    int32_t *table_out, *new_page, *live;
    int32_t* flag;    // ws [n_pages]: in use
    int32_t* counts;  // ws [2 * kPlanCtas]
    int32_t* holes;   // ws [n_pages]
    int2* moves;      // ws [n_pages]
    int32_t* n_moves;  // ws [1]
    int B, M, n_pages;
};

__global__ void __launch_bounds__(kPlanThreads) pages_compact_kernel(const CompactArgs a) {
    __shared__ int s_warp[32];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, rank = blockIdx.x;
    const int gtid = rank * kPlanThreads + tid, gthreads = kPlanCtas * kPlanThreads;
    const int n = a.n_pages;
    const long long entries = (long long)a.B * a.M;
    for (int p = gtid; p < n; p += gthreads) a.flag[p] = a.held && a.held[p] > 0;
    umma::cluster_sync();
    for (long long x = gtid; x < entries; x += gthreads) {
        const int p = a.table[x];
        if (p >= 0 && p < n) a.flag[p] = 1;
    }
    umma::cluster_sync();

    const int per = (n + kPlanCtas - 1) / kPlanCtas;
    const int p0 = min(rank * per, n), p1 = min(p0 + per, n);
    int mine = 0, slice;
    for (int p = p0 + tid; p < p1; p += kPlanThreads) mine += __ldcg(&a.flag[p]);
    block_scan(mine, s_warp, &slice);
    if (tid == 0) a.counts[rank] = slice;
    umma::cluster_sync();
    int count = 0;
    for (int r = 0; r < kPlanCtas; ++r) count += __ldcg(&a.counts[r]);
    // holes lie below `count`, the pages that fill them at or above it; there are
    // as many of the one as of the other
    mine = 0;
    for (int p = p0 + tid; p < p1; p += kPlanThreads) mine += p < count ? 1 - __ldcg(&a.flag[p]) : 0;
    int holes;
    block_scan(mine, s_warp, &holes);
    if (tid == 0) a.counts[kPlanCtas + rank] = holes;
    umma::cluster_sync();
    int hole_at = 0, move_at = 0, n_moves = 0;
    for (int r = 0; r < kPlanCtas; ++r) {
        const int h = __ldcg(&a.counts[kPlanCtas + r]), l = __ldcg(&a.counts[r]);
        const int q0 = min(r * per, n), q1 = min(q0 + per, n);
        const int below = max(0, min(q1, count) - q0) - h;  // the slice's live pages below `count`
        if (r < rank) { hole_at += h; move_at += l - below; }
        n_moves += h;
    }
    for (int q = p0; q < p1; q += kPlanThreads) {
        const int p = q + tid;
        const int f = p < p1 ? __ldcg(&a.flag[p]) : 0;
        const int hole = p < p1 && p < count && !f;
        int sum;
        const int h = hole_at + block_scan(hole, s_warp, &sum);
        if (hole) a.holes[h] = p;
        hole_at += sum;
    }
    umma::cluster_sync();
    for (int q = p0; q < p1; q += kPlanThreads) {
        const int p = q + tid;
        const int f = p < p1 ? __ldcg(&a.flag[p]) : 0;
        const int moved = p >= count && f;
        int sum;
        const int m = move_at + block_scan(moved, s_warp, &sum);
        if (p < p1) {
            int to = f ? p : -1;
            if (moved) {
                to = __ldcg(&a.holes[m]);
                a.moves[m] = make_int2(p, to);
            }
            a.new_page[p] = to;
        }
        move_at += sum;
    }
    if (gtid == 0) {
        *a.live = count;
        *a.n_moves = n_moves;
    }
    umma::cluster_sync();
    for (long long x = gtid; x < entries; x += gthreads) {
        const int p = a.table[x];
        a.table_out[x] = p >= 0 && p < n ? __ldcg(&a.new_page[p]) : -1;
    }
}

// Contents of the moved pages.  Sources lie behind every destination, so no
// move reads what another writes.  Item = (move, K or V, piece of the page).
constexpr int kMoveThreads = 256;
constexpr int kMovePiece = 1024;  // 16-byte words per item: four per thread
__global__ void __launch_bounds__(kMoveThreads) pages_move_kernel(uint4* __restrict__ kp, uint4* __restrict__ vp,
                                                                  float* __restrict__ ks, float* __restrict__ vs,
                                                                  const int2* __restrict__ moves,
                                                                  const int32_t* __restrict__ n_moves, int Hkv,
                                                                  int page16, int pieces) {
    pdl_wait();
    pdl_trigger();
    const long long items = 2ll * *n_moves * pieces;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int piece = (int)(it % pieces), kv = (int)(it / pieces & 1);
        const int2 m = moves[it / pieces >> 1];
        uint4* pages = kv ? vp : kp;
        const uint4* src = pages + (size_t)m.x * page16;
        uint4* dst = pages + (size_t)m.y * page16;
        const int i0 = piece * kMovePiece + threadIdx.x;
        uint4 w[kMovePiece / kMoveThreads];
#pragma unroll
        for (int k = 0; k < kMovePiece / kMoveThreads; ++k)
            if (i0 + k * kMoveThreads < page16) w[k] = src[i0 + k * kMoveThreads];
#pragma unroll
        for (int k = 0; k < kMovePiece / kMoveThreads; ++k)
            if (i0 + k * kMoveThreads < page16) dst[i0 + k * kMoveThreads] = w[k];
        if (piece == 0)
            for (int h = threadIdx.x; h < Hkv; h += kMoveThreads) {
                float* s = kv ? vs : ks;
                s[(size_t)m.y * Hkv + h] = s[(size_t)m.x * Hkv + h];
            }
    }
}

// workspace of the fork: int32 words, the int2 lists first
struct ForkWs {
    size_t copies, rows, run, counts, list, bytes;
    ForkWs(int B, int n_pages) {
        copies = 0;
        rows = copies + (size_t)B * 8;
        run = rows + (size_t)B * 4;
        counts = run + (size_t)B * 4;
        list = counts + kPlanCtas * 4;
        bytes = align_up(list + (size_t)n_pages * 4, 16);
    }
};
struct CompactWs {
    size_t moves, flag, holes, counts, n_moves, bytes;
    explicit CompactWs(int n_pages) {
        moves = 0;
        flag = moves + (size_t)n_pages * 8;
        holes = flag + (size_t)n_pages * 4;
        counts = holes + (size_t)n_pages * 4;
        n_moves = counts + 2 * kPlanCtas * 4;
        bytes = align_up(n_moves + 4, 16);
    }
};

}  // namespace
}  // namespace medusa

using namespace medusa;

extern "C" size_t medusa_kv_pages_fork_workspace(int B, int n_pages) {
    return B < 1 || n_pages < 1 ? 0 : ForkWs(B, n_pages).bytes;
}

extern "C" int medusa_kv_pages_fork(void* k_pages, void* v_pages, float* k_scale, float* v_scale,
                                    const int32_t* page_table, const int32_t* kv_len, const int32_t* src,
                                    const int32_t* need, const int32_t* held, int B, int Hkv, int D, int P,
                                    int n_pages, int M, int32_t* page_table_out, int32_t* kv_len_out, int32_t* refs,
                                    int32_t* taken, void* ws, size_t ws_bytes, void* stream) {
    if (B < 1 || Hkv < 1 || n_pages < 1 || M < 1)
        return fail(MEDUSA_ERR_INVALID_ARG, "kv_pages_fork: sizes must be positive");
    if (int rc = q8::check_pool("kv_pages_fork", B, Hkv, D, P, n_pages, M)) return rc;
    if (!k_pages || !v_pages || !k_scale || !v_scale || !page_table || !kv_len || !page_table_out || !kv_len_out ||
        !refs || !taken)
        return fail(MEDUSA_ERR_INVALID_ARG, "kv_pages_fork: null pointer");
    if (page_table_out == page_table || kv_len_out == kv_len)
        return fail(MEDUSA_ERR_INVALID_ARG, "kv_pages_fork: outputs must not be the table or lengths read");
    if (!aligned16(k_pages) || !aligned16(v_pages))
        return fail(MEDUSA_ERR_INVALID_ARG, "kv_pages_fork: pages must be 16-byte aligned");
    const ForkWs w(B, n_pages);
    if (!ws || ws_bytes < w.bytes)
        return fail(MEDUSA_ERR_WORKSPACE, "kv_pages_fork: workspace of %zu bytes needed", w.bytes);
    if (!aligned16(ws)) return fail(MEDUSA_ERR_INVALID_ARG, "kv_pages_fork: ws must be 16-byte aligned");
    char* p = static_cast<char*>(ws);
    ForkArgs a{};
    a.table = page_table; a.kv_len = kv_len; a.src = src; a.need = need; a.held = held;
    a.table_out = page_table_out; a.kv_len_out = kv_len_out; a.refs = refs; a.taken = taken;
    a.copies = (int2*)(p + w.copies); a.copy_rows = (int32_t*)(p + w.rows); a.run = (int32_t*)(p + w.run);
    a.counts = (int32_t*)(p + w.counts); a.free_list = (int32_t*)(p + w.list);
    a.B = B; a.M = M; a.P = P; a.n_pages = n_pages;
    cudaStream_t st = as_stream(stream);
    cudaError_t e = launch_cluster(pages_fork_kernel, dim3(kPlanCtas), dim3(kPlanThreads), 0, st, kPlanCtas, a);
    if (e == cudaSuccess && src)  // without src every row keeps its own open page
        e = launch(pages_copy_open_kernel, dim3(2 * Hkv, B), dim3(256), 0, st, (uint4*)k_pages, (uint4*)v_pages, k_scale,
                   v_scale, a.copies, a.copy_rows, Hkv, P, D / 16);
    if (e != cudaSuccess) return fail(MEDUSA_ERR_CUDA, "kv_pages_fork: launch failed: %s", cudaGetErrorString(e));
    return MEDUSA_OK;
}

extern "C" size_t medusa_kv_pages_compact_workspace(int n_pages) { return n_pages < 1 ? 0 : CompactWs(n_pages).bytes; }

extern "C" int medusa_kv_pages_compact(void* k_pages, void* v_pages, float* k_scale, float* v_scale,
                                       const int32_t* page_table, const int32_t* held, int B, int Hkv, int D, int P,
                                       int n_pages, int M, int32_t* page_table_out, int32_t* new_page, int32_t* live,
                                       void* ws, size_t ws_bytes, void* stream) {
    if (B < 1 || Hkv < 1 || n_pages < 1 || M < 1)
        return fail(MEDUSA_ERR_INVALID_ARG, "kv_pages_compact: sizes must be positive");
    if (int rc = q8::check_pool("kv_pages_compact", B, Hkv, D, P, n_pages, M)) return rc;
    if (!k_pages || !v_pages || !k_scale || !v_scale || !page_table || !page_table_out || !new_page || !live)
        return fail(MEDUSA_ERR_INVALID_ARG, "kv_pages_compact: null pointer");
    if (!aligned16(k_pages) || !aligned16(v_pages))
        return fail(MEDUSA_ERR_INVALID_ARG, "kv_pages_compact: pages must be 16-byte aligned");
    const CompactWs w(n_pages);
    if (!ws || ws_bytes < w.bytes)
        return fail(MEDUSA_ERR_WORKSPACE, "kv_pages_compact: workspace of %zu bytes needed", w.bytes);
    if (!aligned16(ws)) return fail(MEDUSA_ERR_INVALID_ARG, "kv_pages_compact: ws must be 16-byte aligned");
    char* p = static_cast<char*>(ws);
    CompactArgs a{};
    a.table = page_table; a.held = held; a.table_out = page_table_out; a.new_page = new_page; a.live = live;
    a.moves = (int2*)(p + w.moves); a.flag = (int32_t*)(p + w.flag); a.holes = (int32_t*)(p + w.holes);
    a.counts = (int32_t*)(p + w.counts); a.n_moves = (int32_t*)(p + w.n_moves);
    a.B = B; a.M = M; a.n_pages = n_pages;
    cudaStream_t st = as_stream(stream);
    cudaError_t e = launch_cluster(pages_compact_kernel, dim3(kPlanCtas), dim3(kPlanThreads), 0, st, kPlanCtas, a);
    const int page16 = Hkv * P * D / 16, pieces = (page16 + kMovePiece - 1) / kMovePiece;
    if (e == cudaSuccess)
        e = launch(pages_move_kernel, dim3(sm_count() * 8), dim3(kMoveThreads), 0, st, (uint4*)k_pages, (uint4*)v_pages,
                   k_scale, v_scale, a.moves, a.n_moves, Hkv, page16, pieces);
    if (e != cudaSuccess) return fail(MEDUSA_ERR_CUDA, "kv_pages_compact: launch failed: %s", cudaGetErrorString(e));
    return MEDUSA_OK;
}
