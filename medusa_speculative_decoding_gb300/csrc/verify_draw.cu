// verify_draw.cu -- acceptance of a tree by tokens drawn from the target's probabilities
// with given random numbers ("Giai ma dau co" page, "Faster without changing the result";
// "Medusa Heads" glossary page, "Tree attention and acceptance").
//
// The candidates are fixed before the target is asked, so the draft is a point mass on each
// of them and the speculative rule becomes: draw a token from the target's row, accept the
// child that holds it, and end with the token itself where no child does.  Every token of the
// round then follows the target's distribution.  The draw at depth d is the smallest v with
//   p_0 + ... + p_v > u_d * (p_0 + ... + p_{V-1}).
//
// A row has V boundaries, each of which could fall next to u: sums in float32 would pick
// another token in V * 2^-23 of the draws, 1.5% at V = 128256.  So a sum is a pair of float32, high
// and low part (in double, of which an SM adds two a cycle, the draws of 64 rows of 32000 took 40 us
// instead of 6).  A thread adds sixteen values in float32 and, beside them, what each addition rounded
// away, which is exact: 2^-24 of the sum at most, so that the sixteen of them are off by 2^-40 of it
// whatever the values' size.  From there on pairs are added, off by 2^-46 of the result each time, at
// most some 270 one after the other (V = 2^24): 2^-37 of a row's total in all at most.
//
// A cluster of CTAs draws from one row: each CTA sums a contiguous slice, the totals are
// pushed to every CTA, and the one whose slice holds the number finds the token in it.
//   draw_walk_kernel  a cluster per sequence walks down the tree, a row per level: reads
//                     only the rows that it visits, one level after the other (52 us for 32
//                     trees of 64 nodes, 128256 tokens: the longest walk, 5 us a level)
//   draw_rows_kernel  a cluster per row draws from all rows at once, and walk_kernel follows
//                     the children: fewer steps in a row where there are few rows (11 us for 64
//                     nodes, 32000 tokens)
#include <algorithm>

#include "common.cuh"
#include "umma.cuh"

namespace medusa {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBatch = 4;         // float4 of a thread with their loads in flight
constexpr int kMaxCluster = 8;
constexpr int kSlice = 8192;      // values of a CTA, where the cluster can be that large
constexpr int kMaxNodes = 512;
// Bytes of rows, and CTAs for them, up to which drawing from all of them beats walking.  All take some 8 us for
// every 304 CTAs (two an SM) or 20 MB, a walk 5 to 9 us a level, whatever the rows.  Measured, us, all / walking (trees
// x nodes x tokens):
//   up to 304 CTAs        9 x 1000 8 / 14; 64 x 8192 10 / 19; 64 x 32000 11 / 19; 300 x 8192 12 / 21; 32 x 128256 14 / 23;
//                         4 x 9 x 128256 (18 MB) 14 / 30
//   up to 1024            341 x 5000 18 / 19; 8 x 64 x 8192 21 / 42; 64 x 64000 20 / 16; 24 x 25 x 8000 (18 MB) 21 / 42; 341 x
//                         10000 27 / 22; 2 x 341 x 6000 27 / 25; 16 x 64 x 4000 33 / 35; 64 x 16 x 2000 31 / 27
//   more                  32 x 64 x 1000 52 / 42; 64 x 64 x 1000 99 / 45
//   more bytes            12 x 64 x 8000 (23 MB) 29 / 47; 64 x 128256 (31 MB) 25 / 16; 38 x 300000 (43 MB) 41 / 27; 8 x 64 x
//                         32000 (62 MB) 64 / 39
constexpr long long kAllRows = 20ll << 20, kAllBlocks = 1024;

struct DrawArgs {
    const float *probs, *u;
    const int32_t *cand, *parent;
    int32_t* drawn;  // ws [B][N]
    int32_t *accept_len, *best_node, *path_nodes, *next_tok;
    int B, N, V, Dmax, slice;  // slice: values of a CTA, a multiple of 128 * kWarps
};

struct DrawSmem {
    float2 total[kMaxCluster];  // of every CTA of the cluster
    float2 warp_total[kWarps];
    int token;
};

// probabilities: negative ones and NaN count as 0, those above 1 as 1
__device__ __forceinline__ float clean(float p) { return fminf(fmaxf(p, 0.f), 1.f); }

// Sums of two float32: x + y exactly, |y| at most half of x's last place.
__device__ __forceinline__ float2 two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t)));
}
__device__ __forceinline__ float2 add(float2 a, float2 b) {
    const float2 s = two_sum(a.x, b.x);
    return two_sum(s.x, __fadd_rn(s.y, __fadd_rn(a.y, b.y)));
}
__device__ __forceinline__ bool greater(float2 a, float2 b) { return a.x > b.x || (a.x == b.x && a.y > b.y); }
__device__ __forceinline__ bool positive(float2 a) { return a.x > 0.f; }
__device__ __forceinline__ float2 shfl_up2(float2 v, int o) {
    return make_float2(__shfl_up_sync(0xffffffffu, v.x, o), __shfl_up_sync(0xffffffffu, v.y, o));
}
__device__ __forceinline__ float2 shfl2(float2 v, int l) {
    return make_float2(__shfl_sync(0xffffffffu, v.x, l), __shfl_sync(0xffffffffu, v.y, l));
}
// inclusive sums over the lanes
__device__ __forceinline__ float2 scan(float2 v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float2 u = shfl_up2(v, o);
        if (lane >= o) v = add(u, v);
    }
    return v;
}
// The lane whose part holds `target`, the parts laid end to end behind `base`: the first whose
// end lies behind it, the last with any weight where rounding leaves none, -1 where all are
// empty.  base becomes what lies before that part (behind all of them where over is false).
__device__ __forceinline__ int part_of(float2 mine, float2 target, float2& base, bool& over) {
    const float2 upto = add(base, scan(mine));
    const unsigned some = __ballot_sync(0xffffffffu, positive(mine)), behind = __ballot_sync(0xffffffffu, positive(mine) && greater(upto, target));
    over = behind != 0;
    if (!some) return -1;
    const int at = behind ? __ffs(behind) - 1 : 31 - __clz(some);
    const float2 before = shfl_up2(upto, 1), end = shfl2(upto, 31);
    base = behind ? (at ? shfl2(before, at) : base) : end;
    return at;
}

__device__ __forceinline__ void st_cluster_s32(uint32_t addr, int v) {
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// four values from v on; behind `end` zero
__device__ __forceinline__ float4 values4(const float* row, int v, int end, bool aligned) {
    if (aligned && v + 4 <= end) {
        const uint4 r = ld_stream16(row + v);
        return make_float4(clean(__uint_as_float(r.x)), clean(__uint_as_float(r.y)), clean(__uint_as_float(r.z)), clean(__uint_as_float(r.w)));
    }
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = v + i < end ? clean(__ldg(row + v + i)) : 0.f;
    return make_float4(x[0], x[1], x[2], x[3]);
}

// The token drawn from row[0 .. V) with the number that `number` gives (called by the first warp, behind
// a barrier of the block), for all threads of the cluster (-1: the row has no weight).  Called by every
// thread of the cluster's CTAs, which arrived at the cluster's barrier before the first call.
template <typename Number>
__device__ __forceinline__ int draw(const DrawArgs& a, const float* row, Number number, DrawSmem& s, int rank, int ctas, bool first) {
    using namespace umma;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool aligned = (reinterpret_cast<uintptr_t>(row) & 15u) == 0;
    const int per_warp = a.slice / kWarps;  // a multiple of 128
    const int begin = min(a.V, rank * a.slice + warp * per_warp), end = min(a.V, begin + per_warp);
    float2 sum = make_float2(0.f, 0.f);
    for (int v0 = begin; v0 < end; v0 += 128 * kBatch) {
        float4 x[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int v = v0 + 128 * k + 4 * lane;
            x[k] = v < end ? values4(row, v, end, aligned) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float hi = 0.f, lo = 0.f;  // lo: what hi's additions rounded away
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const float y[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 t = two_sum(hi, y[i]);
                hi = t.x;
                lo = __fadd_rn(lo, t.y);
            }
        }
        sum = add(sum, two_sum(hi, lo));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum = add(sum, make_float2(__shfl_xor_sync(0xffffffffu, sum.x, o), __shfl_xor_sync(0xffffffffu, sum.y, o)));
    if (lane == 0) s.warp_total[warp] = sum;
    __syncthreads();
    if (first) cluster_wait();  // every CTA of the cluster runs: its shared memory can be written
    const float2 none = make_float2(0.f, 0.f);
    if (warp == 0) {
        float2 t = lane < kWarps ? s.warp_total[lane] : none;
        t = shfl2(scan(t), 31);
        if (lane < ctas) st_cluster_f32x2(cluster_map(smem_addr(&s.total[rank]), lane), t.x, t.y);
    }
    cluster_sync();
    if (warp == 0) {
        // Every CTA finds the same CTA of the cluster, and that one the warp's part and the token.
        const float2 part = lane < ctas ? s.total[lane] : none;
        const float2 all = shfl2(scan(part), 31);
        const float un = fmaxf(number(), 0.f), ph = __fmul_rn(un, all.x);
        // (from 1 on the last token: no sum, whatever order it was added up in, lies behind infinity)
        const float2 target = un >= 1.f ? make_float2(INFINITY, 0.f) : two_sum(ph, __fadd_rn(__fmaf_rn(un, all.x, -ph), __fmul_rn(un, all.y)));
        float2 base = none;
        bool over;
        const int winner = part_of(part, target, base, over);
        if (rank == max(winner, 0)) {
            int token = -1;
            if (winner >= 0) {
                if (!over) base = none;  // (the last weight of all: every sum counts as too small)
                const float2 goal = over ? target : make_float2(INFINITY, 0.f);
                const int w_at = part_of(lane < kWarps ? s.warp_total[lane] : none, goal, base, over);
                const int b0 = min(a.V, rank * a.slice + w_at * per_warp), b1 = min(a.V, b0 + per_warp);
                // 1024 values at a time, 32 a lane, then a lane's values one a lane
                const bool found_warp = over;
                for (int v0 = b0; v0 < b1; v0 += 1024) {
                    float2 mine = none;
                    const int from = v0 + 32 * lane;
                    float4 x[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = from + 4 * k < b1 ? values4(row, from + 4 * k, b1, aligned) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        mine = add(mine, two_sum(x[k].x, x[k].y));
                        mine = add(mine, two_sum(x[k].z, x[k].w));
                    }
                    bool in_chunk, in_lane;
                    const int l = part_of(mine, found_warp ? goal : make_float2(INFINITY, 0.f), base, in_chunk);
                    if (l < 0) continue;
                    const int v = v0 + 32 * l + lane;
                    float2 before = base;
                    const int e = part_of(make_float2(v < b1 ? clean(__ldg(row + v)) : 0.f, 0.f), in_chunk ? goal : make_float2(INFINITY, 0.f), before, in_lane);
                    token = v0 + 32 * l + e;
                    if (in_chunk) break;
                }
            }
            if (lane < ctas) st_cluster_s32(cluster_map(smem_addr(&s.token), lane), token);
        }
    }
    cluster_sync();
    return s.token;
}

// The child of `node` that holds token t, the lowest one; N: none.  Called by the whole block.
__device__ __forceinline__ int child_of(const int* parent, const int* cand, int N, int node, int t, int* s_child) {
    if (threadIdx.x == 0) *s_child = N;
    __syncthreads();
    if (t >= 0)
        for (int j = threadIdx.x; j < N; j += blockDim.x)
            if (j > node && parent[j] == node && cand[j] == t) atomicMin(s_child, j);
    __syncthreads();
    return *s_child;
}

// path: how the round went, written by the block's threads
__device__ __forceinline__ void finish(const DrawArgs& a, int b, int steps, int node, int token, const int* path) {
    for (int i = threadIdx.x; i <= a.Dmax; i += blockDim.x) a.path_nodes[(size_t)b * (a.Dmax + 1) + i] = i <= steps ? path[i] : -1;
    if (threadIdx.x == 0) {
        a.accept_len[b] = steps;
        a.best_node[b] = node;
        a.next_tok[b] = token;
    }
}

__global__ void __launch_bounds__(kThreads, 2) draw_walk_kernel(const DrawArgs a) {
    __shared__ DrawSmem s;
    __shared__ int s_parent[kMaxNodes], s_cand[kMaxNodes], s_path[kMaxNodes], s_child;
    const int ctas = gridDim.x, rank = blockIdx.x, b = blockIdx.y;
    umma::cluster_arrive_relaxed();
    pdl_wait();
    pdl_trigger();
    for (int i = threadIdx.x; i < a.N; i += kThreads) {
        s_parent[i] = a.parent[i];
        s_cand[i] = a.cand[(size_t)b * a.N + i];
    }
    int node = 0, token = -1, steps = 0;
    if (threadIdx.x == 0) s_path[0] = 0;
    for (;;) {
        const float u = a.u[(size_t)b * (a.Dmax + 1) + steps];
        token = draw(a, a.probs + ((size_t)b * a.N + node) * a.V, [=] { return u; }, s, rank, ctas, steps == 0);
        if (steps == a.Dmax) break;
        const int child = child_of(s_parent, s_cand, a.N, node, token, &s_child);
        if (child == a.N) break;
        node = child;
        ++steps;
        if (threadIdx.x == 0) s_path[steps] = node;
        __syncthreads();  // s_child is set anew
    }
    __syncthreads();
    if (rank == 0) finish(a, b, steps, node, token, s_path);
}

__global__ void __launch_bounds__(kThreads, 2) draw_rows_kernel(const DrawArgs a) {
    __shared__ DrawSmem s;
    __shared__ int s_parent[kMaxNodes];
    __shared__ float s_u[kMaxNodes];
    static_assert(kThreads >= kMaxNodes, "one node and one number a thread");
    const int ctas = gridDim.x, rank = blockIdx.x, node = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    umma::cluster_arrive_relaxed();
    pdl_wait();
    pdl_trigger();
    if (tid < a.N) s_parent[tid] = a.parent[tid];
    if (tid <= a.Dmax) s_u[tid] = a.u[(size_t)b * (a.Dmax + 1) + tid];
    // The steps that a walk takes to this node; any number where none gets here.
    auto number = [&] {
        int d = 0;
        for (int j = node; j > 0 && d < a.Dmax; ++d) {
            const int up = s_parent[j];
            j = up < j ? up : 0;
        }
        return s_u[d];
    };
    const int token = draw(a, a.probs + ((size_t)b * a.N + node) * a.V, number, s, rank, ctas, true);
    if (rank == 0 && threadIdx.x == 0) a.drawn[(size_t)b * a.N + node] = token;
}

__global__ void __launch_bounds__(256) walk_kernel(const DrawArgs a) {
    __shared__ int s_parent[kMaxNodes], s_cand[kMaxNodes], s_drawn[kMaxNodes], s_path[kMaxNodes], s_child;
    const int b = blockIdx.x;
    pdl_wait();
    pdl_trigger();
    for (int i = threadIdx.x; i < a.N; i += blockDim.x) {
        s_parent[i] = a.parent[i];
        s_cand[i] = a.cand[(size_t)b * a.N + i];
        s_drawn[i] = a.drawn[(size_t)b * a.N + i];
    }
    if (threadIdx.x == 0) s_path[0] = 0;
    __syncthreads();
    int node = 0, steps = 0;
    while (steps < a.Dmax) {
        const int child = child_of(s_parent, s_cand, a.N, node, s_drawn[node], &s_child);
        if (child == a.N) break;
        node = child;
        ++steps;
        if (threadIdx.x == 0) s_path[steps] = node;
        __syncthreads();
    }
    __syncthreads();
    finish(a, b, steps, node, s_drawn[node], s_path);
}

int check_draw(int B, int N, int V, int Dmax) {
    if (B < 1 || N < 1 || V < 1 || Dmax < 0)
        return fail(MEDUSA_ERR_INVALID_ARG, "verify_accept_tree_draw: sizes must be positive");
    if (N > kMaxNodes || Dmax >= kMaxNodes || B > 65535 || V > 1 << 24)
        return fail(MEDUSA_ERR_UNSUPPORTED, "verify_accept_tree_draw: at most %d nodes, 65535 sequences and 2^24 tokens", kMaxNodes);
    return MEDUSA_OK;
}

}  // namespace
}  // namespace medusa

using namespace medusa;

extern "C" size_t medusa_verify_draw_workspace(int B, int N, int V) {
    (void)V;
    return B < 1 || N < 1 ? 0 : (size_t)B * N * sizeof(int32_t);
}

extern "C" int medusa_verify_accept_tree_draw(const float* probs, const int32_t* cand, const int32_t* parent,
                                              const int32_t* depth, const float* u, int B, int N, int V, int Dmax,
                                              int32_t* accept_len, int32_t* best_node, int32_t* path_nodes,
                                              int32_t* next_tok, void* ws, size_t ws_bytes, void* stream) {
    if (int rc = check_draw(B, N, V, Dmax)) return rc;
    if (!probs || !cand || !parent || !depth || !u || !accept_len || !best_node || !path_nodes || !next_tok)
        return fail(MEDUSA_ERR_INVALID_ARG, "verify_accept_tree_draw: null pointer");
    const size_t need = medusa_verify_draw_workspace(B, N, V);
    if (!ws || ws_bytes < need)
        return fail(MEDUSA_ERR_WORKSPACE, "verify_accept_tree_draw: workspace of %zu bytes needed", need);
    if (reinterpret_cast<uintptr_t>(ws) & 3u)
        return fail(MEDUSA_ERR_INVALID_ARG, "verify_accept_tree_draw: ws must be 4-byte aligned");
    DrawArgs a{probs, u, cand, parent, (int32_t*)ws, accept_len, best_node, path_nodes, next_tok, B, N, V, Dmax, 0};
    const int ctas = std::min(kMaxCluster, (V + kSlice - 1) / kSlice), unit = 128 * kWarps;
    a.slice = (int)(((long long)(V + ctas - 1) / ctas + unit - 1) / unit * unit);
    cudaStream_t st = as_stream(stream);
    cudaError_t e;
    if (((long long)B * N * V * 4 <= kAllRows && (long long)B * N * ctas <= kAllBlocks) || N == 1) {
        e = launch_cluster(draw_rows_kernel, dim3(ctas, N, B), dim3(kThreads), 0, st, ctas, a);
        if (e == cudaSuccess) e = launch(walk_kernel, dim3(B), dim3(256), 0, st, a);
    } else {
        e = launch_cluster(draw_walk_kernel, dim3(ctas, B), dim3(kThreads), 0, st, ctas, a);
    }
    if (e != cudaSuccess)
        return fail(MEDUSA_ERR_CUDA, "verify_accept_tree_draw: launch failed: %s", cudaGetErrorString(e));
    return MEDUSA_OK;
}
