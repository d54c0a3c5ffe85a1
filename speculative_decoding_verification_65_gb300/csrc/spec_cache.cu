// spec_cache.cu -- the plan of a tree-attention step and the commit of the
// accepted path's keys and values to the cache (include/spec_attn.h).
//
// Plan.  One CTA per sequence, one thread per node.  A node's ancestors are a
// closure over parent links, and following them one by one costs the depth in
// dependent loads (1023 for a chain of 1024).  Here each warp closes its own
// 32 nodes by pointer doubling in registers (5 rounds of shuffles: the
// ancestors inside the block as one word, and the first ancestor below the
// block, its exit); then the blocks, in order, take over the finished row of
// their exits word by word.  That is 5 shuffle rounds and at most 31 short
// steps for any shape.  One more CTA sums the key tiles of all sequences,
// which the attention divides among its CTAs.  Latency-bound: 256 nodes take
// 8 steps.
//
// Commit.  A copy of (accepted + 1) rows of Hkv * D elements per sequence,
// layer and side, in the widest vectors (16, 4 or 2 bytes) that every address
// allows.  Every CTA of a sequence checks its whole path first, so a bad
// sequence is left alone by all of them, and keeps where its rows go in shared
// memory; then each warp copies whole rows, four vectors of a lane in flight.
// Bound by the chain of loads (lengths, path and pages, rows), not by bytes:
// 34 MB for 32 layers of 32 sequences are 5 us of HBM time.
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include <atomic>

#include "spec_attn.h"
#include "spec_verify.h"
#include "attn_plan.cuh"
#include "device_common.cuh"

namespace {

using namespace spec_dev;
using namespace spec_attn;

// ------------------------------------------------------------------- plan

struct PlanParams {
    const int32_t *parent, *n_nodes, *cache_len, *page_table;
    int32_t B, N, page_size, pages_per_seq, num_pages;
    uint8_t *plan;
    PlanLayout lay;
};

__device__ __forceinline__ bool lengths_ok(const PlanParams &P, int n, int len)
{
    return n >= 0 && n <= P.N && len >= 0 &&
           (long long)len <= (long long)P.pages_per_seq * P.page_size;
}

// Tile prefix sums over the sequences, by one CTA of up to 32 warps.  A
// sequence whose parents or pages turn out bad keeps the tiles of its lengths:
// its share of the schedule is then idle.
__device__ void plan_scan(const PlanParams &P)
{
    __shared__ long long part[32];
    __shared__ long long base;
    long long *cum = reinterpret_cast<long long *>(P.plan + P.lay.cum);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        base = 0;
        cum[0] = 0;
        reinterpret_cast<WsHeader *>(P.plan)->status = SPEC_DEV_OK;
    }
    __syncthreads();
    for (int b0 = 0; b0 < P.B; b0 += (int)blockDim.x) {
        const int b = b0 + (int)threadIdx.x;
        long long v = 0;
        if (b < P.B) {
            const int n = P.n_nodes[b], len = P.cache_len[b];
            v = lengths_ok(P, n, len) ? plan_tiles(len, n) : 1;
        }
        for (int d = 1; d < 32; d <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d)
                v += o;
        }
        if (lane == 31)
            part[warp] = v;
        __syncthreads();
        long long before = base;
        for (int w = 0; w < warp; ++w)
            before += part[w];
        if (b < P.B)
            cum[b + 1] = before + v;
        __syncthreads();
        if (threadIdx.x == blockDim.x - 1)
            base = before + v;
        __syncthreads();
    }
}

__global__ void __launch_bounds__(1024) plan_kernel(const PlanParams P)
{
    extern __shared__ uint32_t rows[];  // [N][NW]: a node's ancestor words
    allow_next_kernel();
    wait_previous_kernel();
    const int b = (int)blockIdx.x;
    if (b == P.B) {
        plan_scan(P);
        return;
    }
    const int N = P.N, NW = (N + 31) / 32, W = P.lay.W;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nn = P.n_nodes[b], len = P.cache_len[b];
    const bool sized = lengths_ok(P, nn, len);
    const int live = sized ? nn : 0;
    bool bad = !sized;

    // this block's closure: node = tid (blockDim.x >= N)
    uint32_t mask = 0;
    int jump = -1, exit_ = -1;  // the in-block ancestor to go on from; the ancestor below the block
    if (tid < live) {
        mask = 1u << lane;
        if (tid > 0) {
            const int p = P.parent[(size_t)b * N + tid];
            if (p < 0 || p >= tid)
                bad = true;
            else if (p >= warp * 32)
                jump = p - warp * 32;
            else
                exit_ = p;
        }
    }
#pragma unroll
    for (int r = 0; r < 5; ++r) {
        const int from = jump >= 0 ? jump : lane;
        const uint32_t m = __shfl_sync(0xffffffffu, mask, from);
        const int e = __shfl_sync(0xffffffffu, exit_, from);
        const int j = __shfl_sync(0xffffffffu, jump, from);
        if (jump >= 0) {
            mask |= m;
            exit_ = e;
            jump = j;
        }
    }
    // pages that hold positions below the length
    if (sized && nn > 0 && P.page_table != nullptr) {
        const int used = (int)(((long long)len + P.page_size - 1) / P.page_size);
        for (int i = tid; i < used; i += (int)blockDim.x) {
            const int pg = P.page_table[(size_t)b * P.pages_per_seq + i];
            bad |= pg < 0 || pg >= P.num_pages;
        }
    }
    bad = __syncthreads_or(bad ? 1 : 0) != 0;
    const bool on = !bad && tid < live;
    if (tid < N) {
        for (int w = 0; w < NW; ++w)
            rows[tid * NW + w] = (on && w == warp) ? mask : 0u;
    }
    // words below the block come from the exit's finished row
    for (int blk = 1; blk < NW; ++blk) {
        __syncthreads();
        if (warp == blk && on && exit_ >= 0)
            for (int w = 0; w < blk; ++w)
                rows[tid * NW + w] = rows[exit_ * NW + w];
    }
    __syncthreads();
    uint32_t *out = reinterpret_cast<uint32_t *>(P.plan + P.lay.mask) + (size_t)b * N * W;
    for (int i = tid; i < N * W; i += (int)blockDim.x) {
        const int n = i / W, w = i - n * W;
        out[i] = w < NW ? rows[n * NW + w] : 0u;
    }
    if (tid < N) {
        int depth = -1;
        for (int w = 0; w < NW; ++w)
            depth += __popc(rows[tid * NW + w]);
        reinterpret_cast<int32_t *>(P.plan + P.lay.positions)[(size_t)b * N + tid] =
            on ? len + depth : -1;
    }
    if (tid == 0) {
        PlanSeq s;
        s.cache_len = bad ? 0 : len;
        s.n_nodes = bad ? 0 : nn;
        s.status = bad ? -1 : 0;
        s.pad = 0;
        reinterpret_cast<PlanSeq *>(P.plan + P.lay.seq)[b] = s;
        reinterpret_cast<int32_t *>(P.plan + P.lay.status)[b] = s.status;
    }
}

constexpr size_t plan_smem(int N) { return (size_t)N * ((N + 31) / 32) * 4; }
static_assert(plan_smem(SPEC_ATTN_MAX_NODES) <= 232448 - 1024, "227 KB per CTA");

std::atomic<bool> g_plan_attr[64];  // opted in, per device

// ----------------------------------------------------------------- commit

struct CommitParams {
    spec_tree_commit_args a;
    int run, runs;  // vectors that lie together (a head's, or all heads'), and runs in a row
};

constexpr int CTH = 256;

template <typename V>
__global__ void __launch_bounds__(CTH) commit_kernel(const __grid_constant__ CommitParams P)
{
    const spec_tree_commit_args &A = P.a;
    __shared__ int node[SPEC_ATTN_MAX_NODES], page[SPEC_ATTN_MAX_NODES];
    const int b = (int)blockIdx.x, tid = (int)threadIdx.x;
    const int warp = tid >> 5, lane = tid & 31;
    wait_previous_kernel();
    const int acc = __ldg(A.out_num_accepted + b), len = __ldg(A.cache_len + b);
    const long long cap = (long long)A.pages_per_seq * A.page_size;
    bool bad = acc < 0 || acc >= A.N || len < 0 || (long long)len + acc + 1 > cap;
    if (!bad)
        for (int i = tid; i <= acc; i += CTH) {
            const int n = (i == 0 || !A.out_nodes) ? i : A.out_nodes[(size_t)b * A.N + i - 1];
            const int pg = A.page_table
                ? A.page_table[(size_t)b * A.pages_per_seq + (len + i) / A.page_size] : b;
            bad |= n < 0 || n >= A.N || pg < 0 || pg >= A.num_pages;
            node[i] = n;
            page[i] = pg;
        }
    bad = __syncthreads_or(bad ? 1 : 0) != 0;
    if (tid == 0 && blockIdx.y == 0 && blockIdx.z == 0)
        A.out_len[b] = bad ? -1 : len + acc + 1;
    if (bad)
        return;
    const int jobs = 2 * (acc + 1) * P.runs;
    for (int layer = (int)blockIdx.y; layer < A.layers; layer += (int)gridDim.y) {
        for (int j = (int)blockIdx.z * (CTH / 32) + warp; j < jobs;
             j += (int)gridDim.z * (CTH / 32)) {
            const int half = j / P.runs, h = j - half * P.runs;
            const int side = half & 1, i = half >> 1;
            const int64_t *ss = side ? A.v_new_stride : A.k_new_stride;
            const int64_t *ds = side ? A.v_cache_stride : A.k_cache_stride;
            const V *src = reinterpret_cast<const V *>(
                static_cast<const uint8_t *>(side ? A.v_new : A.k_new) +
                (layer * ss[0] + b * ss[1] + node[i] * ss[2] + h * ss[3]) * A.elem_size);
            V *dst = reinterpret_cast<V *>(
                static_cast<uint8_t *>(side ? A.v_cache : A.k_cache) +
                (layer * ds[0] + page[i] * ds[1] + ((len + i) % A.page_size) * ds[2] + h * ds[3]) *
                    A.elem_size);
            for (int v = lane; v < P.run; v += 4 * 32) {
                V x[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (v + u * 32 < P.run)
                        x[u] = __ldg(src + v + u * 32);
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (v + u * 32 < P.run)
                        dst[v + u * 32] = x[u];
            }
        }
    }
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// whether the int32 arrays p [n] and q [m] have a word in common (a null one has none)
bool overlap(const int32_t *p, uint64_t n, const int32_t *q, uint64_t m)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && a < b + m * 4 && b < a + n * 4;
}

bool plan_sizes_ok(int32_t B, int32_t N)
{
    return B >= 0 && B <= 65535 && N >= 1 && N <= SPEC_ATTN_MAX_NODES;
}

}  // namespace

extern "C" {

size_t spec_tree_plan_size(int32_t B, int32_t N)
{
    return plan_sizes_ok(B, N) ? plan_layout(B, N).total : 0;
}

size_t spec_tree_plan_offset(int32_t B, int32_t N, int32_t part)
{
    if (!plan_sizes_ok(B, N))
        return 0;
    const PlanLayout l = plan_layout(B, N);
    switch (part) {
    case SPEC_PLAN_POSITIONS: return l.positions;
    case SPEC_PLAN_STATUS: return l.status;
    case SPEC_PLAN_MASK: return l.mask;
    default: return 0;
    }
}

int32_t spec_tree_plan(const int32_t *parent, const int32_t *n_nodes, const int32_t *cache_len,
                       const int32_t *page_table, int32_t B, int32_t N, int32_t page_size,
                       int32_t pages_per_seq, int32_t num_pages, void *plan, size_t plan_bytes,
                       void *stream)
{
    if (!plan_sizes_ok(B, N) || page_size < 1 || pages_per_seq < 1 || num_pages < 0 ||
        (long long)pages_per_seq * page_size > INT32_MAX - SPEC_ATTN_MAX_NODES)
        return SPEC_EINVAL;
    if (B == 0)
        return SPEC_OK;
    if (!parent || !n_nodes || !cache_len || !plan || !aligned(parent, 4) ||
        !aligned(n_nodes, 4) || !aligned(cache_len, 4) || !aligned(page_table, 4) ||
        !aligned(plan, 256) || (!page_table && (pages_per_seq != 1 || num_pages < B)))
        return SPEC_EINVAL;
    PlanParams P;
    P.lay = plan_layout(B, N);
    if (plan_bytes < P.lay.total)
        return SPEC_ENOSPACE;
    P.parent = parent;
    P.n_nodes = n_nodes;
    P.cache_len = cache_len;
    P.page_table = page_table;
    P.B = B;
    P.N = N;
    P.page_size = page_size;
    P.pages_per_seq = pages_per_seq;
    P.num_pages = num_pages;
    P.plan = static_cast<uint8_t *>(plan);
    const int NW = (N + 31) / 32;
    const int threads = NW < 4 ? 128 : NW * 32;
    // The limit belongs to the function, so one for every size: another thread's call may
    // come between a call's own and its launch.  (48 KB without it hold the static part too.)
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return SPEC_ECUDA;
    if (!g_plan_attr[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)plan_smem(SPEC_ATTN_MAX_NODES)) != cudaSuccess) {
            (void)cudaGetLastError();
            return SPEC_ECUDA;
        }
        g_plan_attr[dev].store(true, std::memory_order_release);
    }
    plan_kernel<<<(unsigned int)B + 1, threads, plan_smem(N),
                  reinterpret_cast<cudaStream_t>(stream)>>>(P);
    if (cudaPeekAtLastError() != cudaSuccess) {
        (void)cudaGetLastError();
        return SPEC_ECUDA;
    }
    return SPEC_OK;
}

int32_t spec_tree_commit(const spec_tree_commit_args *args, void *stream)
{
    if (!args)
        return SPEC_EINVAL;
    const spec_tree_commit_args &a = *args;
    if (a.layers < 0 || a.B < 0 || a.B > 65535 * 1024 || a.N < 1 || a.N > SPEC_ATTN_MAX_NODES ||
        a.Hkv < 1 || a.D < 1 || a.page_size < 1 || a.pages_per_seq < 1 || a.num_pages < 0 ||
        (long long)a.pages_per_seq * a.page_size > INT32_MAX - SPEC_ATTN_MAX_NODES ||
        (long long)a.Hkv * a.D > (1 << 24) || (a.elem_size != 2 && a.elem_size != 4))
        return SPEC_EINVAL;
    if (a.B == 0)
        return SPEC_OK;
    const size_t es = (size_t)a.elem_size;
    // CTAs read a sequence's inputs while one of them writes its length
    const uint64_t B = (uint64_t)a.B;
    if (overlap(a.out_len, B, a.cache_len, B) || overlap(a.out_len, B, a.out_num_accepted, B) ||
        overlap(a.out_len, B, a.out_nodes, B * a.N) ||
        overlap(a.out_len, B, a.page_table, B * a.pages_per_seq))
        return SPEC_EINVAL;
    if (!a.cache_len || !a.out_num_accepted || !a.out_len ||
        !aligned(a.cache_len, 4) || !aligned(a.out_num_accepted, 4) || !aligned(a.out_len, 4) ||
        !aligned(a.out_nodes, 4) || !aligned(a.page_table, 4) ||
        (!a.page_table && (a.pages_per_seq != 1 || a.num_pages < a.B)))
        return SPEC_EINVAL;
    if (a.layers > 0 && (!a.k_new || !a.v_new || !a.k_cache || !a.v_cache ||
                         !aligned(a.k_new, es) || !aligned(a.v_new, es) ||
                         !aligned(a.k_cache, es) || !aligned(a.v_cache, es)))
        return SPEC_EINVAL;
    // the widest vector that every address allows
    uint64_t bits = reinterpret_cast<uintptr_t>(a.k_new) | reinterpret_cast<uintptr_t>(a.v_new) |
                    reinterpret_cast<uintptr_t>(a.k_cache) |
                    reinterpret_cast<uintptr_t>(a.v_cache) | (uint64_t)a.D * es;
    for (int i = 0; i < 4; ++i)
        bits |= (uint64_t)(a.k_new_stride[i] | a.v_new_stride[i] | a.k_cache_stride[i] |
                           a.v_cache_stride[i]) * es;
    CommitParams P;
    P.a = a;
    const size_t vec = (bits & 15) == 0 ? 16 : (bits & 3) == 0 ? 4 : 2;
    // heads that lie one after the other everywhere are copied as one run
    const bool flat = a.k_new_stride[3] == a.D && a.v_new_stride[3] == a.D &&
                      a.k_cache_stride[3] == a.D && a.v_cache_stride[3] == a.D;
    P.runs = flat ? 1 : a.Hkv;
    if (2ll * a.N * P.runs > INT_MAX / 2)
        return SPEC_EINVAL;  // a sequence's runs are counted in 32 bits
    P.run = (int)((size_t)a.D * es / vec) * (flat ? a.Hkv : 1);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const unsigned int gy = a.layers < 1 ? 1u : a.layers > 65535 ? 65535u : (unsigned int)a.layers;
    // few sequences and layers: several CTAs share a sequence's rows
    unsigned int gz = 1;
    while ((size_t)a.B * gy * gz < 304 && gz < (unsigned int)a.N && gz < 64)
        gz *= 2;
    const dim3 grid((unsigned int)a.B, gy, gz);
    if (vec == 16)
        commit_kernel<uint4><<<grid, CTH, 0, st>>>(P);
    else if (vec == 4)
        commit_kernel<uint32_t><<<grid, CTH, 0, st>>>(P);
    else
        commit_kernel<unsigned short><<<grid, CTH, 0, st>>>(P);
    if (cudaPeekAtLastError() != cudaSuccess) {
        (void)cudaGetLastError();
        return SPEC_ECUDA;
    }
    return SPEC_OK;
}

}  // extern "C"
