// spec_append.cu -- the plan of a step over chunks of new tokens, and the append of their keys
// and values to the cache (include/spec_chunk.h).
//
// Plan.  A CTA per sequence checks its lengths and pages; one more lists the row groups of all
// sequences (the tokens that a CTA of the attention works on at a time) with the key tiles that
// they see and those tiles' running sum, by which the attention deals out its work.
// Bound by latency: loads of the lengths, two block sums, one store per group.  4 us for 1 sequence or 8.
//
// Append.  A copy of every row's Hkv * D elements to its position, in the widest vectors that
// every address allows.  A warp takes whole runs of a row (all heads, where they lie together),
// looks up its sequence (a search of row_start) and page once per run, four vectors of a lane in flight.
// A sequence whose new pages are bad is left alone, so every CTA first checks the pages of the
// sequences that its rows belong to.  Bound by bytes where there are many: 6400 rows of 8 x 128 bf16,
// 52 MB read and written, 12.3 us cold, 4.3 TB/s; 40 rows 5.5 us, latency.
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "spec_chunk.h"
#include "spec_verify.h"
#include "chunk_plan.cuh"
#include "device_common.cuh"

namespace {

using namespace spec_dev;
using namespace spec_attn;

// ------------------------------------------------------------------- plan

constexpr int PTH = 256;

struct PlanParams {
    const int32_t *row_start, *kv_len, *page_table;
    int32_t B, rows, page_size, pages_per_seq, num_pages;
    uint8_t *plan;
    ChunkLayout lay;
};

// Whether row_start does not decrease and stays in 0 .. rows; the whole CTA asks.
__device__ bool rows_ok(const int32_t *start, int B, int rows)
{
    bool bad = false;
    for (int i = (int)threadIdx.x; i <= B; i += (int)blockDim.x) {
        const int at = start[i];
        bad |= at < 0 || at > rows || (i < B && start[i + 1] < at);
    }
    return __syncthreads_or(bad ? 1 : 0) == 0;
}

// Inclusive sums of a and c over the CTA's threads, and their totals.
__device__ void block_sums(long long &a, long long &c, long long &all_a, long long &all_c)
{
    __shared__ long long part[2][PTH / 32];
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
    for (int d = 1; d < 32; d <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, a, d), y = __shfl_up_sync(0xffffffffu, c, d);
        if (lane >= d) {
            a += x;
            c += y;
        }
    }
    if (lane == 31) {
        part[0][warp] = a;
        part[1][warp] = c;
    }
    __syncthreads();
    all_a = all_c = 0;
    for (int w = 0; w < PTH / 32; ++w) {
        if (w == warp) {
            a += all_a;
            c += all_c;
        }
        all_a += part[0][w];
        all_c += part[1][w];
    }
    __syncthreads();
}

// The list of row groups, in the order of the sequences and their tokens: thread t of a round
// has group g0 + t, whose sequence it finds in the groups before each (at most PTH
// sequences at a time lie in shared memory).
__device__ void list_groups(const PlanParams &P)
{
    __shared__ int first[PTH + 1];  // groups before a sequence, in this round of sequences
    ChunkGroup *groups = reinterpret_cast<ChunkGroup *>(P.plan + P.lay.group);
    long long *cum = reinterpret_cast<long long *>(P.plan + P.lay.cum);
    const int tid = (int)threadIdx.x, T = P.lay.tokens;
    const bool ok = rows_ok(P.row_start, P.B, P.rows);
    const int B = ok ? P.B : 1;  // otherwise one sequence of all rows, in error
    long long done = 0, tiles = 0;
    for (int b0 = 0; b0 < B; b0 += PTH) {
        const int b = b0 + tid;
        const int n = b < B ? (ok ? P.row_start[b + 1] - P.row_start[b] : P.rows) : 0;
        long long mine = (n + T - 1) / T, zero = 0, all, none;
        const long long own = mine;
        block_sums(mine, zero, all, none);
        first[tid] = (int)(mine - own);
        if (tid == 0)
            first[PTH] = (int)all;
        __syncthreads();
        for (int g0 = 0; g0 < (int)all; g0 += PTH) {
            const int g = g0 + tid;
            ChunkGroup x = {};
            if (g < (int)all) {
                int lo = 0, hi = PTH;  // the last sequence with first <= g that has groups
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (first[mid] <= g)
                        lo = mid;
                    else
                        hi = mid;
                }
                const int start = ok ? P.row_start[b0 + lo] : 0;
                const int count = ok ? P.row_start[b0 + lo + 1] - start : P.rows;
                const int len = ok ? P.kv_len[b0 + lo] : -1, tok0 = (g - first[lo]) * T;
                x.b = b0 + lo;
                x.row0 = start + tok0;
                x.ntok = min(T, count - tok0);
                x.bad = len < count || (long long)len > (long long)P.pages_per_seq * P.page_size;
                x.pos0 = x.bad ? 0 : len - count + tok0;
                x.tiles = x.bad ? 1 : (x.pos0 + x.ntok + KT - 1) / KT;
            }
            long long t = x.tiles, z = 0, round, nothing;
            block_sums(t, z, round, nothing);
            if (g < (int)all) {
                groups[done + g] = x;
                cum[done + g + 1] = tiles + t;
            }
            tiles += round;
        }
        done += all;
        __syncthreads();
    }
    if (tid == 0) {
        cum[0] = 0;
        ChunkHeader *h = reinterpret_cast<ChunkHeader *>(P.plan);
        h->status = SPEC_DEV_OK;
        h->groups = (int)done;
        h->tiles = tiles;
    }
}

__global__ void __launch_bounds__(PTH) chunk_plan_kernel(const PlanParams P)
{
    allow_next_kernel();
    wait_previous_kernel();
    const int b = (int)blockIdx.x;
    if (b == P.B) {
        list_groups(P);
        return;
    }
    bool bad = !rows_ok(P.row_start, P.B, P.rows);
    if (!bad) {
        const int n = P.row_start[b + 1] - P.row_start[b], len = P.kv_len[b];
        bad = len < n || (long long)len > (long long)P.pages_per_seq * P.page_size;
        if (!bad && n > 0 && P.page_table) {
            const int used = (int)(((long long)len + P.page_size - 1) / P.page_size);
            bool out = false;
            for (int i = (int)threadIdx.x; i < used; i += PTH) {
                const int pg = P.page_table[(size_t)b * P.pages_per_seq + i];
                out |= pg < 0 || pg >= P.num_pages;
            }
            bad = __syncthreads_or(out ? 1 : 0) != 0;
        }
    }
    if (threadIdx.x == 0)
        reinterpret_cast<int32_t *>(P.plan + P.lay.status)[b] = bad ? -1 : 0;
}

// ----------------------------------------------------------------- append

struct AppendParams {
    spec_chunk_append_args a;
    int run, runs;     // vectors that lie together (a head's, or all heads'), and runs in a row
    int rows_per_cta;
};

constexpr int ATH = 256;

template <typename V>
__global__ void __launch_bounds__(ATH) append_kernel(const __grid_constant__ AppendParams P)
{
    const spec_chunk_append_args &A = P.a;
    const int tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31;
    allow_next_kernel();
    wait_previous_kernel();
    const bool ok = rows_ok(A.row_start, A.B, A.rows);
    const long long cap = (long long)A.pages_per_seq * A.page_size;
    // the pages of sequence b's new positions; the whole CTA asks
    auto seq_ok = [&](int b, int start, int n, int len) -> bool {
        if (len < 0 || (long long)len + n > cap)
            return false;
        bool out = false;
        if (A.page_table && n > 0) {
            const int e0 = len / A.page_size, e1 = (len + n - 1) / A.page_size;
            for (int e = e0 + tid; e <= e1; e += ATH) {
                const int pg = A.page_table[(size_t)b * A.pages_per_seq + e];
                out |= pg < 0 || pg >= A.num_pages;
            }
        }
        return __syncthreads_or(out ? 1 : 0) == 0;
    };
    // the lengths, sequences shared out among the CTAs of the first layer
    if (blockIdx.y == 0)
        for (int b = (int)blockIdx.x; b < A.B; b += (int)gridDim.x) {
            const int start = A.row_start[b], n = ok ? A.row_start[b + 1] - start : 0;
            const int len = A.cache_len[b];
            const bool fine = ok && seq_ok(b, start, n, len);
            if (tid == 0)
                A.out_len[b] = fine ? len + n : -1;
        }
    if (!ok)
        return;
    int r = max((int)blockIdx.x * P.rows_per_cta, A.row_start[0]);
    const int end = min((int)min((long long)(blockIdx.x + 1) * P.rows_per_cta, (long long)A.rows),
                        A.row_start[A.B]);
    if (r >= end)
        return;
    int b = 0, hi = A.B;  // the last sequence with row_start <= r: its rows hold r
    while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if (A.row_start[mid] <= r)
            b = mid;
        else
            hi = mid;
    }
    for (; r < end; ++b) {
        const int start = A.row_start[b], stop = A.row_start[b + 1], len = A.cache_len[b];
        const int to = min(end, stop);
        if (to <= r)
            continue;
        if (seq_ok(b, start, stop - start, len)) {
            const int jobs = 2 * (to - r) * P.runs;
            for (int layer = (int)blockIdx.y; layer < A.layers; layer += (int)gridDim.y)
                for (int j = warp; j < jobs; j += ATH / 32) {
                    const int half = j / P.runs, h = j - half * P.runs;
                    const int side = half & 1, row = r + (half >> 1), pos = len + row - start;
                    const int e = pos / A.page_size, slot = pos - e * A.page_size;
                    const int page = A.page_table
                        ? __ldg(A.page_table + (size_t)b * A.pages_per_seq + e) : b;
                    const int64_t *ss = side ? A.v_new_stride : A.k_new_stride;
                    const int64_t *ds = side ? A.v_cache_stride : A.k_cache_stride;
                    const V *src = reinterpret_cast<const V *>(
                        static_cast<const uint8_t *>(side ? A.v_new : A.k_new) +
                        (layer * ss[0] + row * ss[1] + h * ss[2]) * A.elem_size);
                    V *dst = reinterpret_cast<V *>(
                        static_cast<uint8_t *>(side ? A.v_cache : A.k_cache) +
                        (layer * ds[0] + page * ds[1] + slot * ds[2] + h * ds[3]) * A.elem_size);
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
        r = to;
    }
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// whether the int32 arrays p [n] and q [m] have a word in common (a null one has none)
bool overlap(const int32_t *p, uint64_t n, const int32_t *q, uint64_t m)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && a < b + m * 4 && b < a + n * 4;
}

bool sizes_ok(int32_t B, int32_t rows, int32_t group)
{
    return B >= 0 && B <= 65535 && rows >= 0 && rows <= SPEC_CHUNK_MAX_ROWS && group >= 1 &&
           group <= 128;
}

template <typename K, typename P>
int launch(K kernel, dim3 grid, int threads, const P &params, void *stream)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned int)threads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, params) != cudaSuccess) {
        (void)cudaGetLastError();
        return SPEC_ECUDA;
    }
    return SPEC_OK;
}

}  // namespace

extern "C" {

size_t spec_chunk_plan_size(int32_t B, int32_t rows, int32_t group)
{
    return sizes_ok(B, rows, group) ? chunk_layout(B, rows, group).total : 0;
}

size_t spec_chunk_plan_status(int32_t B, int32_t rows, int32_t group)
{
    return sizes_ok(B, rows, group) ? chunk_layout(B, rows, group).status : 0;
}

int32_t spec_chunk_plan(const int32_t *row_start, const int32_t *kv_len, const int32_t *page_table,
                        int32_t B, int32_t rows, int32_t group, int32_t page_size,
                        int32_t pages_per_seq, int32_t num_pages, void *plan, size_t plan_bytes,
                        void *stream)
{
    if (!sizes_ok(B, rows, group) || page_size < 1 || pages_per_seq < 1 || num_pages < 0 ||
        (long long)pages_per_seq * page_size > INT32_MAX - SPEC_CHUNK_MAX_ROWS)
        return SPEC_EINVAL;
    if (B == 0)
        return SPEC_OK;
    if (!row_start || !kv_len || !plan || !aligned(row_start, 4) || !aligned(kv_len, 4) ||
        !aligned(page_table, 4) || !aligned(plan, 256) ||
        (!page_table && (pages_per_seq != 1 || num_pages < B)))
        return SPEC_EINVAL;
    PlanParams P;
    P.lay = chunk_layout(B, rows, group);
    if (plan_bytes < P.lay.total)
        return SPEC_ENOSPACE;
    P.row_start = row_start;
    P.kv_len = kv_len;
    P.page_table = page_table;
    P.B = B;
    P.rows = rows;
    P.page_size = page_size;
    P.pages_per_seq = pages_per_seq;
    P.num_pages = num_pages;
    P.plan = static_cast<uint8_t *>(plan);
    return launch(chunk_plan_kernel, dim3((unsigned int)B + 1), PTH, P, stream);
}

int32_t spec_chunk_append(const spec_chunk_append_args *args, void *stream)
{
    if (!args)
        return SPEC_EINVAL;
    const spec_chunk_append_args &a = *args;
    if (a.layers < 0 || !sizes_ok(a.B, a.rows, 1) || a.Hkv < 1 || a.D < 1 || a.page_size < 1 ||
        a.pages_per_seq < 1 || a.num_pages < 0 ||
        (long long)a.pages_per_seq * a.page_size > INT32_MAX - SPEC_CHUNK_MAX_ROWS ||
        (long long)a.Hkv * a.D > (1 << 24) || (a.elem_size != 2 && a.elem_size != 4))
        return SPEC_EINVAL;
    if (a.B == 0)
        return SPEC_OK;
    const size_t es = (size_t)a.elem_size;
    const uint64_t B = (uint64_t)a.B;
    // CTAs read a sequence's inputs while one of them writes its length
    if (!a.row_start || !a.cache_len || !a.out_len || !aligned(a.row_start, 4) ||
        !aligned(a.cache_len, 4) || !aligned(a.out_len, 4) || !aligned(a.page_table, 4) ||
        (!a.page_table && (a.pages_per_seq != 1 || a.num_pages < a.B)) ||
        overlap(a.out_len, B, a.row_start, B + 1) || overlap(a.out_len, B, a.cache_len, B) ||
        overlap(a.out_len, B, a.page_table, B * a.pages_per_seq))
        return SPEC_EINVAL;
    if (a.layers > 0 && a.rows > 0 &&
        (!a.k_new || !a.v_new || !a.k_cache || !a.v_cache || !aligned(a.k_new, es) ||
         !aligned(a.v_new, es) || !aligned(a.k_cache, es) || !aligned(a.v_cache, es)))
        return SPEC_EINVAL;
    // the widest vector that every address allows
    uint64_t bits = reinterpret_cast<uintptr_t>(a.k_new) | reinterpret_cast<uintptr_t>(a.v_new) |
                    reinterpret_cast<uintptr_t>(a.k_cache) |
                    reinterpret_cast<uintptr_t>(a.v_cache) | (uint64_t)a.D * es;
    for (int i = 0; i < 3; ++i)
        bits |= (uint64_t)(a.k_new_stride[i] | a.v_new_stride[i]) * es;
    for (int i = 0; i < 4; ++i)
        bits |= (uint64_t)(a.k_cache_stride[i] | a.v_cache_stride[i]) * es;
    AppendParams P;
    P.a = a;
    const size_t vec = (bits & 15) == 0 ? 16 : (bits & 3) == 0 ? 4 : 2;
    // heads that lie one after the other everywhere are copied as one run
    const bool flat = a.Hkv == 1 ||
                      (a.k_new_stride[2] == a.D && a.v_new_stride[2] == a.D &&
                       a.k_cache_stride[3] == a.D && a.v_cache_stride[3] == a.D);
    P.runs = flat ? 1 : a.Hkv;
    P.run = (int)((size_t)a.D * es / vec) * (flat ? a.Hkv : 1);
    const unsigned int gy = a.layers < 1 ? 1u : a.layers > 65535 ? 65535u : (unsigned int)a.layers;
    // a warp's row or two at a time, more where that makes more than 8 CTAs per SM
    long long per = 4;
    while (((long long)a.rows + per - 1) / per * gy > 1216 && per < 512)
        per *= 2;
    if (P.runs > 1 << 20)
        return SPEC_EINVAL;  // a CTA's runs, of 512 rows at most, are counted in 32 bits
    P.rows_per_cta = (int)per;
    long long ctas = ((long long)a.rows + per - 1) / per;
    const dim3 grid((unsigned int)(ctas < 1 ? 1 : ctas), gy);
    if (vec == 16)
        return launch(append_kernel<uint4>, grid, ATH, P, stream);
    if (vec == 4)
        return launch(append_kernel<uint32_t>, grid, ATH, P, stream);
    return launch(append_kernel<unsigned short>, grid, ATH, P, stream);
}

}  // extern "C"
