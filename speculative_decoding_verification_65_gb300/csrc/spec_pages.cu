// spec_pages.cu -- the pages of a cache: tables forked, pages taken, shared, freed and copied, and
// the pages in use moved to the front of the pool (include/spec_pages.h).
//
// The only state is a count of references per page, so the j-th free page is found by counting
// zeros: a first kernel counts them per block of 4096 pages and lists each block's in order; the
// second adds the blocks up (in every CTA: a few numbers) and looks up the j-th by its block.  In
// fork the first kernel works out beside it, a warp per new row, how many pages the row takes; the
// second sums those of the rows before.  Both are bound by the chain of their loads, not by bytes: 6.5 and
// 9.9 us for 512 rows of 100 pages, each cold.  Compaction's three take 4.2, 9.9 and 4.8 us for a pool of 22
// thousand pages.  Counts change by atomic additions of whole numbers, whose order does not matter.
//
// The copy moves whole rows of slots, 256 vectors per warp at a time, in the widest vectors that the
// addresses allow.  A warp looks at 32 entries of the list at once and works on those that copy
// something.  Bound by bytes: 2.2 GB of moved pages read and written in 326 us, 6.7 TB/s, the rate
// of a plain copy.
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include <algorithm>

#include "spec_pages.h"
#include "spec_verify.h"
#include "device_common.cuh"

namespace {

using namespace spec_dev;

constexpr int TH = 256;
constexpr int WARPS = TH / 32;
constexpr int PB = 4096;           // pages of a block
constexpr int MAX_BLOCKS = SPEC_PAGES_MAX / PB;

// One CTA does all where it has up to SMALL_ROWS rows or SMALL_ENTRIES entries of a table, and one block
// of pages: a launch costs the host 2.5 us.  (4 beams of 600 tokens forked, with their copies: 8.3 us of
// the GPU's time and 10 us of the host's, by two kernels 8.7 and 13; 512 pages compacted and
// copied: 22 and 10, by three kernels 25 and 16.)
constexpr int SMALL_ROWS = 16;
constexpr uint64_t SMALL_ENTRIES = 4096;

struct Work {
    int *free_of;    // [blocks] free pages of a block
    int *free_list;  // [num_pages] a block's free pages in order, from block * PB on
    int *need;       // [rows] pages that a new row takes
    int *state;      // [rows] what a new row is: an error, empty, a parent's first child, another
    int *holes;      // [num_pages] compaction: free pages below the number in use, in order
    int *movers;     // [num_pages] pages in use from it on, in order
    int *rank;       // [num_pages] a mover's place among them
    int *moves;      // [2] their number, and that of the pages in use
};

// A word of the work that an earlier kernel wrote, or (SMALL) this CTA, whose work lies in shared
// memory.
template <bool SMALL>
__device__ __forceinline__ int got(const int *p)
{
    return SMALL ? *p : __ldcg(p);
}

enum { ROW_ERROR = -1, ROW_EMPTY = 0, ROW_FIRST = 1, ROW_OTHER = 2 };

// A block of pages: free ones (count 0, or for USED not above 0) counted, and for a fork listed in
// order and the counts copied.  The whole CTA.
template <bool USED>
__device__ void list_free(const int32_t *ref, int32_t *ref_out, int num_pages, int block,
                          const Work &W)
{
    __shared__ int part[WARPS];
    constexpr int EACH = PB / TH;
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
    const int base = block * PB + warp * (PB / WARPS);
    uint32_t zero[EACH];
    int mine = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int p = base + i * 32 + lane;
        int c = 1;
        if (p < num_pages) {
            c = __ldg(ref + p);
            if (!USED)
                ref_out[p] = c;
        }
        zero[i] = __ballot_sync(0xffffffffu, USED ? c <= 0 : c == 0);
        mine += __popc(zero[i]);
    }
    if (lane == 0)
        part[warp] = mine;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < WARPS; ++w) {
        before += w < warp ? part[w] : 0;
        all += part[w];
    }
    if (threadIdx.x == 0)
        W.free_of[block] = all;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        if (!USED && ((zero[i] >> lane) & 1u))
            W.free_list[block * PB + before + __popc(zero[i] & ((1u << lane) - 1u))] =
                base + i * 32 + lane;
        before += __popc(zero[i]);
    }
}

// Free pages before each block, to smem[0 .. blocks]; the whole CTA.
template <bool SMALL>
__device__ void sum_blocks(const int *free_of, int blocks, int *sums)
{
    __shared__ int part[WARPS];
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int base = 0;
    for (int i0 = 0; i0 < blocks; i0 += TH) {
        const int own = i0 + tid < blocks ? got<SMALL>(free_of + i0 + tid) : 0;
        int v = own;
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d)
                v += o;
        }
        if (lane == 31)
            part[warp] = v;
        __syncthreads();
        int before = base;
        for (int w = 0; w < WARPS; ++w) {
            before += w < warp ? part[w] : 0;
            base += part[w];
        }
        if (i0 + tid < blocks)
            sums[i0 + tid] = before + v - own;
        __syncthreads();
    }
    if (tid == 0)
        sums[blocks] = base;
    __syncthreads();
}

// ------------------------------------------------------------------- fork

struct ForkParams {
    spec_pages_fork_args a;
    Work w;
    int blocks;
};

// An old row, looked at by a warp: its length and pages held, or an error.
struct Old {
    int length, held;
    bool ok;
};

constexpr int AHEAD = 4;  // 32 entries each that a warp has in flight

__device__ __forceinline__ Old old_row(const spec_pages_fork_args &A, int o)
{
    const int lane = (int)threadIdx.x & 31, M = A.pages_per_seq;
    const int32_t *row = A.table_in + (size_t)o * M;
    Old r;
    r.length = __ldg(A.length_in + o);
    r.held = M;
    bool bad = false;
    for (int i0 = 0; i0 < M && r.held == M; i0 += 32 * AHEAD) {
        int e[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            e[u] = i0 + u * 32 + lane < M ? __ldg(row + i0 + u * 32 + lane) : -1;
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int at = i0 + u * 32;
            const uint32_t none = __ballot_sync(0xffffffffu, e[u] < 0);
            if (at < r.held && none)
                r.held = min(at + __ffs((int)none) - 1, M);
            // (entries behind the first -1 are not looked at)
            bad |= e[u] >= A.num_pages && at + lane < r.held;
        }
    }
    r.ok = !__any_sync(0xffffffffu, bad) && r.length >= 0 &&
           (long long)r.length <= (long long)r.held * A.page_size;
    return r;
}

// Pages that a child of this length with this reserve has to hold; -1 where the row has no room.
__device__ __forceinline__ int pages_for(const spec_pages_fork_args &A, int length, int reserve)
{
    const long long pages = ((long long)length + reserve + A.page_size - 1) / A.page_size;
    return reserve < 0 || pages > A.pages_per_seq ? -1 : (int)pages;
}

// Whether one of new rows 0 .. end - 1 is a child of old row o (whose length is given); a warp asks.
__device__ bool has_child(const spec_pages_fork_args &A, int o, int length, int end)
{
    const int lane = (int)threadIdx.x & 31;
    for (int i0 = 0; i0 < end; i0 += 32 * AHEAD) {
        int parent[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int i = i0 + u * 32 + lane;
            parent[u] = i < end ? __ldg(A.parent + i) : -1;
        }
        bool hit = false;
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (parent[u] == o)
                hit |= pages_for(A, length, A.reserve ? __ldg(A.reserve + i0 + u * 32 + lane) : 0) >= 0;
        if (__any_sync(0xffffffffu, hit))
            return true;
    }
    return false;
}

// What a new row is, and the pages that it takes; a warp asks.
__device__ void count_row(const ForkParams &P, int r)
{
    const spec_pages_fork_args &A = P.a;
    const int lane = (int)threadIdx.x & 31;
    if (r >= A.rows_out)
        return;
    const int parent = __ldg(A.parent + r);
    int state = ROW_ERROR, need = 0;
    if (parent == -1) {
        const int pages = pages_for(A, 0, A.reserve ? __ldg(A.reserve + r) : 0);
        if (pages >= 0) {
            state = ROW_EMPTY;
            need = pages;
        }
    } else if (parent >= 0 && parent < A.rows_in) {
        const Old o = old_row(A, parent);
        const int pages = o.ok
            ? pages_for(A, o.length, A.reserve ? __ldg(A.reserve + r) : 0) : -1;
        if (pages >= 0) {
            const int whole = o.length / A.page_size;
            if (has_child(A, parent, o.length, r)) {
                state = ROW_OTHER;
                need = max(0, pages - whole);
            } else {
                state = ROW_FIRST;
                for (int i = whole + lane; i < pages; i += 32) {
                    bool keep = i < o.held;
                    if (keep)
                        keep = __ldg(A.ref_in + __ldg(A.table_in +
                                                     (size_t)parent * A.pages_per_seq + i)) == 1;
                    need += keep ? 0 : 1;
                }
                need = __reduce_add_sync(0xffffffffu, need);
            }
        }
    }
    if (lane == 0) {
        P.w.state[r] = state;
        P.w.need[r] = need;
    }
}

extern __shared__ int sums[];  // free pages before each block

// New rows r0 .. r0 + 7 and old rows of these numbers, by a whole CTA.
template <bool SMALL>
__device__ void write_rows(const ForkParams &P, int r0)
{
    __shared__ long long part[WARPS][2];
    __shared__ int own[WARPS];      // pages that this CTA's rows take
    const spec_pages_fork_args &A = P.a;
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int M = A.pages_per_seq, r = r0 + warp;
    // what does not hang on the sums is looked at before they are there
    int state = ROW_ERROR, parent = -1, reserve = 0;
    if (r < A.rows_out) {
        state = got<SMALL>(P.w.state + r);
        parent = __ldg(A.parent + r);
        reserve = A.reserve ? __ldg(A.reserve + r) : 0;
    }
    Old o = {0, 0, true};
    if (state == ROW_FIRST || state == ROW_OTHER)
        o = old_row(A, parent);
    Old given_up = {0, 0, false};  // an old row that nobody takes over
    if (r < A.rows_in) {
        given_up = old_row(A, r);
        given_up.ok = given_up.ok && !has_child(A, r, given_up.length, A.rows_out);
    }
    // pages that the rows before this CTA's take, and all rows
    long long before = 0, all = 0;
    if (tid < WARPS)
        own[tid] = r0 + tid < A.rows_out ? got<SMALL>(P.w.need + r0 + tid) : 0;
    for (int i = tid; i < A.rows_out; i += TH) {
        const int n = got<SMALL>(P.w.need + i);
        all += n;
        before += i < r0 ? n : 0;
    }
    for (int d = 16; d; d >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, d);
        all += __shfl_xor_sync(0xffffffffu, all, d);
    }
    if (lane == 0) {
        part[warp][0] = before;
        part[warp][1] = all;
    }
    sum_blocks<SMALL>(P.w.free_of, P.blocks, sums);  // (and all have written theirs)
    before = all = 0;
    for (int w = 0; w < WARPS; ++w) {
        before += part[w][0];
        all += part[w][1];
    }
    const bool enough = all <= sums[P.blocks];
    if (r < A.rows_out) {
        // -------------------------------------------------- a new row
        if (!enough)
            state = ROW_ERROR;
        int32_t *row = A.table_out + (size_t)r * M;
        int src = -1, dst = -1, slots = 0, length = -1;
        if (state != ROW_ERROR) {
            const int pages = pages_for(A, o.length, reserve);
            const int whole = o.length / A.page_size, tail = o.length - whole * A.page_size;
            const int32_t *old = A.table_in + (size_t)max(parent, 0) * M;
            length = o.length;
            long long next = before;
            for (int w = 0; w < warp; ++w)
                next += own[w];
            for (int i0 = 0; i0 < M; i0 += 32) {
                const int i = i0 + lane;
                const int e = i < o.held ? __ldg(old + i) : -1;
                bool keep = e >= 0 && i < pages;
                if (i >= whole && keep)
                    keep = state == ROW_FIRST && __ldg(A.ref_in + e) == 1;
                const bool fresh = i >= whole && i < pages && !keep;
                const uint32_t takes = __ballot_sync(0xffffffffu, fresh);
                int page = keep ? e : -1;
                if (fresh) {
                    const int j = (int)(next + __popc(takes & ((1u << lane) - 1u)));
                    int lo = 0, hi = P.blocks;  // the last block with sums <= j
                    while (hi - lo > 1) {
                        const int mid = (lo + hi) / 2;
                        if (sums[mid] <= j)
                            lo = mid;
                        else
                            hi = mid;
                    }
                    page = got<SMALL>(P.w.free_list + lo * PB + (j - sums[lo]));
                }
                next += __popc(takes);
                if (i < M)
                    row[i] = page;
                // the first child has taken over its parent's references
                if (fresh || (keep && state == ROW_OTHER))
                    atomicAdd(A.ref_out + page, 1);
                if (state == ROW_FIRST && e >= 0 && !keep)
                    atomicAdd(A.ref_out + e, -1);
                if (i == whole && tail > 0 && fresh) {
                    src = e;
                    dst = page;
                    slots = tail;
                }
            }
            const int at = whole & 31;
            src = __shfl_sync(0xffffffffu, src, at);
            dst = __shfl_sync(0xffffffffu, dst, at);
            slots = __shfl_sync(0xffffffffu, slots, at);
        } else {
            for (int i = lane; i < M; i += 32)
                row[i] = -1;
        }
        if (lane == 0) {
            A.length_out[r] = length;
            A.copies[r] = src;
            A.copies[(size_t)A.rows_out + r] = dst;
            A.copies[2 * (size_t)A.rows_out + r] = slots;
        }
    }
    if (given_up.ok && enough)
        for (int i = lane; i < given_up.held; i += 32)
            atomicAdd(A.ref_out + __ldg(A.table_in + (size_t)r * M + i), -1);
}

__global__ void __launch_bounds__(TH) fork_count_kernel(const __grid_constant__ ForkParams P)
{
    allow_next_kernel();
    wait_previous_kernel();
    const int x = (int)blockIdx.x - P.blocks;
    if (x < 0)
        list_free<false>(P.a.ref_in, P.a.ref_out, P.a.num_pages, (int)blockIdx.x, P.w);
    else
        count_row(P, x * WARPS + ((int)threadIdx.x >> 5));
}

__global__ void __launch_bounds__(TH) fork_rows_kernel(const __grid_constant__ ForkParams P)
{
    allow_next_kernel();
    wait_previous_kernel();
    write_rows<false>(P, (int)blockIdx.x * WARPS);
}

// Both by one CTA, where that has little more to do than any CTA: one launch for two, and what the first
// part leaves for the second in shared memory.
__global__ void __launch_bounds__(TH) fork_small_kernel(const __grid_constant__ ForkParams given)
{
    __shared__ int free_of, free_list[PB], need[SMALL_ROWS], state[SMALL_ROWS];
    __shared__ ForkParams P;
    if (threadIdx.x == 0) {
        P = given;
        P.w.free_of = &free_of;
        P.w.free_list = free_list;
        P.w.need = need;
        P.w.state = state;
    }
    allow_next_kernel();
    wait_previous_kernel();
    __syncthreads();
    if (P.blocks > 0)
        list_free<false>(P.a.ref_in, P.a.ref_out, P.a.num_pages, 0, P.w);
    for (int r = (int)threadIdx.x >> 5; r < P.a.rows_out; r += WARPS)
        count_row(P, r);
    __syncthreads();
    for (int r0 = 0; r0 < max(P.a.rows_in, P.a.rows_out); r0 += WARPS) {
        write_rows<true>(P, r0);
        __syncthreads();
    }
}

// ---------------------------------------------------------------- compact

struct CompactParams {
    spec_pages_compact_args a;
    Work w;
    int blocks;
};

// A block's holes below the number in use and its pages in use from it on, with their places; the
// whole CTA.
template <bool SMALL>
__device__ void list_moves(const CompactParams &P, int block)
{
    __shared__ int part[WARPS];
    const spec_pages_compact_args &A = P.a;
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    sum_blocks<SMALL>(P.w.free_of, P.blocks, sums);
    const int used = A.num_pages - sums[P.blocks];
    // free pages below `used`: those of the whole blocks before it, and of its own up to it
    const int bu = min(used / PB, P.blocks - 1);
    int some = 0;
    for (int p = bu * PB + tid; p < used; p += TH)
        some += __ldg(A.ref_in + p) <= 0 ? 1 : 0;
    some = __reduce_add_sync(0xffffffffu, some);
    if (lane == 0)
        part[warp] = some;
    __syncthreads();
    int holes = sums[bu];
    for (int w = 0; w < WARPS; ++w)
        holes += part[w];
    __syncthreads();
    if (block == 0 && tid == 0) {
        P.w.moves[0] = holes;
        P.w.moves[1] = used;
        A.used[0] = used;
    }
    constexpr int EACH = PB / TH;
    const int base = block * PB + warp * (PB / WARPS);
    uint32_t zero[EACH];
    int count[EACH], mine = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int p = base + i * 32 + lane;
        count[i] = p < A.num_pages ? __ldg(A.ref_in + p) : 1;
        zero[i] = __ballot_sync(0xffffffffu, count[i] <= 0);
        mine += __popc(zero[i]);
    }
    if (lane == 0)
        part[warp] = mine;
    __syncthreads();
    int before = sums[block];  // free pages before this one
    for (int w = 0; w < warp; ++w)
        before += part[w];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int p = base + i * 32 + lane;
        const int z = before + __popc(zero[i] & ((1u << lane) - 1u));
        const bool is_free = (zero[i] >> lane) & 1u;
        before += __popc(zero[i]);
        if (p >= A.num_pages)
            continue;
        if (p < used) {
            if (is_free)
                P.w.holes[z] = p;
            else
                A.ref_out[p] = count[i];
        } else {
            A.ref_out[p] = 0;
            if (!is_free) {
                const int k = (p - z) - (used - holes);  // pages in use between `used` and p
                P.w.movers[k] = p;
                P.w.rank[p] = k;
            }
        }
    }
}

// The moves and the table after them, by all CTAs.
template <bool SMALL>
__device__ void move_rows(const CompactParams &P)
{
    const spec_pages_compact_args &A = P.a;
    const int moves = got<SMALL>(P.w.moves), used = got<SMALL>(P.w.moves + 1), most = A.num_pages / 2;
    const long long step = (long long)gridDim.x * TH;
    const long long first = (long long)blockIdx.x * TH + threadIdx.x;
    for (long long i = first; i < most; i += step) {
        int src = -1, dst = -1;
        if (i < moves) {
            src = got<SMALL>(P.w.movers + i);
            dst = got<SMALL>(P.w.holes + i);
            A.ref_out[dst] = __ldg(A.ref_in + src);
        }
        A.copies[i] = src;
        A.copies[most + i] = dst;
        A.copies[2ll * most + i] = i < moves ? A.page_size : 0;
    }
    const long long entries = (long long)A.rows * A.pages_per_seq;
    for (long long i = first; i < entries; i += step) {
        int e = __ldg(A.table_in + i);
        if (e >= used && e < A.num_pages && __ldg(A.ref_in + e) > 0)
            e = got<SMALL>(P.w.holes + got<SMALL>(P.w.rank + e));
        A.table_out[i] = e;
    }
}

__global__ void __launch_bounds__(TH) compact_count_kernel(const __grid_constant__ CompactParams P)
{
    allow_next_kernel();
    wait_previous_kernel();
    list_free<true>(P.a.ref_in, nullptr, P.a.num_pages, (int)blockIdx.x, P.w);
}

__global__ void __launch_bounds__(TH) compact_list_kernel(const __grid_constant__ CompactParams P)
{
    allow_next_kernel();
    wait_previous_kernel();
    list_moves<false>(P, (int)blockIdx.x);
}

__global__ void __launch_bounds__(TH) compact_rows_kernel(const __grid_constant__ CompactParams P)
{
    allow_next_kernel();
    wait_previous_kernel();
    move_rows<false>(P);
}

// All three by one CTA, where it has one block of pages and a small table.
__global__ void __launch_bounds__(TH) compact_small_kernel(const __grid_constant__ CompactParams given)
{
    __shared__ int free_of, moves[2], holes[PB / 2], movers[PB / 2], rank[PB];
    __shared__ CompactParams P;
    if (threadIdx.x == 0) {
        P = given;
        P.w.free_of = &free_of;
        P.w.moves = moves;
        P.w.holes = holes;  // no more than there are pages in use behind them
        P.w.movers = movers;
        P.w.rank = rank;
    }
    allow_next_kernel();
    wait_previous_kernel();
    __syncthreads();
    list_free<true>(P.a.ref_in, nullptr, P.a.num_pages, 0, P.w);
    __syncthreads();
    list_moves<true>(P, 0);
    __syncthreads();
    move_rows<true>(P);
}

// ------------------------------------------------------------------- copy

struct CopyParams {
    spec_pages_copy_args a;
    int head, row;     // vectors of a head and of a slot
    int parts;         // pieces of a page, PIECE vectors each
};

constexpr int PIECE = 256;

// FLAT: a page's slots and heads lie one after the other.
template <typename V, bool FLAT>
__global__ void __launch_bounds__(TH) copy_kernel(const __grid_constant__ CopyParams P)
{
    const spec_pages_copy_args &A = P.a;
    const int lane = (int)threadIdx.x & 31;
    allow_next_kernel();
    wait_previous_kernel();
    const long long jobs = (long long)A.n * P.parts;
    const long long W = (long long)gridDim.x * WARPS;
    for (int side = (int)blockIdx.y; side < 2 * A.layers; side += (int)gridDim.y) {
        const int64_t *st = side & 1 ? A.v_cache_stride : A.k_cache_stride;
        uint8_t *base = static_cast<uint8_t *>(side & 1 ? A.v_cache : A.k_cache) +
                        (side >> 1) * st[0] * A.elem_size;
        for (long long j0 = (long long)blockIdx.x * WARPS + (threadIdx.x >> 5); j0 < jobs;
             j0 += 32 * W) {
            // lane l looks at job j0 + l W
            const long long j = j0 + lane * W;
            int src = -1, dst = -1, from = 0, to = 0;
            if (j < jobs) {
                const int e = (int)(j / P.parts);
                src = __ldg(A.copies + e);
                dst = __ldg(A.copies + A.n + e);
                const int slots = __ldg(A.copies + 2 * (size_t)A.n + e);
                from = (int)(j - (long long)e * P.parts) * PIECE;
                if (slots > 0 && slots <= A.page_size)
                    to = min(slots * P.row, from + PIECE);
            }
            const bool on = src >= 0 && src < A.num_pages && dst >= 0 && dst < A.num_pages &&
                            from < to;
            for (uint32_t left = __ballot_sync(0xffffffffu, on); left; left &= left - 1) {
                const int l = __ffs((int)left) - 1;
                const int f = __shfl_sync(0xffffffffu, from, l), t = __shfl_sync(0xffffffffu, to, l);
                const V *s = reinterpret_cast<const V *>(
                    base + __shfl_sync(0xffffffffu, src, l) * st[1] * A.elem_size);
                V *d = reinterpret_cast<V *>(
                    base + __shfl_sync(0xffffffffu, dst, l) * st[1] * A.elem_size);
                auto at = [&](int v) -> int64_t {
                    if (FLAT)
                        return v;
                    const int slot = v / P.row, in = v - slot * P.row, h = in / P.head;
                    return (slot * st[2] + h * st[3]) * A.elem_size / (int)sizeof(V) + in - h * P.head;
                };
                for (int v = f + lane; v < t; v += 8 * 32) {
                    V x[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        if (v + u * 32 < t)
                            x[u] = s[at(v + u * 32)];
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        if (v + u * 32 < t)
                            d[at(v + u * 32)] = x[u];
                }
            }
        }
    }
}

// ------------------------------------------------------------------- host

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t up(size_t x) { return (x + 255) / 256 * 256; }
int blocks_of(int pages) { return (pages + PB - 1) / PB; }

struct Span {
    const int32_t *p;
    uint64_t n;
};

// A null array, a misaligned one, or an output that shares a word with another array.
template <size_t I, size_t O>
bool arrays_bad(const Span (&in)[I], const Span (&out)[O])
{
    auto shares = [](const Span &x, const Span &y) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
        return x.n && y.n && a < b + y.n * 4 && b < a + x.n * 4;
    };
    for (const Span &s : in)
        if (s.n && (!s.p || !aligned(s.p, 4)))
            return true;
    for (size_t i = 0; i < O; ++i) {
        if (out[i].n && (!out[i].p || !aligned(out[i].p, 4)))
            return true;
        for (const Span &s : in)
            if (shares(out[i], s))
                return true;
        for (size_t j = 0; j < i; ++j)
            if (shares(out[i], out[j]))
                return true;
    }
    return false;
}

bool sizes_ok(int32_t rows, int32_t pages)
{
    return rows >= 0 && rows <= 65535 && pages >= 0 && pages <= SPEC_PAGES_MAX;
}

bool geometry_ok(int32_t pages_per_seq, int32_t page_size)
{
    return pages_per_seq >= 1 && page_size >= 1 &&
           (long long)pages_per_seq * page_size <= INT_MAX;
}

// The workspace's parts, from `at` on; returns its size.
size_t lay_out(int rows, int pages, uint8_t *at, Work &w)
{
    size_t used = 0;
    auto part = [&](size_t n) {
        int *p = reinterpret_cast<int *>(at + used);
        used += up(n * 4);
        return p;
    };
    w.free_of = part((size_t)blocks_of(pages));
    w.free_list = part((size_t)pages);
    w.need = part((size_t)rows);
    w.state = part((size_t)rows);
    w.holes = part((size_t)pages);
    w.movers = part((size_t)pages);
    w.rank = part((size_t)pages);
    w.moves = part(2);
    return used;
}

template <typename K, typename P>
int launch(K kernel, dim3 grid, size_t smem, const P &params, void *stream)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(TH);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, params) != cudaSuccess) {
        (void)cudaGetLastError();
        return SPEC_ECUDA;
    }
    return SPEC_OK;
}

static_assert((MAX_BLOCKS + 1) * 4 <= 48 * 1024 - 1024, "block sums without an opt-in");

}  // namespace

extern "C" {

size_t spec_pages_workspace_size(int32_t rows_out, int32_t num_pages)
{
    Work w;
    return sizes_ok(rows_out, num_pages) ? lay_out(rows_out, num_pages, nullptr, w) : 0;
}

int32_t spec_pages_fork(const spec_pages_fork_args *args, void *workspace, size_t workspace_bytes,
                        void *stream)
{
    if (!args)
        return SPEC_EINVAL;
    const spec_pages_fork_args &a = *args;
    if (!sizes_ok(a.rows_in, a.num_pages) || !sizes_ok(a.rows_out, a.num_pages) ||
        !geometry_ok(a.pages_per_seq, a.page_size))
        return SPEC_EINVAL;
    const uint64_t in = (uint64_t)a.rows_in, out = (uint64_t)a.rows_out;
    const Span ins[] = {{a.table_in, in * a.pages_per_seq}, {a.length_in, in}, {a.parent, out},
                        {a.reserve, a.reserve ? out : 0}, {a.ref_in, (uint64_t)a.num_pages}};
    const Span outs[] = {{a.table_out, out * a.pages_per_seq}, {a.length_out, out},
                         {a.ref_out, (uint64_t)a.num_pages}, {a.copies, 3 * out}};
    if (arrays_bad(ins, outs) || !workspace || !aligned(workspace, 256))
        return SPEC_EINVAL;
    ForkParams P;
    P.a = a;
    P.blocks = blocks_of(a.num_pages);
    if (workspace_bytes < lay_out(a.rows_out, a.num_pages, static_cast<uint8_t *>(workspace), P.w))
        return SPEC_ENOSPACE;
    if (P.blocks <= 1 && std::max(a.rows_in, a.rows_out) <= SMALL_ROWS && a.rows_out > 0)
        return launch(fork_small_kernel, dim3(1), (P.blocks + 1) * 4, P, stream);
    const unsigned int first = (unsigned int)(P.blocks + (a.rows_out + WARPS - 1) / WARPS);
    const unsigned int second =
        (unsigned int)((std::max(a.rows_in, a.rows_out) + WARPS - 1) / WARPS);
    if (first > 0) {
        const int rc = launch(fork_count_kernel, dim3(first), 0, P, stream);
        if (rc != SPEC_OK)
            return rc;
    }
    return second == 0 ? SPEC_OK
                       : launch(fork_rows_kernel, dim3(second), (P.blocks + 1) * 4, P, stream);
}

int32_t spec_pages_compact(const spec_pages_compact_args *args, void *workspace,
                           size_t workspace_bytes, void *stream)
{
    if (!args)
        return SPEC_EINVAL;
    const spec_pages_compact_args &a = *args;
    if (!sizes_ok(a.rows, a.num_pages) || a.num_pages < 1 ||
        !geometry_ok(a.pages_per_seq, a.page_size))
        return SPEC_EINVAL;
    const uint64_t entries = (uint64_t)a.rows * a.pages_per_seq, pages = (uint64_t)a.num_pages;
    const Span ins[] = {{a.table_in, entries}, {a.ref_in, pages}};
    const Span outs[] = {{a.table_out, entries}, {a.ref_out, pages}, {a.copies, 3 * (pages / 2)},
                         {a.used, 1}};
    if (arrays_bad(ins, outs) || !workspace || !aligned(workspace, 256))
        return SPEC_EINVAL;
    CompactParams P;
    P.a = a;
    P.blocks = blocks_of(a.num_pages);
    if (workspace_bytes < lay_out(a.rows, a.num_pages, static_cast<uint8_t *>(workspace), P.w))
        return SPEC_ENOSPACE;
    if (P.blocks == 1 && entries <= SMALL_ENTRIES)
        return launch(compact_small_kernel, dim3(1), 2 * 4, P, stream);
    int rc = launch(compact_count_kernel, dim3((unsigned int)P.blocks), 0, P, stream);
    if (rc == SPEC_OK)
        rc = launch(compact_list_kernel, dim3((unsigned int)P.blocks), (P.blocks + 1) * 4, P, stream);
    if (rc != SPEC_OK)
        return rc;
    const uint64_t most = std::max<uint64_t>(entries, pages / 2);
    const unsigned int grid = (unsigned int)std::min<uint64_t>((most + TH - 1) / TH, 1216);
    return launch(compact_rows_kernel, dim3(grid < 1 ? 1 : grid), 0, P, stream);
}

int32_t spec_pages_copy(const spec_pages_copy_args *args, void *stream)
{
    if (!args)
        return SPEC_EINVAL;
    const spec_pages_copy_args &a = *args;
    if (a.n < 0 || a.n > SPEC_PAGES_MAX || a.layers < 0 || a.Hkv < 1 || a.D < 1 || a.page_size < 1 ||
        a.num_pages < 0 || (a.elem_size != 2 && a.elem_size != 4) ||
        (long long)a.Hkv * a.D > (1 << 30) || (long long)a.page_size * a.Hkv * a.D > (1 << 30))
        return SPEC_EINVAL;
    if (a.n == 0 || a.layers == 0 || a.num_pages == 0)
        return SPEC_OK;
    const size_t es = (size_t)a.elem_size;
    if (!a.copies || !aligned(a.copies, 4) || !a.k_cache || !a.v_cache || !aligned(a.k_cache, es) ||
        !aligned(a.v_cache, es))
        return SPEC_EINVAL;
    const bool flat_heads = a.Hkv == 1 || (a.k_cache_stride[3] == a.D && a.v_cache_stride[3] == a.D);
    const int64_t slot = (int64_t)a.Hkv * a.D;
    const bool flat = flat_heads && (a.page_size == 1 || (a.k_cache_stride[2] == slot &&
                                                          a.v_cache_stride[2] == slot));
    // the widest vector that every address allows
    uint64_t bits = reinterpret_cast<uintptr_t>(a.k_cache) |
                    reinterpret_cast<uintptr_t>(a.v_cache) | (uint64_t)a.D * es;
    for (int i = 0; i < 4; ++i)
        bits |= (uint64_t)(a.k_cache_stride[i] | a.v_cache_stride[i]) * es;
    const size_t vec = (bits & 15) == 0 ? 16 : (bits & 3) == 0 ? 4 : 2;
    CopyParams P;
    P.a = a;
    P.head = (int)((size_t)a.D * es / vec);
    P.row = P.head * a.Hkv;
    P.parts = (int)(((long long)a.page_size * P.row + PIECE - 1) / PIECE);
    const unsigned int gy = (unsigned int)std::min(2ll * a.layers, 65535ll);
    const long long jobs = ((long long)a.n * P.parts + WARPS - 1) / WARPS;
    const long long most = std::max(1ll, 1216ll / gy);  // eight CTAs per SM
    const dim3 grid((unsigned int)std::min(jobs, most), gy);
    if (vec == 16)
        return flat ? launch(copy_kernel<uint4, true>, grid, 0, P, stream)
                    : launch(copy_kernel<uint4, false>, grid, 0, P, stream);
    if (vec == 4)
        return flat ? launch(copy_kernel<uint32_t, true>, grid, 0, P, stream)
                    : launch(copy_kernel<uint32_t, false>, grid, 0, P, stream);
    return flat ? launch(copy_kernel<unsigned short, true>, grid, 0, P, stream)
                : launch(copy_kernel<unsigned short, false>, grid, 0, P, stream);
}

}  // extern "C"
