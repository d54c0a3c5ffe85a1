// spec_beam.cu -- beam search's selection over beams and vocabulary, and the beams' states in the
// order of the selected (include/spec_beam.h).
//
// Selection, first kernel: one pass over the logits of the live beams.  A row is cut into segments,
// one per CTA.  A thread reads 4 vectors at a time (a group), adds to its running sum of exponentials
// and notes the group's maximum; no thread waits for another.  Within a beam candidates are ordered by
// their logits alone (one constant per beam makes scores of them), so no candidate needs the row's
// total: when the segment has been read, the n-th largest of the threads' own maxima (of 8 threads per
// warp) bounds its n best logits from below, the few groups that reach the bound are
// read again, and their elements that do are sorted.
// The last CTA of a sequence joins its rows' totals and merges the sorted lists of all segments: the
// n-th best head bounds the result, so at most n lists have entries in it; those are sorted.
// Bound by the bytes of the logits, and by what comes behind them when all segments end at one
// time: 64 x 8 rows of 128256 bf16 (440 of them live, 113 MB) are read by 22 us (half of them by 20, 5.6
// TB/s), their best are chosen by 28 and merged by 34; 32 x 5 rows of 151936 fp32 (83 MB) by 17, 21
// and 28.  More bytes in flight (rings in shared memory, prefetches into L2) did not shorten the reading,
// nor did rows that begin at different places.
//
// Orders between beams hang on the difference of two logarithms of sums, which fp32 gives to a few
// 1e-6.  Where two neighbours of different beams lie nearer than that, the sequence is listed,
// and the second kernel takes the sums of its beams again in exact integers (units of 2^-51 of the row's
// largest weight, resolve.cuh) and merges once more, so the order is that of 64 bits.
//
// Reorder: a gather of rows, 128 vectors of a row per warp, in the widest vectors that the
// addresses allow.  Bound by bytes, or by latency: 1024 rows of 8 KB, 4.8 us.
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "spec_beam.h"
#include "spec_verify.h"
#include "device_common.cuh"
#include "resolve.cuh"
#include "row_cut.h"

namespace {

using namespace spec_dev;

typedef unsigned long long u64;

constexpr int TH = 256;            // threads of a CTA
constexpr int WARPS = TH / 32;
static_assert(8 * WARPS >= SPEC_BEAM_MAX, "the first bound comes from 8 threads of a warp");
constexpr int UN = 4;              // vectors of a group
constexpr int GROUPS = 32;         // most groups of a thread, in a segment
static_assert(GROUPS <= 32, "a thread's groups are bits of a word");
constexpr int CAP = 1024;          // candidates of a segment before they are cut
constexpr int MAX_LISTS = 2048;    // segments of a sequence's beams: 608, or 9 of each of 64 long rows
constexpr int EXACT_CTAS = 152;
constexpr size_t MAX_B = 65536;    // sequences that the counters have room for
// How far a row's logarithm of its total may be off, in nats: exponents' rounding (2^-23 of up to
// 24 binary digits, and the constant's 2^-25: 2.5e-6), ex2 three times (2^-22 each: 0.7e-6), some 26
// fp32 additions and products of 2^-24 (1.6e-6)
constexpr double LSE_OFF = 5e-6;
constexpr float SLACK = 5.0f;      // nats that a maximum may run ahead of its sum's scale

struct BeamParams {
    spec_beam_select_args a;
    int segs;        // of a row
    int chunks;      // of a row in the exact sums
    WsHeader *hdr;   // n_flag: sequences listed; next_item: CTAs of the exact kernel that are done
    int *arrived;    // [B] CTAs of the first kernel
    int *summed;     // [B] items of the exact kernel, by place in the list
    int *listed;     // [B]
    float2 *stats;   // [B K segs] (largest logit, sum of exp(x - largest)); NaN: an error
    u64 *lists;      // [B K segs n] candidates, best first; 0: none
    long long *sums; // [B K chunks] by place in the list
};

// Floats in an order of unsigned numbers (-0 is 0), and a candidate: larger is better, of equal
// logits the lower token.
constexpr uint32_t NONE = 0x007fffffu;  // of -inf: no candidate
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(u64 key)
{
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ u64 candidate(uint32_t order, int col)
{
    return (u64)order << 32 | (uint32_t)~col;
}
__device__ __forceinline__ int token_of(u64 key) { return (int)~(uint32_t)key; }
__device__ __forceinline__ u64 ordered(double x)
{
    const u64 b = (u64)__double_as_longlong(x + 0.0);
    return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double rank_of(u64 o)
{
    return __longlong_as_double((long long)(o >> 63 ? o & ~(1ull << 63) : ~o));
}

struct ScanSmem {
    u64 cand[CAP];
    u64 best[8 * WARPS];
    float part[WARPS][2];
    u64 most[WARPS];
    uint32_t bound;
    int count;
};

struct PickSmem {
    double lse[SPEC_BEAM_MAX], score[SPEC_BEAM_MAX], inv[SPEC_BEAM_MAX];
    float2 total[SPEC_BEAM_MAX];  // a row's largest logit and sum of exp(x - largest)
    u64 rank[SPEC_BEAM_MAX];      // the best n, sorted
    int flat[SPEC_BEAM_MAX];
    float value[SPEC_BEAM_MAX];   // logits
    u64 least;
    int least_flat;
    int widest;                   // the largest 1 / norm, as a float's bits
    int count;
};

// Shared memory that a kernel is launched with: the groups' maxima of the scan, or a merge's first
// entries of lists (order, k V + x; 4 n of them, or one of each list) and then what it has to
// sort, up to n entries of n lists (a place too).
constexpr int FEW = 128;
constexpr size_t larger(size_t a, size_t b) { return a > b ? a : b; }
constexpr size_t merge_bytes(int n, int lists)
{
    return larger(larger((size_t)n * n, (size_t)FEW) * 16, larger((size_t)lists, (size_t)4 * n) * 12);
}
constexpr size_t SCAN_BYTES = (size_t)GROUPS * TH * 4;
extern __shared__ __align__(16) uint8_t dyn[];

__device__ __forceinline__ bool better(u64 r1, int f1, u64 r2, int f2)
{
    return r1 > r2 || (r1 == r2 && f1 < f2);
}

// The places of m things in their order, by the whole CTA: `is_better(j, i)` compares two, `found(i, place)`
// is told once for each.  Four lanes share one thing's comparisons: with a warp for each thing
// a merge of 128 took 0.6 us more.
template <typename B, typename F>
__device__ __forceinline__ void places(int m, B is_better, F found)
{
    const int quarter = (int)threadIdx.x & 3;
    for (int i0 = 0; i0 < m; i0 += TH / 4) {
        const int i = i0 + (int)(threadIdx.x >> 2);
        int place = 0;
        if (i < m)
#pragma unroll 4
            for (int j = quarter; j < m; j += 4)
                place += is_better(j, i) ? 1 : 0;
        place += __shfl_xor_sync(0xffffffffu, place, 1);
        place += __shfl_xor_sync(0xffffffffu, place, 2);
        if (i < m && quarter == 0)
            found(i, place);
    }
}

// The candidates' best n, sorted, to S.cand; returns the order that a later one has to exceed.
// The whole CTA; S.count candidates (at most CAP).
__device__ uint32_t cut(ScanSmem &S, int n)
{
    const int tid = (int)threadIdx.x;
    __syncthreads();
    const int m = S.count;
    if (tid < n)
        S.best[tid] = 0;
    __syncthreads();
    places(m, [&](int j, int i) { return S.cand[j] > S.cand[i]; },
           [&](int i, int place) {
               if (place < n)
                   S.best[place] = S.cand[i];
           });
    __syncthreads();
    if (tid < n)
        S.cand[tid] = S.best[tid];
    if (tid == 0)
        S.count = m < n ? m : n;
    __syncthreads();
    return m < n ? NONE : (uint32_t)(S.best[n - 1] >> 32);
}

// A whole CTA merges the lists of sequence b.  `exact`: S.lse holds the beams' logarithms;
// otherwise they come from the segments' totals, and the answer says whether the order stands.
template <bool EXACT>
__device__ bool pick(const BeamParams &P, int b, PickSmem &S)
{
    const spec_beam_select_args &A = P.a;
    const int tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31;
    bool bad = false;
    if (tid == 0)
        S.widest = 0;
    // candidate `at` of list l: 0 for none, ENDED for an ended beam's one
    constexpr u64 ENDED = 1;
    const int lists = A.K * P.segs, n = A.n;
    auto fetch = [&](int l, int at) -> u64 {
        const int k = l / P.segs, row = b * A.K + k;
        const float s = A.scores[row];
        const bool fin = A.finished && A.finished[row] != 0;
        const u64 key = __ldcg(&P.lists[((size_t)row * P.segs + (l - k * P.segs)) * n + at]);
        return !(s > -INFINITY) ? 0 : !fin ? key : at == 0 && l == k * P.segs ? ENDED : 0;
    };
    // Few candidates in all: each has a thread, whose load is on its way from here on, and all are
    // compared (64: 1.5 us less than by the bound below; 128: 0.25 less; 150: 2.2 more)
    const bool few = lists * n <= FEW;
    const u64 mine = few && tid < lists * n ? fetch(tid / n, tid % n) : 0;
    // (and so is what a row has of its own)
    const bool own = tid < A.K;
    const float norm = own && A.norm ? A.norm[b * A.K + tid] : 1.0f;
    const float s = own ? A.scores[b * A.K + tid] : -INFINITY;
    const bool fin = own && A.finished && A.finished[b * A.K + tid] != 0;
    // the rows' totals, a row per warp; what takes 64 bits for all rows at once, a row per lane (this
    // GPU has two 64-bit lanes per SM: by the warps one after the other it took 10 us)
    if (!EXACT)
        for (int k = warp; k < A.K; k += WARPS) {
            const size_t first = ((size_t)b * A.K + k) * P.segs;
            float2 x = make_float2(-INFINITY, 0.0f), y = x;
            if (lane < P.segs)
                x = __ldcg(&P.stats[first + lane]);
            if (!(A.scores[b * A.K + k] > -INFINITY) ||
                (A.finished && A.finished[b * A.K + k] != 0))
                continue;
            float top = x.x, z = 0.0f;
            bad |= isnan(x.x);
            for (int g = lane + 32; g < P.segs; g += 32) {
                y = __ldcg(&P.stats[first + g]);
                bad |= isnan(y.x);
                top = fmaxf(top, y.x);
            }
            for (int d = 16; d; d >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            if (x.x > -INFINITY)
                z = x.y * ex2((x.x - top) * LOG2E);
            for (int g = lane + 32; g < P.segs; g += 32) {
                y = __ldcg(&P.stats[first + g]);
                if (y.x > -INFINITY)
                    z += y.y * ex2((y.x - top) * LOG2E);
            }
            for (int d = 16; d; d >>= 1)
                z += __shfl_xor_sync(0xffffffffu, z, d);
            if (lane == 0)
                S.total[k] = make_float2(top, z);
        }
    __syncthreads();
    if (own) {
        bad |= isnan(s) || s == INFINITY;
        if (s > -INFINITY) {
            bad |= !(norm > 0.0f) || isinf(norm);
            S.score[tid] = (double)s;
            if (!EXACT) {
                // 1 / norm: fp32's, and a step of Newton's iteration, far from fp32's ends
                const float to = norm < 0x1p-64f ? 0x1p64f : norm > 0x1p64f ? 0x1p-64f : 1.0f;
                const double guess = (double)(1.0f / (norm * to));
                S.inv[tid] =
                    A.norm ? guess * (2.0 - (double)(norm * to) * guess) * (double)to : 1.0;
                // (rounded up; infinity where a float has no room)
                if (norm > 0.0f)
                    atomicMax(&S.widest, __float_as_int(__double2float_ru(S.inv[tid])));
                // ln z = e ln 2 + ln m, m in [2/3, 4/3)
                const float2 x = fin ? make_float2(0.0f, 1.0f) : S.total[tid];
                int e;
                float m = frexpf(x.y, &e);
                if (m < 2.0f / 3.0f) {
                    m *= 2.0f;
                    --e;
                }
                S.lse[tid] = x.x > -INFINITY
                    ? (double)x.x + ((double)e * 0.693147180559945309 + (double)logf(m)) : 0.0;
            }
        }
    }
    bad = __syncthreads_or(bad ? 1 : 0) != 0;
    const size_t out = (size_t)b * A.n;
    if (bad) {
        for (int i = tid; i < A.n; i += TH) {
            A.out_tokens[out + i] = -1;
            A.out_beams[out + i] = -1;
            A.out_scores[out + i] = NAN;
        }
        return true;
    }
    auto rank_by = [&](double score, int k) -> u64 {
        return ordered(EXACT ? score / (A.norm ? (double)A.norm[b * A.K + k] : 1.0)
                             : score * S.inv[k]);
    };
    // a candidate's order (0: none), and k V + x
    auto worth = [&](int l, u64 key, int &flat, float &value) -> u64 {
        const int k = l / P.segs;
        flat = key == 0 ? INT_MAX : k * A.V + (key == ENDED ? A.end_token : token_of(key));
        if (key <= ENDED)
            return key == 0 ? 0 : rank_by(S.score[k], k);
        value = value_of(key);
        return rank_by(S.score[k] + ((double)value - S.lse[k]), k);
    };
    u64 *rank = reinterpret_cast<u64 *>(dyn);
    int *flat;
    float *value;
    int m;  // candidates among which the n best are
    bool open = false;
    if (tid < n)
        S.rank[tid] = 0;
    if (few) {
        m = lists * n;
        flat = reinterpret_cast<int *>(rank + m);
        value = reinterpret_cast<float *>(flat + m);
        if (tid < m)
            rank[tid] = worth(tid / n, mine, flat[tid], value[tid]);
    } else {
        // the n-th best of the lists' first entries: no more than n lists reach it, and where a few of
        // each list are looked at, not many more than n entries
        const int deep = min(n, max(1, 4 * n / lists)), firsts = lists * deep;
        flat = reinterpret_cast<int *>(rank + firsts);
        float x = 0.0f;
        for (int e = tid; e < firsts; e += TH)
            rank[e] = worth(e / deep, fetch(e / deep, e % deep), flat[e], x);
        if (tid == 0) {
            S.least = 0;
            S.least_flat = INT_MAX;
            S.count = 0;
        }
        __syncthreads();
        places(firsts, [&](int j, int i) { return better(rank[j], flat[j], rank[i], flat[i]); },
               [&](int i, int place) {
                   if (rank[i] != 0 && place == n - 1) {
                       S.least = rank[i];
                       S.least_flat = flat[i];
                   }
               });
        __syncthreads();
        // the entries that reach it (n n of them at most, in the place of the heads); where the order
        // may be open, also those that might after all
        flat = reinterpret_cast<int *>(rank + n * n);
        value = reinterpret_cast<float *>(flat + n * n);
        const int least_flat = S.least_flat;
        u64 least = S.least;
        if (!EXACT && least != 0) {
            const double low =
                rank_of(least) - 2.0 * LSE_OFF * (double)__int_as_float(S.widest);
            least = low > -INFINITY ? ordered(low) : 0;
        }
        for (int e = tid; e < lists * n; e += TH) {
            int f;
            const u64 r = worth(e / n, fetch(e / n, e % n), f, x);
            if (r != 0 && (EXACT ? !better(least, least_flat, r, f) : r >= least)) {
                const int i = atomicAdd(&S.count, 1);
                if (i < n * n) {
                    rank[i] = r;
                    flat[i] = f;
                    value[i] = x;
                }
            }
        }
        __syncthreads();
        open = !EXACT && S.count > n * n;
        m = min(S.count, n * n);
    }
    __syncthreads();
    places(m, [&](int j, int i) { return better(rank[j], flat[j], rank[i], flat[i]); },
           [&](int i, int place) {
               if (rank[i] != 0 && place < n) {
                   S.rank[place] = rank[i];
                   S.flat[place] = flat[i];
                   S.value[place] = value[i];
               }
           });
    __syncthreads();
    // two candidates of different beams lie too near: neighbours among the best, or the last of these
    // and any that is left (no other pair's order can be open then)
    auto near = [&](u64 r1, int f1, u64 r2, int f2) {
        const double off = LSE_OFF * (S.inv[f1 / A.V] + S.inv[f2 / A.V]);
        return f1 / A.V != f2 / A.V && !(rank_of(r1) - rank_of(r2) > off);
    };
    if (!EXACT && S.rank[n - 1] != 0)
        for (int i = tid; i < m; i += TH)
            open |= rank[i] != 0 && better(S.rank[n - 1], S.flat[n - 1], rank[i], flat[i]) &&
                    near(S.rank[n - 1], S.flat[n - 1], rank[i], flat[i]);
    if (tid < n) {
        int token = -1, beam = -1;
        float score = -INFINITY;
        if (S.rank[tid] != 0) {
            const int k = S.flat[tid] / A.V;
            beam = k;
            token = S.flat[tid] - k * A.V;
            score = (float)S.score[k];
            if (!(A.finished && A.finished[b * A.K + k] != 0))
                score = (float)(S.score[k] + ((double)S.value[tid] - S.lse[k]));
            if (!EXACT && tid + 1 < n && S.rank[tid + 1] != 0)
                open |= near(S.rank[tid], S.flat[tid], S.rank[tid + 1], S.flat[tid + 1]);
        }
        A.out_tokens[out + tid] = token;
        A.out_beams[out + tid] = beam;
        A.out_scores[out + tid] = score;
    }
    return __syncthreads_or(open ? 1 : 0) == 0;
}

// A row's segment: whole vectors of the array.  The row's elements before its first one and behind
// its last (fewer than two vectors) belong to the first segment, one for each of its first threads.
template <int DT>
struct Segment {
    using L = Lg<DT>;
    const uint4 *src;
    int mis, v0, v1;
    int head, tail, edges;  // elements before the vectors, the first one behind, and how many in all
    const void *base;
    size_t e0;

    __device__ __forceinline__ Segment(const BeamParams &P, int row, int seg)
    {
        const int V = P.a.V;
        base = P.a.logits;
        e0 = (size_t)row * V;
        src = reinterpret_cast<const uint4 *>(base) + e0 / L::VEC;
        const RowCut cut = cut_row<L::VEC>(e0, V);
        const int per = (cut.f1 - cut.f0 + P.segs - 1) / P.segs;
        mis = cut.mis;  // elements of the row's first vector before it
        v0 = cut.f0 + seg * per;
        v1 = min(cut.f1, v0 + per);
        head = cut.head;
        tail = cut.tail;
        edges = seg == 0 ? head + V - tail : 0;
    }
    // (past L1, which holds no segment: 64 x 8 rows of 128256 bf16 40.4 -> 36.8 us, 32 x 5 of 151936
    // fp32 32.5 -> 30.3, with inputs that L2 does not hold.  Volatile and with a clobber: without, the
    // compiler may take it for arithmetic on the address and move it before the wait for the kernel that
    // writes the logits.  That costs nothing: 37.4 us either way, and 30.6.)
    __device__ __forceinline__ uint4 fetch(int v) const
    {
        uint4 r = neg_inf_vec(L::NEG_INF_WORD);
        if (v < v1)
            asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(src + v) : "memory");
        return r;
    }
    __device__ __forceinline__ int col(int v, int j) const { return v * L::VEC + j - mis; }
    __device__ __forceinline__ int edge_col(int i) const { return i < head ? i : tail + i - head; }
    __device__ __forceinline__ float edge(int i) const
    {
        return i < edges ? L::load1(base, e0 + edge_col(i)) : -INFINITY;
    }
};

// The segment's n best where too many reach the bound (equal logits): tile by tile in order, each
// tile's best one by one where there are too many of them too.  The whole CTA; to S.cand.
template <int DT>
__device__ __noinline__ void scan_again(const Segment<DT> &G, int n, ScanSmem &S)
{
    using L = Lg<DT>;
    const int tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t above = NONE;
    int held = 0;  // candidates before the tile
    auto push_edge = [&](bool head) {
        const float x = G.edge(tid);
        if (tid < G.edges && (tid < G.head) == head && ordered(x) > above)
            S.cand[atomicAdd(&S.count, 1)] = candidate(ordered(x), G.edge_col(tid));
    };
    __syncthreads();
    if (tid == 0)
        S.count = 0;
    __syncthreads();
    push_edge(true);
    __syncthreads();
    held = S.count;
    __syncthreads();
    for (int t = G.v0; t < G.v1; t += TH * UN) {
        u64 lower = ~0ull;
        for (int u = 0; u < UN; ++u) {
            float x[L::VEC];
            L::unpack(G.fetch(t + u * TH + tid), x);
            for (int j = 0; j < L::VEC; ++j) {
                const uint32_t o = ordered(x[j]);
                if (o > above) {
                    const int i = atomicAdd(&S.count, 1);
                    if (i < CAP)
                        S.cand[i] = candidate(o, G.col(t + u * TH + tid, j));
                }
            }
        }
        __syncthreads();
        int now = S.count;
        __syncthreads();
        for (int got = 0; now > CAP; ++got) {
            u64 most = 0;
            if (got < n)
                for (int u = 0; u < UN; ++u) {
                    float x[L::VEC];
                    L::unpack(G.fetch(t + u * TH + tid), x);
                    for (int j = 0; j < L::VEC; ++j) {
                        const uint32_t o = ordered(x[j]);
                        const u64 key = candidate(o, G.col(t + u * TH + tid, j));
                        if (o > above && key < lower && key > most)
                            most = key;
                    }
                }
            for (int d = 16; d; d >>= 1) {
                const u64 other = __shfl_xor_sync(0xffffffffu, most, d);
                most = other > most ? other : most;
            }
            if (lane == 0)
                S.most[warp] = most;
            __syncthreads();
            for (int w = 0; w < WARPS; ++w)
                most = S.most[w] > most ? S.most[w] : most;
            __syncthreads();
            if (most == 0) {
                now = held + got;
                if (tid == 0)
                    S.count = now;
            } else {
                if (tid == 0)
                    S.cand[held + got] = most;
                lower = most;
            }
        }
        above = cut(S, n);
        held = min(now, n);
    }
    push_edge(false);
    (void)cut(S, n);
}

template <int DT>
__global__ void __launch_bounds__(TH, 4) beam_kernel(const __grid_constant__ BeamParams P)
{
    using L = Lg<DT>;
    const spec_beam_select_args &A = P.a;
    __shared__ union {
        ScanSmem scan;
        PickSmem pick;
    } U;
    __shared__ int last;
    ScanSmem &S = U.scan;
    const int tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = (int)(blockIdx.x / P.segs), seg = (int)(blockIdx.x - row * P.segs);
    const int b = row / A.K, n = A.n;
    allow_next_kernel();
    wait_previous_kernel();
    const Segment<DT> G(P, row, seg);
    uint4 raw[UN], ahead[UN];
    // Logits of a beam that has ended or does not exist are not read.  (To have the first group on its way
    // before that is known took 0.4 us less of 31 on 32 x 5 rows of 151936 fp32, 0.1 of 37.5 on
    // 64 x 8 of 128256 bf16.)
    const bool counts = A.scores[row] > -INFINITY && !(A.finished && A.finished[row] != 0);
    if (counts) {
#pragma unroll
        for (int u = 0; u < UN; ++u)
            raw[u] = G.fetch(G.v0 + u * TH + tid);
        float *maxima = reinterpret_cast<float *>(dyn) + tid;  // of the thread's groups
        float m = -INFINITY, top = -INFINITY, sum = 0.0f, low = 0.0f;  // sum + low in units of e^m
        bool bad = false;
        const u64 c2 = f2(LOG2E, LOG2E);
        const float lone = G.edge(tid);
        if (G.edges > 0) {
            bad = !(lone < INFINITY);
            m = top = lone;
            sum = lone > -INFINITY ? 1.0f : 0.0f;
        }
        int groups = 0;
        for (int t = G.v0; t < G.v1; t += TH * UN) {
#pragma unroll
            for (int u = 0; u < UN; ++u)
                ahead[u] = G.fetch(t + TH * UN + u * TH + tid);
            const float tm = L::tile_max(raw);
            maxima[groups++ * TH] = tm;
            bad |= !(tm < INFINITY);
            top = fmaxf(top, tm);
            if (tm > m + SLACK || m == -INFINITY) {
                const float f = m == -INFINITY ? 0.0f : ex2((m - tm) * LOG2E);
                sum *= f;
                low *= f;
                m = tm;
            }
            if (m > -INFINITY) {
                u64 acc = L::expsum2(raw[0], -m, c2);
#pragma unroll
                for (int u = 1; u < UN; ++u)
                    acc = add2(acc, L::expsum2(raw[u], -m, c2));
                float x, y;
                f2_split(acc, x, y);
                x += y;
                // sum + x exactly, as a float and what it leaves (Knuth's two-sum)
                const float s = __fadd_rn(sum, x), back = __fsub_rn(s, sum);
                low += __fadd_rn(__fsub_rn(sum, __fsub_rn(s, back)), __fsub_rn(x, back));
                sum = s;
            }
#pragma unroll
            for (int u = 0; u < UN; ++u)
                raw[u] = ahead[u];
        }
        // the bound: the n-th of the warps' 8 best threads, whose maxima each warp sorts (a bitonic
        // network over its lanes)
        uint32_t mine = bad ? NONE : ordered(top);
#pragma unroll
        for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
            for (int d = size >> 1; d; d >>= 1) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, d);
                const bool larger_one = ((lane & d) == 0) == ((lane & size) == 0 || size == 32);
                mine = larger_one ? max(mine, other) : min(mine, other);
            }
        if (lane < 8)
            S.best[warp * 8 + lane] = (u64)mine << 32 | (uint32_t)(warp * 8 + lane);
        if (lane == 0)
            S.part[warp][0] = mine == NONE ? -INFINITY : value_of((u64)mine << 32);
        if (tid == 0)
            S.count = 0;
        bad = __syncthreads_or(bad ? 1 : 0) != 0;
        places(8 * WARPS, [&](int j, int i) { return S.best[j] > S.best[i]; },
               [&](int i, int place) {
                   if (place == n - 1)
                       S.bound = (uint32_t)(S.best[i] >> 32);
               });
        float most = -INFINITY;
        // the segment's total
        for (int w = 0; w < WARPS; ++w)
            most = fmaxf(most, S.part[w][0]);
        float z = m > -INFINITY ? (sum + low) * ex2((m - most) * LOG2E) : 0.0f;
        for (int d = 16; d; d >>= 1)
            z += __shfl_xor_sync(0xffffffffu, z, d);
        if (lane == 0)
            S.part[warp][1] = z;
        __syncthreads();
        if (tid == 0) {
            z = 0.0f;
            for (int w = 0; w < WARPS; ++w)
                z += S.part[w][1];
            P.stats[(size_t)row * P.segs + seg] =
                bad ? make_float2(NAN, NAN) : make_float2(most, z);
        }
        if (!bad) {
            const uint32_t above = max(S.bound, NONE + 1) - 1;  // the bound itself included
            if (ordered(lone) > above)
                S.cand[atomicAdd(&S.count, 1)] = candidate(ordered(lone), G.edge_col(tid));
            uint32_t reach = 0;  // the thread's groups that do, each lane's next one at a time
#pragma unroll 4
            for (int g = 0; g < groups; ++g)
                reach |= (ordered(maxima[g * TH]) > above ? 1u : 0u) << g;
            for (; reach; reach &= reach - 1) {
                const int v = G.v0 + (__ffs((int)reach) - 1) * TH * UN + tid;
#pragma unroll
                for (int u = 0; u < UN; ++u)
                    raw[u] = G.fetch(v + u * TH);
#pragma unroll
                for (int u = 0; u < UN; ++u) {
                    if (ordered(L::vmax(raw[u])) <= above)
                        continue;
                    float x[L::VEC];
                    L::unpack(raw[u], x);
#pragma unroll
                    for (int j = 0; j < L::VEC; ++j) {
                        const uint32_t o = ordered(x[j]);
                        if (o > above) {
                            const int i = atomicAdd(&S.count, 1);
                            if (i < CAP)
                                S.cand[i] = candidate(o, G.col(v + u * TH, j));
                        }
                    }
                }
            }
            __syncthreads();
            if (S.count > CAP)
                scan_again(G, n, S);
            else
                (void)cut(S, n);
            u64 *list = P.lists + ((size_t)row * P.segs + seg) * n;
            for (int i = tid; i < n; i += TH)
                list[i] = i < S.count ? S.cand[i] : 0;
        }
    }
    // the sequence's last CTA merges
    __syncthreads();
    if (tid == 0) {
        // (release, of what the others wrote before the barrier too, and acquire)
        int had;
        asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;"
                     : "=r"(had) : "l"(P.arrived + b) : "memory");
        last = had == A.K * P.segs - 1;
        if (last)
            P.arrived[b] = 0;
    }
    __syncthreads();
    if (!last)
        return;
    if (!pick<false>(P, b, U.pick) && tid == 0)
        P.listed[atomicAdd(&P.hdr->n_flag, 1u)] = b;
}

struct ExactSmem {
    float2 tab[256];
    long long part[WARPS];
    int last;
};

// The exact sums of the listed sequences' beams, 2048 logits at a time, and their merge.
template <int DT>
__global__ void __launch_bounds__(TH, 4) beam_exact_kernel(const __grid_constant__ BeamParams P)
{
    using L = Lg<DT>;
    const spec_beam_select_args &A = P.a;
    __shared__ ExactSmem S;
    __shared__ PickSmem K;
    const int tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31;
    allow_next_kernel();
    wait_previous_kernel();
    const int listed = (int)*reinterpret_cast<volatile unsigned int *>(&P.hdr->n_flag);
    if (listed == 0)
        return;
    load_exp2_table(S.tab);
    __syncthreads();
    auto counts = [&](int row) {
        return A.scores[row] > -INFINITY && !(A.finished && A.finished[row] != 0);
    };
    auto top_of = [&](int row) -> float {
        float top = -INFINITY;
        for (int g = 0; g < P.segs; ++g)
            top = fmaxf(top, __ldcg(&P.stats[(size_t)row * P.segs + g]).x);
        return top;
    };
    const long long per = (long long)A.K * P.chunks, items = per * listed;
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
        const int i = (int)(item / per), k = (int)(item - i * per) / P.chunks;
        const int chunk = (int)(item - i * per) - k * P.chunks;
        const int b = __ldcg(&P.listed[i]), row = b * A.K + k;
        const float top = counts(row) ? top_of(row) : -INFINITY;
        if (top > -INFINITY) {
            long long sum = 0;
            for (int c = chunk * RCH + 2 * tid; c < min(A.V, (chunk + 1) * RCH); c += 2 * TH) {
                const bool two = c + 1 < A.V;
                const float x0 = L::load1(A.logits, (size_t)row * A.V + c);
                const float x1 = two ? L::load1(A.logits, (size_t)row * A.V + c + 1) : -INFINITY;
                long long E0, E1;
                float a0, a1;
                efix2(x0, x1, top, top, true, two, LOG2E_HI, LOG2E_LO, S.tab, E0, E1, a0, a1);
                sum += E0 + E1;
            }
            for (int d = 16; d; d >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, d);
            if (lane == 0)
                S.part[warp] = sum;
            __syncthreads();
            if (tid == 0) {
                for (int w = 1; w < WARPS; ++w)
                    sum += S.part[w];
                P.sums[((size_t)i * A.K + k) * P.chunks + chunk] = sum;
            }
        }
        __threadfence();
        __syncthreads();
        if (tid == 0) {
            S.last = atomicAdd(&P.summed[i], 1) == (int)per - 1;
            if (S.last)
                P.summed[i] = 0;
        }
        __syncthreads();
        if (!S.last)
            continue;
        __threadfence();
        for (int q = warp; q < A.K; q += WARPS) {
            const int r = b * A.K + q;
            const float high = counts(r) ? top_of(r) : -INFINITY;
            double z = 0.0;
            if (high > -INFINITY)
                for (int c = lane; c < P.chunks; c += 32)
                    z += (double)__ldcg(&P.sums[((size_t)i * A.K + q) * P.chunks + c]);
            for (int d = 16; d; d >>= 1)
                z += __shfl_xor_sync(0xffffffffu, z, d);
            if (lane == 0)
                K.lse[q] = high > -INFINITY ? (double)high + log(z * 0x1p-51) : 0.0;
        }
        __syncthreads();
        (void)pick<true>(P, b, K);
        __syncthreads();
    }
    // the list is empty again once every CTA has been through it
    if (tid == 0) {
        __threadfence();
        if (atomicAdd(&P.hdr->next_item, 1u) == gridDim.x - 1) {
            P.hdr->next_item = 0;
            P.hdr->n_flag = 0;
        }
    }
}

// ---------------------------------------------------------------- reorder

struct ReorderParams {
    const void *in;
    void *out;
    const int32_t *beams;
    long long rows;      // of out: lead * B * n
    int per, K, n;       // B * n, beams in and out
    long long vecs;      // of a row
    int parts;           // pieces of a row, PIECE vectors each
};

constexpr int PIECE = 128;

template <typename V>
__global__ void __launch_bounds__(TH) reorder_kernel(const __grid_constant__ ReorderParams P)
{
    const int lane = (int)threadIdx.x & 31;
    allow_next_kernel();
    wait_previous_kernel();
    const long long jobs = P.rows * P.parts;
    for (long long j = (long long)blockIdx.x * WARPS + (threadIdx.x >> 5); j < jobs;
         j += (long long)gridDim.x * WARPS) {
        const long long row = j / P.parts;
        const long long first = (j - row * P.parts) * PIECE;
        const long long l = row / P.per;
        const int at = (int)(row - l * P.per), b = at / P.n, beam = __ldg(P.beams + at);
        const bool some = beam >= 0 && beam < P.K;
        const V *src = static_cast<const V *>(P.in) +
                       ((l * (P.per / P.n) + b) * P.K + (some ? beam : 0)) * P.vecs;
        V *dst = static_cast<V *>(P.out) + row * P.vecs;
        const long long end = min(P.vecs, first + PIECE);
        for (long long v = first + lane; v < end; v += 4 * 32) {
            V x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                x[u] = V{};
                if (some && v + u * 32 < end)
                    x[u] = __ldg(src + v + u * 32);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (v + u * 32 < end)
                    dst[v + u * 32] = x[u];
        }
    }
}

// ------------------------------------------------------------------- host

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t up(size_t x) { return (x + 255) / 256 * 256; }

// An output of a selection that shares a byte with an input or another output: CTAs read the scores
// of sequences that others have finished with, and where an order is open a second time.
bool outputs_apart(const spec_beam_select_args &a)
{
    struct Span {
        const void *p;
        uint64_t bytes;
    };
    const uint64_t rows = (uint64_t)a.B * a.K, each = (uint64_t)a.B * a.n * 4;
    const Span in[] = {{a.logits, rows * a.V * (a.dtype == SPEC_F32 ? 4 : 2)}, {a.scores, rows * 4},
                       {a.norm, rows * 4}, {a.finished, rows * 4}};
    const Span out[] = {{a.out_tokens, each}, {a.out_beams, each}, {a.out_scores, each}};
    auto apart = [](const Span &x, const Span &y) {
        const uintptr_t i = reinterpret_cast<uintptr_t>(x.p), j = reinterpret_cast<uintptr_t>(y.p);
        return !x.p || !y.p || i >= j + y.bytes || j >= i + x.bytes;
    };
    for (int o = 0; o < 3; ++o) {
        for (const Span &x : in)
            if (!apart(out[o], x))
                return false;
        for (int q = 0; q < o; ++q)
            if (!apart(out[o], out[q]))
                return false;
    }
    return true;
}

bool sizes_ok(int32_t B, int32_t K, int32_t V, int32_t n, int32_t dtype)
{
    return B >= 0 && B <= 65535 && K >= 1 && K <= SPEC_BEAM_MAX && n >= 1 && n <= SPEC_BEAM_MAX &&
           V >= 2 && V <= SPEC_MAX_V && (dtype == SPEC_F32 || dtype == SPEC_BF16);
}

// Segments of a row: as many CTAs in all as run at a time (four per SM), each of which ends with some
// us of choosing; no more groups than a thread has room for, and no fewer than one.  (64 x 8 rows of
// 128256 bf16 with the reordering: in one segment 37.4 us, in two 43.0, in three 47.9.)
int segments(int32_t B, int32_t K, int32_t V, int32_t dtype)
{
    const long long rows = (long long)B * K;
    const int vecs = V / (dtype == SPEC_F32 ? 4 : 8) + 2;
    const int tiles = (vecs + TH * UN - 1) / (TH * UN), least = (tiles + GROUPS - 2) / (GROUPS - 1);
    long long s = rows > 0 ? 608 / rows : 1;
    s = s < tiles ? s : tiles;
    return s < least ? least : (int)s;
}

struct BeamLayout {
    size_t arrived, summed, listed, stats, lists, sums, total;
};

BeamLayout beam_layout(int32_t B, int32_t K, int32_t V, int32_t n, int32_t dtype)
{
    const size_t rows = (size_t)B * K, segs = (size_t)segments(B, K, V, dtype);
    const size_t chunks = (size_t)(V + RCH - 1) / RCH;
    BeamLayout w;
    // the counters, zero between calls, lie where calls of any sizes have them
    w.arrived = sizeof(WsHeader);
    w.summed = w.arrived + MAX_B * 4;
    w.listed = w.summed + MAX_B * 4;
    w.stats = up(w.listed + (size_t)B * 4);
    w.lists = up(w.stats + rows * segs * sizeof(float2));
    w.sums = up(w.lists + rows * segs * n * sizeof(u64));
    w.total = up(w.sums + rows * chunks * sizeof(long long));
    return w;
}

template <typename K, typename P>
int launch(K kernel, unsigned int grid, size_t smem, const P &params, void *stream)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
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

std::atomic<bool> g_attr[64][2];  // opted in to a merge's shared memory, per device and dtype

template <int DT>
int select_beams(const BeamParams &P, void *stream)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return SPEC_ECUDA;
    if (!g_attr[dev][DT].load(std::memory_order_acquire)) {
        constexpr int most = (int)merge_bytes(SPEC_BEAM_MAX, MAX_LISTS);
        if (cudaFuncSetAttribute(beam_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 most) != cudaSuccess ||
            cudaFuncSetAttribute(beam_exact_kernel<DT>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess) {
            (void)cudaGetLastError();
            return SPEC_ECUDA;
        }
        g_attr[dev][DT].store(true, std::memory_order_release);
    }
    const size_t merge = merge_bytes(P.a.n, P.a.K * P.segs);
    const int rc = launch(beam_kernel<DT>, (unsigned int)(P.a.B * P.a.K * P.segs),
                          larger(merge, SCAN_BYTES), P, stream);
    return rc != SPEC_OK ? rc : launch(beam_exact_kernel<DT>, EXACT_CTAS, merge, P, stream);
}

}  // namespace

extern "C" {

size_t spec_beam_workspace_size(int32_t B, int32_t K, int32_t V, int32_t n, int32_t dtype)
{
    return sizes_ok(B, K, V, n, dtype) ? beam_layout(B, K, V, n, dtype).total : 0;
}

int32_t spec_beam_select(const spec_beam_select_args *args, void *workspace,
                         size_t workspace_bytes, void *stream)
{
    if (!args)
        return SPEC_EINVAL;
    const spec_beam_select_args &a = *args;
    if (!sizes_ok(a.B, a.K, a.V, a.n, a.dtype) || a.end_token < 0 || a.end_token >= a.V)
        return SPEC_EINVAL;
    if (a.B == 0)
        return SPEC_OK;
    if (!a.logits || !aligned(a.logits, 16) || !a.scores || !aligned(a.scores, 4) ||
        !aligned(a.finished, 4) || !aligned(a.norm, 4) || !a.out_tokens ||
        !aligned(a.out_tokens, 4) || !a.out_beams || !aligned(a.out_beams, 4) || !a.out_scores ||
        !aligned(a.out_scores, 4) || !workspace || !aligned(workspace, 256))
        return SPEC_EINVAL;
    const BeamLayout w = beam_layout(a.B, a.K, a.V, a.n, a.dtype);
    if (workspace_bytes < w.total)
        return SPEC_ENOSPACE;
    if (!outputs_apart(a))
        return SPEC_EINVAL;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    BeamParams P;
    P.a = a;
    P.segs = segments(a.B, a.K, a.V, a.dtype);
    P.chunks = (a.V + RCH - 1) / RCH;
    P.hdr = reinterpret_cast<WsHeader *>(ws);
    P.arrived = reinterpret_cast<int *>(ws + w.arrived);
    P.summed = reinterpret_cast<int *>(ws + w.summed);
    P.listed = reinterpret_cast<int *>(ws + w.listed);
    P.stats = reinterpret_cast<float2 *>(ws + w.stats);
    P.lists = reinterpret_cast<u64 *>(ws + w.lists);
    P.sums = reinterpret_cast<long long *>(ws + w.sums);
    return a.dtype == SPEC_F32 ? select_beams<SPEC_F32>(P, stream)
                               : select_beams<SPEC_BF16>(P, stream);
}

int32_t spec_beam_reorder(const void *in, const int32_t *beams, void *out, int32_t lead,
                          int32_t B, int32_t K, int32_t n, int64_t row_bytes, void *stream)
{
    if (lead < 0 || B < 0 || K < 0 || n < 0 || row_bytes < 0 ||
        (long long)B * n > INT_MAX || (long long)lead * B > INT_MAX ||
        (long long)lead * B * n > INT_MAX || row_bytes > 1ll << 40)
        return SPEC_EINVAL;
    if (lead == 0 || B == 0 || n == 0 || row_bytes == 0)
        return SPEC_OK;
    if (!beams || !aligned(beams, 4) || !out || (K > 0 && !in))
        return SPEC_EINVAL;
    const uintptr_t i0 = reinterpret_cast<uintptr_t>(in), o0 = reinterpret_cast<uintptr_t>(out);
    const uint64_t in_bytes = (uint64_t)lead * B * K * (uint64_t)row_bytes;
    const uint64_t out_bytes = (uint64_t)lead * B * n * (uint64_t)row_bytes;
    if (in && i0 < o0 + out_bytes && o0 < i0 + in_bytes)
        return SPEC_EINVAL;
    const uint64_t bits = i0 | o0 | (uint64_t)row_bytes;
    const int vec = (bits & 15) == 0 ? 16 : (bits & 3) == 0 ? 4 : 1;
    ReorderParams P;
    P.in = in;
    P.out = out;
    P.beams = beams;
    P.rows = (long long)lead * B * n;
    P.per = B * n;
    P.K = K;
    P.n = n;
    P.vecs = row_bytes / vec;
    const long long parts = (P.vecs + PIECE - 1) / PIECE;
    if (parts > INT_MAX)
        return SPEC_EINVAL;
    P.parts = (int)parts;
    const long long ctas = (P.rows * parts + WARPS - 1) / WARPS;
    const unsigned int grid = ctas < 1216 ? (unsigned int)ctas : 1216u;
    if (vec == 16)
        return launch(reorder_kernel<uint4>, grid, 0, P, stream);
    if (vec == 4)
        return launch(reorder_kernel<uint32_t>, grid, 0, P, stream);
    return launch(reorder_kernel<unsigned char>, grid, 0, P, stream);
}

}  // extern "C"
