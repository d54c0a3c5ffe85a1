// spec_logits.cu -- penalties for repeated tokens, biases and grammar masks on
// logits (include/spec_logits.h): one pass that reads each row once and
// writes it once.
//
// A CTA owns one tile of the vocabulary for (some of) the rows of one
// sequence.  It first counts, in shared memory, the tokens of the sequence's
// history that fall in its tile (integer adds: any order gives the same
// count), marks the drafted ones and sums the biases, and keeps one bit per
// column that any of these touched.  The history is read once per tile from
// L2, which costs H * 4 bytes against the tile's 2 * R * C * size from HBM, so
// no table of V counters per sequence has to exist between calls.  A drafted
// token's own count differs from row to row; it is found by walking the row's
// path, for columns marked as drafted.
//
// Bound by HBM: 2 * V * size bytes a row, nearly all of them copied as they are.
// So the copy is bulk copies through a ring of shared-memory stages, one tile of
// one row each.  In the stage the tile's touched columns, listed once, are
// shared out among the threads (found by their vectors' bits instead, the few
// touched ones of a warp took its time one by one, 40 % of the call under
// trees and masks), then a mask forbids what it does, and the stage is stored.
// A bulk copy moves whole 16-byte vectors of the array.  Where V is a multiple
// of the vector that is the tile; other rows start anywhere, their stages hold
// the vectors that the tile reaches into, and the tile's elements in the first
// and last of them are stored one by one.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "spec_logits.h"
#include "spec_verify.h"
#include "device_common.cuh"

namespace {

using namespace spec_dev;

constexpr int LTH = 256;      // threads per CTA
// Tiles of a row in flight per CTA: 24 KB of fp32, 16 of bf16.  A fourth fp32 stage takes
// more from the number of CTAs than it gives (256 x 9 x 151936: 403 us with
// three, 425 with four); bf16 gains by it (64 x 29 x 128256 under masks: 171 us
// with four, 178 with three).
template <int DT>
__host__ __device__ constexpr int stages() { return DT == SPEC_F32 ? 3 : 4; }
constexpr int MOST_STAGES = 4;
constexpr int MOST_C = 2048;  // columns of a tile, fewer where there would be few CTAs
constexpr int HUN = 8;        // history tokens in flight per thread
constexpr uint32_t IN_PROMPT = 0x80000000u;  // flags of a column's word; the rest is its count
constexpr uint32_t DRAFTED = 0x40000000u;    // in the generated part of the history
constexpr uint32_t COUNT = 0x3fffffffu;
constexpr uint32_t NO_BIAS = 0x80000000u;    // a column's bias without an entry: -0, which adds nothing

struct LParams {
    spec_process_logits_args a;
    int C;             // columns per tile, a multiple of 32
    int rows_per_cta;
    uint32_t list_at, ring_at;  // byte offsets in shared memory, multiples of 16
};

// shared memory: count words [C] | touched bits [C / 32] | bits of columns with several
// biases [C / 32] | bias [C] (when
// there are biases) | drafted tokens [R] | parents [R] (tree) | touched columns [C] |
// stages [stages][C + a vector]
struct LSmem {
    uint32_t *cnt, *touched, *again;
    float *bias;
    int *tok, *par;
};

template <int DT>
__device__ __forceinline__ uint32_t round_bits(float y)
{
    if (DT == SPEC_F32)
        return __float_as_uint(y);
    return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(y));
}

__device__ __forceinline__ void bulk_copy_s2g(void *dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\t"
                 "cp.async.bulk.commit_group;"
                 :: "l"(dst), "r"(smem_addr(src)), "r"(bytes) : "memory");
}

struct Penalty {
    float rep, freq, pres;
};

// Changes logit x of row r at a touched column c of the tile; false where only other rows
// touch it (a token drafted on their paths), and it keeps its bits.
__device__ bool touch(const spec_process_logits_args &A, const LSmem &S, int t0, int c, int r,
                      float &x, const Penalty &pen)
{
    const uint32_t w = S.cnt[c];
    int n = (int)(w & COUNT);
    if (w & DRAFTED) {
        const int token = t0 + c;
        if (A.parent) {
            // (every parent has been found below its node, so at most r steps)
            for (int i = r, left = r; i > 0 && left > 0; i = S.par[i], --left)
                n += S.tok[i] == token;
        } else {
            for (int i = 0; i < r; ++i)
                n += S.tok[i] == token;
        }
    }
    const float bias = S.bias ? S.bias[c] : __uint_as_float(NO_BIAS);
    const bool seen = n > 0 || (w & IN_PROMPT);
    if (seen)
        x = x > 0.0f ? x / pen.rep : x * pen.rep;
    if (n > 0) {
        x -= pen.freq * (float)n;
        x -= pen.pres;
    }
    x += bias;
    return seen || __float_as_uint(bias) != NO_BIAS;
}

// -inf where the bits of `ok` are 0
template <int DT>
__device__ __forceinline__ void forbid(uint4 &raw, uint32_t ok)
{
    uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (DT == SPEC_F32) {
            w[i] = (ok >> i) & 1u ? w[i] : 0xff800000u;
        } else {
            const uint32_t keep = ((ok >> (2 * i)) & 1u ? 0xffffu : 0u) |
                                  ((ok >> (2 * i + 1)) & 1u ? 0xffff0000u : 0u);
            w[i] = (w[i] & keep) | (0xff80ff80u & ~keep);
        }
    }
    raw = make_uint4(w[0], w[1], w[2], w[3]);
}

// ALIGNED: V is a multiple of the vector.
template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(LTH) logits_kernel(const __grid_constant__ LParams P)
{
    using L = Lg<DT>;
    constexpr int STAGES = stages<DT>();
    extern __shared__ __align__(16) uint32_t lsm[];
    const spec_process_logits_args &A = P.a;
    const int tid = (int)threadIdx.x;
    const int b = (int)blockIdx.y;
    const int t0 = (int)blockIdx.x * P.C;
    const int cols = min(P.C, A.V - t0);
    LSmem S;
    S.cnt = lsm;
    S.touched = S.cnt + P.C;
    S.again = S.touched + P.C / 32;
    float *fb = reinterpret_cast<float *>(S.again + P.C / 32);
    S.bias = A.bias_cols > 0 ? fb : nullptr;
    S.tok = reinterpret_cast<int *>(fb + (A.bias_cols > 0 ? P.C : 0));
    S.par = S.tok + A.R;

    wait_previous_kernel();
    for (int i = tid; i < P.C + 2 * (P.C / 32); i += LTH)
        lsm[i] = 0;
    if (S.bias)
        for (int i = tid; i < P.C; i += LTH)
            S.bias[i] = __uint_as_float(NO_BIAS);

    Penalty pen;
    pen.rep = A.repetition ? A.repetition[b] : 1.0f;
    pen.freq = A.frequency ? A.frequency[b] : 0.0f;
    pen.pres = A.presence ? A.presence[b] : 0.0f;
    const int hl = A.H > 0 ? A.history_len[b] : 0;
    const int pl = A.H > 0 ? A.prompt_len[b] : 0;
    int nn = A.n_nodes ? A.n_nodes[b] : A.R;
    bool bad = !(pen.rep > 0.0f) || isinf(pen.rep) || !isfinite(pen.freq) ||
               !isfinite(pen.pres) || pl < 0 || hl < pl || hl > A.H || nn < 1 || nn > A.R;
    if (nn < 1 || nn > A.R)
        nn = A.R;
    const int r0 = (int)blockIdx.z * P.rows_per_cta;
    const int rows = min(nn, r0 + P.rows_per_cta) - r0;
    if (rows <= 0)
        return;
    __shared__ __align__(8) unsigned long long full[STAGES];
    __shared__ int listed;          // touched columns
    __shared__ volatile int stuck;  // a copy's wait gave up
    // Row r of the CTA: its tile's first element in the array, how far into a vector it
    // lies, and the tile's whole vectors of the array (the array's last, broken one is not)
    uint8_t *ring = reinterpret_cast<uint8_t *>(lsm) + P.ring_at;
    const uint32_t stage_bytes = (uint32_t)(P.C + L::VEC) * L::ES;
    auto first_of = [&](int r) -> size_t { return ((size_t)b * A.R + r0 + r) * A.V + t0; };
    auto shift_of = [&](int r) -> int { return ALIGNED ? 0 : (int)(first_of(r) % L::VEC); };
    auto vectors_of = [&](int r) -> int {
        if (ALIGNED)
            return cols / L::VEC;
        const size_t v0 = first_of(r) / L::VEC, all = (size_t)A.B * A.R * A.V / L::VEC;
        const int want = (shift_of(r) + cols + L::VEC - 1) / L::VEC;
        return v0 + want <= all ? want : (int)(all - v0);
    };
    auto load_row = [&](int r) {  // one thread
        const int st = r % STAGES;
        const uint32_t bytes = (uint32_t)vectors_of(r) * 16;
        mbar_arrive_expect_tx(&full[st], bytes);
        if (bytes > 0)
            bulk_copy_g2s(ring + st * stage_bytes,
                          static_cast<const uint8_t *>(A.logits) + first_of(r) / L::VEC * 16,
                          bytes, &full[st]);
    };
    if (tid == 0) {
        listed = 0;
        stuck = 0;
        for (int st = 0; st < STAGES; ++st)
            mbar_init(&full[st], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        for (int r = 0; r < STAGES && r < rows; ++r)
            load_row(r);
    }
    __syncthreads();

    const int32_t *bt = A.bias_tokens + (size_t)b * A.bias_cols;
    const float *bv = A.bias_values + (size_t)b * A.bias_cols;
    // the history's tokens of this tile
    if (!bad) {
        const int32_t *hist = A.history + (size_t)b * A.H;
        for (int i0 = tid; i0 < hl; i0 += HUN * LTH) {
            int tok[HUN];
#pragma unroll
            for (int u = 0; u < HUN; ++u)
                tok[u] = i0 + u * LTH < hl ? __ldg(hist + i0 + u * LTH) : t0 + cols;
#pragma unroll
            for (int u = 0; u < HUN; ++u) {
                const int i = i0 + u * LTH, c = tok[u] - t0;
                bad |= (tok[u] < 0 || tok[u] >= A.V) && i < hl;
                if (c >= 0 && c < cols) {
                    if (i < pl)
                        atomicOr(&S.cnt[c], IN_PROMPT);
                    else
                        atomicAdd(&S.cnt[c], 1u);
                    atomicOr(&S.touched[c >> 5], 1u << (c & 31));
                }
            }
        }
        // drafted tokens: a chain's token i follows row i, a tree's belongs to node i
        const int first = A.parent ? 1 : 0;
        const int last = A.parent ? nn : min(nn - 1, A.draft_cols);
        if (A.draft_cols > 0)
            for (int i = first + tid; i < last; i += LTH) {
                const int t = A.draft_tokens[(size_t)b * A.draft_cols + i];
                bad |= t < 0 || t >= A.V;
                S.tok[i] = t;
                if (A.parent) {
                    const int p = A.parent[(size_t)b * A.R + i];
                    bad |= p < 0 || p >= i;
                    S.par[i] = p;
                }
                const int c = t - t0;
                if (c >= 0 && c < cols) {
                    atomicOr(&S.cnt[c], DRAFTED);
                    atomicOr(&S.touched[c >> 5], 1u << (c & 31));
                }
            }
        // biases: entry i bids bias_cols - i for its column, so the first one wins
        for (int i = tid; i < A.bias_cols; i += LTH) {
            const int t = bt[i];
            bad |= t < -1 || t >= A.V;
            const int c = t - t0;
            if (t < 0 || c < 0 || c >= cols)
                continue;
            if (atomicMax(reinterpret_cast<int *>(&S.bias[c]), A.bias_cols - i) > 0)
                atomicOr(&S.again[c >> 5], 1u << (c & 31));
            atomicOr(&S.touched[c >> 5], 1u << (c & 31));
        }
    }
    bad = __syncthreads_or(bad ? 1 : 0) != 0;
    if (A.bias_cols > 0) {
        uint32_t won = 0;  // which of the thread's entries
        if (!bad)
            for (int i = tid, k = 0; i < A.bias_cols; i += LTH, ++k) {
                const int c = bt[i] - t0;
                if (bt[i] >= 0 && c >= 0 && c < cols &&
                    __float_as_int(S.bias[c]) == A.bias_cols - i)
                    won |= 1u << k;
            }
        __syncthreads();
        // the first entry of a token sums all of its entries in order
        for (int i = tid; won; i += LTH, won >>= 1) {
            if (!(won & 1u))
                continue;
            const int t = bt[i], c = t - t0;
            float sum = bv[i];
            if ((S.again[c >> 5] >> (c & 31)) & 1u)
                for (int j = i + 1; j < A.bias_cols; ++j)
                    if (bt[j] == t)
                        sum += bv[j];
            S.bias[c] = sum;
        }
    }

    // the touched columns, in any order: each is worked out by itself
    uint16_t *list = reinterpret_cast<uint16_t *>(reinterpret_cast<uint8_t *>(lsm) + P.list_at);
    for (int c = tid; c < cols; c += LTH)
        if ((S.touched[c >> 5] >> (c & 31)) & 1u)
            list[atomicAdd(&listed, 1)] = (uint16_t)c;
    constexpr uint32_t ALL = (1u << L::VEC) - 1u;
    constexpr int VPT = MOST_C / L::VEC / LTH + (ALIGNED ? 0 : 1);  // a thread's vectors of a row
    // The mask words that their elements' bits lie in, loaded a row ahead and not looked at
    // before (a second word where vectors lie anywhere).
    uint32_t next_lo[VPT], next_hi[VPT];
    auto load_mask = [&](int r) {
        const uint32_t *mask = A.allowed + b * A.allowed_stride_b + (r0 + r) * A.allowed_stride_r;
        const int mis = shift_of(r);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = (tid + k * LTH) * L::VEC - mis, w = (t0 + max(c, 0)) >> 5;
            next_lo[k] = c < cols ? __ldg(mask + w) : ~0u;
            if (!ALIGNED)
                next_hi[k] = c < cols && w < (A.V - 1) >> 5 ? __ldg(mask + w + 1) : ~0u;
        }
    };
    if (A.allowed)
        load_mask(0);
    __syncthreads();
    const int n_listed = bad ? 0 : listed;
    for (int r = 0; r < rows; ++r) {
        const int st = r % STAGES;
        if (!mbar_wait(&full[st], (uint32_t)(r / STAGES) & 1u))
            stuck = 1;
        uint8_t *stage = ring + st * stage_bytes;
        const int mis = shift_of(r), have = vectors_of(r) * L::VEC - mis;
        if (!ALIGNED && have < cols) {
            // the array's last elements, past its last whole vector
            for (int c = max(have, 0) + tid; c < cols; c += LTH) {
                if (DT == SPEC_F32)
                    reinterpret_cast<uint32_t *>(stage)[c + mis] =
                        reinterpret_cast<const uint32_t *>(A.logits)[first_of(r) + c];
                else
                    reinterpret_cast<unsigned short *>(stage)[c + mis] =
                        reinterpret_cast<const unsigned short *>(A.logits)[first_of(r) + c];
            }
            __syncthreads();
        }
        for (int i = tid; i < n_listed; i += LTH) {
            const int c = list[i];
            if (DT == SPEC_F32) {
                float *at = reinterpret_cast<float *>(stage) + c + mis, x = *at;
                if (touch(A, S, t0, c, r0 + r, x, pen))
                    *at = x;
            } else {
                unsigned short *at = reinterpret_cast<unsigned short *>(stage) + c + mis;
                float x = __uint_as_float((uint32_t)*at << 16);
                const unsigned short was = *at;  // (stored back: to skip the store took 1 % more)
                const bool on = touch(A, S, t0, c, r0 + r, x, pen);
                *at = on ? (unsigned short)round_bits<DT>(x) : was;
            }
        }
        if (bad) {
            for (int v = tid; v * L::VEC - mis < cols; v += LTH)
                reinterpret_cast<uint4 *>(stage)[v] =
                    make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
        } else if (A.allowed) {
            uint32_t ok[VPT];  // (elements outside the tile are not stored, whatever becomes of them)
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = (tid + k * LTH) * L::VEC - mis, lo = max(c, 0);
                if (ALIGNED)
                    ok[k] = (next_lo[k] >> ((t0 + c) & 31)) & ALL;
                else
                    ok[k] = (__funnelshift_r(next_lo[k], next_hi[k], (t0 + lo) & 31) << (lo - c)) &
                            ALL;
            }
            if (r + 1 < rows)
                load_mask(r + 1);
            if (n_listed > 0)
                __syncthreads();
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int v = tid + k * LTH;
                if (v * L::VEC - mis >= cols || ok[k] == ALL)
                    continue;
                uint4 *at = reinterpret_cast<uint4 *>(stage) + v;
                uint4 raw = *at;
                forbid<DT>(raw, ok[k]);
                *at = raw;
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
        if (stuck) {
            // a copy never came: the rest is marked like a bad sequence's
            for (int c = tid; c < cols; c += LTH)
                for (int y = r; y < rows; ++y) {
                    if (DT == SPEC_F32)
                        reinterpret_cast<uint32_t *>(A.out)[first_of(y) + c] = 0x7fff7fffu;
                    else
                        reinterpret_cast<unsigned short *>(A.out)[first_of(y) + c] = 0x7fffu;
                }
            break;
        }
        // the vectors that are the tile's alone, and its elements in the others
        const int v0 = mis ? 1 : 0, v1 = (mis + cols) / L::VEC;
        if (!ALIGNED && tid < 2 * L::VEC) {
            const int c = tid < L::VEC ? tid : cols - 1 - (tid - L::VEC);
            if (c >= 0 && c < cols && (c + mis < v0 * L::VEC || c + mis >= v1 * L::VEC)) {
                if (DT == SPEC_F32)
                    reinterpret_cast<uint32_t *>(A.out)[first_of(r) + c] =
                        reinterpret_cast<const uint32_t *>(stage)[c + mis];
                else
                    reinterpret_cast<unsigned short *>(A.out)[first_of(r) + c] =
                        reinterpret_cast<const unsigned short *>(stage)[c + mis];
            }
        }
        if (tid == 0) {
            if (v1 > v0)
                bulk_copy_s2g(static_cast<uint8_t *>(A.out) +
                                  (first_of(r) / L::VEC + (size_t)v0) * 16,
                              stage + v0 * 16, (uint32_t)(v1 - v0) * 16);
            else  // (a group all the same: they are counted)
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            // the stage of the row before is free once its store has read it
            if (r > 0 && r - 1 + STAGES < rows) {
                asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                load_row(r - 1 + STAGES);
            }
        }
    }
    if (tid == 0) {
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        if (stuck)  // copies still in flight end first (bounded)
            for (int st = 0; st < STAGES; ++st)
                (void)mbar_wait(&full[st], 0u), (void)mbar_wait(&full[st], 1u);
    }
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

size_t smem_bytes(const spec_process_logits_args &a, int C)
{
    return (4 * ((size_t)C + 2 * (C / 32) + (a.bias_cols > 0 ? C : 0) + 2 * (size_t)a.R) + 15) / 16 * 16;
}

// the largest tile's words, bits, biases, drafts, list and fp32 stages
constexpr size_t MOST_SMEM =
    4 * (MOST_C + 2 * (MOST_C / 32) + MOST_C + 2 * SPEC_LOGITS_MAX_ROWS) + 16 + MOST_C * 2 +
    (size_t)MOST_STAGES * (MOST_C * 4 + 16);
static_assert(MOST_SMEM <= 232448 - 64, "227 KB per CTA");
static_assert(SPEC_LOGITS_MAX_BIAS <= 32 * LTH, "a thread's bias entries in one word");
std::atomic<bool> g_attr[64][2][2];  // opted in, per device, dtype and alignment

template <int DT, bool ALIGNED>
int launch(const LParams &P, dim3 grid, cudaStream_t st)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return SPEC_ECUDA;
    if (!g_attr[dev][DT][ALIGNED].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(logits_kernel<DT, ALIGNED>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)MOST_SMEM) != cudaSuccess)
            return SPEC_ECUDA;
        g_attr[dev][DT][ALIGNED].store(true, std::memory_order_release);
    }
    const size_t stage = (size_t)(P.C + Lg<DT>::VEC) * Lg<DT>::ES;
    logits_kernel<DT, ALIGNED><<<grid, LTH, P.ring_at + stages<DT>() * stage, st>>>(P);
    return SPEC_OK;
}

}  // namespace

extern "C" int32_t spec_process_logits(const spec_process_logits_args *args, void *stream)
{
    if (!args)
        return SPEC_EINVAL;
    const spec_process_logits_args &a = *args;
    if (a.B < 0 || a.B > 65535 || a.R < 1 || a.R > SPEC_LOGITS_MAX_ROWS || a.V < 2 ||
        a.V > SPEC_MAX_V || a.H < 0 || a.H > (1 << 24) || a.bias_cols < 0 ||
        a.bias_cols > SPEC_LOGITS_MAX_BIAS || (a.dtype != SPEC_F32 && a.dtype != SPEC_BF16) ||
        a.allowed_stride_b < 0 || a.allowed_stride_r < 0)
        return SPEC_EINVAL;
    if (a.B == 0)
        return SPEC_OK;
    if (!a.logits || !a.out || !aligned(a.logits, 16) || !aligned(a.out, 16))
        return SPEC_EINVAL;
    const void *words[] = {a.history, a.history_len, a.prompt_len, a.draft_tokens, a.parent,
                           a.n_nodes, a.repetition, a.frequency, a.presence, a.bias_tokens,
                           a.bias_values, a.allowed};
    for (const void *p : words)
        if (!aligned(p, 4))
            return SPEC_EINVAL;
    if ((a.H > 0 && (!a.history || !a.history_len || !a.prompt_len)) ||
        (a.bias_cols > 0 && (!a.bias_tokens || !a.bias_values)))
        return SPEC_EINVAL;
    if (a.parent ? (a.draft_cols != a.R)
                 : (a.draft_cols != 0 && a.draft_cols != a.R && a.draft_cols != a.R - 1))
        return SPEC_EINVAL;
    if (a.draft_cols > 0 && !a.draft_tokens)
        return SPEC_EINVAL;

    LParams P;
    P.a = a;
    P.C = MOST_C;
    auto tiles = [&] { return (long long)a.B * ((a.V + P.C - 1) / P.C); };
    while (P.C > 1024 && tiles() < 304)
        P.C /= 2;
    int splits = 1;
    while (tiles() * splits < 304 && splits < a.R)
        splits *= 2;
    P.rows_per_cta = (a.R + splits - 1) / splits;
    const size_t smem = smem_bytes(a, P.C);  // at most 25 KB, a list of 4 and a ring of 24
    P.list_at = (uint32_t)smem;
    P.ring_at = P.list_at + (uint32_t)P.C * 2;
    const dim3 grid((unsigned int)((a.V + P.C - 1) / P.C), (unsigned int)a.B,
                    (unsigned int)((a.R + P.rows_per_cta - 1) / P.rows_per_cta));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    int rc;
    if (a.dtype == SPEC_F32)
        rc = a.V % 4 == 0 ? launch<SPEC_F32, true>(P, grid, st) : launch<SPEC_F32, false>(P, grid, st);
    else
        rc = a.V % 8 == 0 ? launch<SPEC_BF16, true>(P, grid, st) : launch<SPEC_BF16, false>(P, grid, st);
    if (rc != SPEC_OK) {
        (void)cudaGetLastError();
        return rc;
    }
    if (cudaPeekAtLastError() != cudaSuccess) {
        (void)cudaGetLastError();
        return SPEC_ECUDA;
    }
    return SPEC_OK;
}
