// spec_attn.cu -- tree attention over a key/value cache on the tcgen05 tensor
// cores (include/spec_attn.h).
//
// For one sequence and one key/value head all query rows that share the head
// (every node of the tree times the Hq / Hkv heads of the group) form the
// rows of a tile of 128: S = Q K^T over 128 keys at a time, a running softmax
// per row, O += P V.  Keys and values are then read once for all rows, which
// is what bounds the kernel: D * 4 bytes per key and head from HBM against
// 4 * D * 128 operations at any number of rows up to 128.  A tile of 64 KB
// takes an SM's share of the HBM rate about 2850 clocks, its two products
// about 1030 and its exponentials 512, so up to 128 rows the products' cost is
// covered whatever part of the rows is in use, and single tokens use the same
// kernel.  More rows are several row tiles (whole nodes each), taken in pairs.
//
// Roles in a CTA (one per SM, 3 warpgroups; the third gives registers to the others):
//   warps 0-3, 4-7  two softmax groups, one thread per row.  Group s takes the
//                   tiles of its parity with scores, weights and sums of its
//                   own (S_s, O_s in TMEM), so that one group's exponentials
//                   run under the other's products.  The weights go back to
//                   TMEM in the place of the scores, as the A operand of P V.
//                   The two groups' sums are joined when the piece ends.
//   warp 8          TMA of the K and V tiles, each a ring of stages; pages
//                   smaller than a tile are boxes of one tile
//   warp 9          issues the products in order: S(i) first two, then
//                   O(i), S(i + 2), ...; a commit behind S(i + 2) so also
//                   says that O(i) is done.  With two row tiles: S(0) of
//                   each, then O(i), S(i + 1) of the one and of the other
//   warp 10         TMA of an item's Q
//   warp 11         walks the CTA's share and hands the pieces of it out
//                   through a small ring: what a piece is costs several
//                   dependent loads, which would stall every role at each item
// TMEM: S_0, S_1 (128 columns each), O_0, O_1 (up to 128 each).
//
// A row's sums are rescaled only when its maximum has grown by more than 2^8
// (2^4 with fp16 weights) since the last time (all of the statistics are fp32,
// so the larger weights in between lose nothing); most tiles then leave O in
// TMEM alone.
//
// Work: the key tiles of all sequences, heads and row groups that hold a node (a
// row tile, or a pair) stand in a line and are dealt to the CTAs in equal runs,
// whatever the lengths and the numbers of nodes.  An
// item (sequence, head, row group) that lies in one CTA's run is written by it; of a
// split item each CTA leaves its unnormalised sums with their maximum and
// total in the workspace, and a second kernel joins them in order, so repeats
// are bit-equal.  No CTA waits for another.
//
// What a row must not see: scores of masked keys are replaced, not added to,
// so NaN keys have no effect.  A value of a masked key does enter P V with
// weight 0, and 0 * NaN is NaN: rows of V past the length are zeroed in shared
// memory, and non-finite elements of new values (which other rows may see)
// are taken out there and added back row by row, where the mask has them.
//
// Every mbarrier wait is bounded; one that gives up sets
// SPEC_DEV_WAIT_TIMEOUT and the CTA's abort flag, after which no role waits
// or issues any more.  When all have ended, the loads and products in flight
// land (bounded again), the rows of the CTA's share become NaN, which the
// verification reports, and TMEM is freed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "spec_attn.h"
#include "spec_bench.h"
#include "spec_verify.h"
#include "attn_plan.cuh"
#include "device_common.cuh"

namespace {

using namespace spec_dev;
using namespace spec_attn;

constexpr int BM = 128;           // rows of a tile (TMEM lanes)
constexpr int PANEL = 64;         // elements of a 128-byte swizzled row
constexpr int PANEL_BYTES = 128 * 128;  // 128 rows (or keys) of one panel
constexpr int SOFT_THREADS = 256;
constexpr int THREADS = SOFT_THREADS + 128;
// 384 threads launch with 168 registers each, 64512; a softmax thread holds a
// row's 128 scores: 256 * 208 + 128 * 88 = 64512
constexpr int SOFT_REGS = 208, HELPER_REGS = 88;
constexpr int MAX_CTAS = 192;     // the grid's and the workspace's bound
constexpr int RING = 4;           // pieces handed out ahead
// log2 of how far a maximum may run ahead of the sums' scale, and of the weight that the scale gives
// it.  bf16 weights have fp32's exponents.  fp16 ones lose bits below 2^-14 and vanish below
// 2^-25, so their scale puts the maximum at 2^11 (2^15 ahead of the scale): weights keep all of
// their bits down to 2^-25 of it, where with 2^0 they had vanished while the total
// counted them.  The constant cancels in the division; it and the earlier rescaling cost nothing
// to speak of (4 trees of up to 256 nodes over up to 16384 positions in fp16: 279 to 280 us).
template <int DT>
__host__ __device__ constexpr float growth() { return DT == SPEC_BF16 ? 8.0f : 4.0f; }
template <int DT>
__host__ __device__ constexpr float lift() { return DT == SPEC_BF16 ? 0.0f : 11.0f; }

// PAIR: a CTA has two row tiles, one for each softmax group, over the same keys.
template <int NP, bool PAIR>
struct Cfg {
    // 160 KB (D > 64, pairs) or 192 KB of K and V in flight or in use: an SM's share of
    // HBM needs about 35 KB in flight
    static constexpr int Q_TILES = PAIR ? 2 : 1;
    static constexpr int KST = NP == 2 ? 3 : 6;
    static constexpr int VST = NP == 2 ? (PAIR ? 2 : 3) : 6;
    static constexpr int TILE = NP * PANEL_BYTES;
    static constexpr int DP = NP * PANEL;  // columns of O
};
// Stages are taken in the order of the CTA's tiles.  A wait for a phase of a
// barrier tells it from the phase before only if that one is known to be over
// (parity), so whoever waits on a stage has gone through its earlier phases: the
// loader and the issuer wait for all of them, and a softmax group that looks
// at V waits for its tile's scores first, which the issuer's products of
// every earlier tile precede.


// A run of one item's key tiles inside a CTA's share.
struct Piece {
    int b, h;
    int rt0;         // first row tile
    int last;        // 1 in the sequence's last row group that holds a node
    int tile0, n;    // first tile and number of tiles (0: the share has ended)
    int tiles;       // of the whole item
    int len, nn;     // cache length and nodes
    int status;
    int idle;        // nothing to compute: no node, or a bad sequence
    int first;       // 1 when the share starts inside the item or with it
};

struct Tail {
    unsigned long long kfull[6], kempty[6], vfull[6], vempty[6];
    unsigned long long qfull, qempty, sfull[2], pready[2], pvdone[2], drain;
    unsigned long long pfull[RING], pempty[RING], join, noted[2];
    Piece piece[RING];
    uint32_t tmem_base;
    int abort_flag;
    uint32_t loaded[3];  // loads that were issued when their warp ended: tiles of K, of V, and Qs
    uint32_t bad[2][2][4];  // keys of a group's tile (alternating) whose values are not all finite
    float m[2][BM], l[2][BM];
};

template <int NP, bool PAIR>
constexpr size_t smem_bytes()
{
    using C = Cfg<NP, PAIR>;
    return (size_t)C::TILE * (C::Q_TILES + C::KST + C::VST) + sizeof(Tail);
}
static_assert(smem_bytes<2, false>() <= 232448 && smem_bytes<1, false>() <= 232448 &&
              smem_bytes<2, true>() <= 232448 && smem_bytes<1, true>() <= 232448,
              "227 KB per CTA");

struct AParams {
    const uint8_t *plan;
    PlanLayout lay;
    const int32_t *page_table;
    const void *v_new;
    int64_t v_new_stride[3];
    void *out;
    float *lse;
    int *status;
    float *part;     // [ctas][Q_TILES][2][DP][BM] unnormalised sums of split items
    float2 *part_ml; // [ctas][Q_TILES][2][BM] (log2 of the weights' unit, total)
    float c;         // scale * log2(e)
    int B, N, Hq, Hkv, D, G;
    int nodes_per_tile;
    int slots;       // CTAs
    int join_rows;   // rows of a join CTA: 32, or the least power of two that holds them
    int page_size, pages_per_seq;
    int page_rows;   // rows of a cache box: min(128, page_size) (contiguous: 128)
    int new_rows;    // rows of a box of new tokens
    int q_rows;      // rows of the Q box
    int lose, lose_after;  // the self-test's CTA (-1: none) and the pieces that it hands out first
};

// ------------------------------------------------------------ PTX wrappers

// 16 consecutive columns of this warp's 32 TMEM lanes, one lane per thread; they have
// arrived when it returns
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16])
{
    __syncwarp();  // .sync.aligned: the whole warp, converged
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15 "
        "}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr) : "memory");
}

// 32 consecutive columns of this warp's 32 TMEM lanes, one lane per thread; they have
// arrived when it returns
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32])
{
    __syncwarp();  // .sync.aligned: the whole warp, converged
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31 "
        "}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr) : "memory");
}

// 32 columns in two halves: the load runs while the code between them does
__device__ __forceinline__ void tmem_ld_start(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31 "
        "}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_finish(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
          "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
          "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]),
          "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
          "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
        :: "memory");
}

__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[16])
{
    __syncwarp();
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {"
        "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16 "
        "};"
        :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
          "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[32])
{
    __syncwarp();
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {"
        "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32 "
        "};"
        :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
          "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
          "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
          "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_async_shared()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, int w, unsigned long long *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w),
           "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, int w, int v, unsigned long long *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w),
           "r"(v), "r"(smem_addr(bar))
        : "memory");
}

// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void mma_commit(unsigned long long *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
        :: "r"(smem_addr(bar)) : "memory");
}

// one lane of a converged warp, always the same one
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// A converged warp's test of a barrier, by one elected lane and without a branch: a test
// by all 32 lanes is served one after the other (150 to 250 clocks for a
// barrier that is ready), and a branch to one lane's test costs about as much.
__device__ __forceinline__ bool warp_try(unsigned long long *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "setp.ne.u32 q, %2, %2;\n\t"
        "@p mbarrier.try_wait.parity.shared::cta.b64 q, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    const bool any = __any_sync(0xffffffffu, ok != 0);
    __syncwarp();
    return any;
}

// The same for two barriers at once.
__device__ __forceinline__ bool warp_try2(unsigned long long *a, uint32_t pa,
                                          unsigned long long *b, uint32_t pb)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q, r;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "setp.ne.u32 q, %2, %2;\n\t"
        "setp.ne.u32 r, %2, %2;\n\t"
        "@p mbarrier.try_wait.parity.shared::cta.b64 q, [%1], %2;\n\t"
        "@p mbarrier.try_wait.parity.shared::cta.b64 r, [%3], %4;\n\t"
        "and.pred q, q, r;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(a)), "r"(pa), "r"(smem_addr(b)), "r"(pb)
        : "memory");
    const bool any = __any_sync(0xffffffffu, ok != 0);
    __syncwarp();
    return any;
}

// Tests of a barrier before a wait gives up.  A test that fails takes 50 ns at least (the
// hardware holds it a while), so this is 0.2 s at least and seconds at most.
constexpr int WAIT_TRIES = 1 << 22;
constexpr int LOSE_TRIES = 1 << 6;  // the self-test's

__device__ __forceinline__ void give_up(volatile int *abort_flag, int *status)
{
    atomicExch(status, SPEC_DEV_WAIT_TIMEOUT);
    *abort_flag = 1;
}

// Shared-memory matrix descriptors, 128-byte swizzle (version 1, mode 2).
// K-major (Q and K): rows of 128 bytes, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// MN-major (V: its 64-element panels run along N, its keys along K): panels
// PANEL_BYTES apart (leading offset), groups of 8 keys 1024 bytes apart (stride).
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(PANEL_BYTES >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Instruction descriptor, kind::f16: fp32 accumulator, A and B both bf16 (1)
// or both fp16 (0), M = 128.
template <int DT>
__host__ __device__ constexpr uint32_t idesc(int n, bool b_mn_major)
{
    constexpr uint32_t T = DT == SPEC_BF16 ? 1u : 0u;
    return (1u << 4) | (T << 7) | (T << 10) | ((b_mn_major ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
}

__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b,
                                                   unsigned long long c)
{
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

template <int DT>
__device__ __forceinline__ uint32_t pack(float lo, float hi)
{
    if (DT == SPEC_BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <int DT>
__device__ __forceinline__ float unpack1(uint32_t half)
{
    if (DT == SPEC_BF16)
        return __uint_as_float(half << 16);
    return __half2float(__ushort_as_half((unsigned short)half));
}

// which halves of a word are NaN or infinite, as masks of 16 bits
template <int DT>
__device__ __forceinline__ uint32_t nonfinite(uint32_t w)
{
    constexpr uint32_t E = DT == SPEC_BF16 ? 0x7f80u : 0x7c00u;
    return ((w & E) == E ? 0xffffu : 0u) | (((w >> 16) & E) == E ? 0xffff0000u : 0u);
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// the largest of 32 scores (two chains); -inf if all are NaN
__device__ __forceinline__ float max32(const uint32_t (&x)[32])
{
    float a = -INFINITY, b = -INFINITY;
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
        a = max3(a, __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
        b = max3(b, __uint_as_float(x[j + 2]), __uint_as_float(x[j + 3]));
    }
    return fmaxf(a, b);
}

// scores with a 0 bit become -inf
__device__ __forceinline__ void hide(uint32_t (&x)[32], uint32_t bits)
{
#pragma unroll
    for (int j = 0; j < 32; ++j)
        x[j] = (int)(bits << (31 - j)) < 0 ? x[j] : 0xff800000u;
}

// weights 2^(x c + shift) of 32 scores, packed, and their sum added to `sum`.  They are rounded
// to the dtype because the product's two operands have one type, and V's is that; the total keeps
// fp32.  Outputs are then 2.3e-3 from 64 bits in bf16 and 2.8e-4 in fp16 (2-norm), where fp32
// weights and one rounding of the result give 1.7e-3 and 2.1e-4.
template <int DT>
__device__ __forceinline__ void weigh(const uint32_t (&x)[32], unsigned long long c2,
                                      unsigned long long shift2, unsigned long long (&sum)[2],
                                      uint32_t (&pk)[16])
{
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        float a0, a1;
        f2_split(fma2(f2_bits(x[2 * j], x[2 * j + 1]), c2, shift2), a0, a1);
        a0 = ex2(a0);
        a1 = ex2(a1);
        sum[j & 1] = add2(sum[j & 1], f2(a0, a1));
        pk[j] = pack<DT>(a0, a1);
    }
}

// ------------------------------------------------------------------- work

// Where a unit lies: its sequence, that sequence's first unit, its key tiles and
// row groups.
struct Place {
    int b;
    long long first;
    int tiles, groups;
    uint4 seq;       // the plan's PlanSeq
};

template <bool PAIR>
__device__ __forceinline__ int row_groups_of(const AParams &P, int nn)
{
    const int per = P.nodes_per_tile * 2;
    return PAIR && nn > per ? (nn + per - 1) / per : 1;
}

// The place of sequence b whose first unit is `first`.
template <bool PAIR>
__device__ __forceinline__ Place place_at(const AParams &P, int b, long long first)
{
    const long long *cum = reinterpret_cast<const long long *>(P.plan + P.lay.cum);
    Place q;
    q.b = b;
    q.first = first;
    q.tiles = (int)(__ldg(cum + b + 1) - __ldg(cum + b));
    q.seq = __ldg(reinterpret_cast<const uint4 *>(P.plan + P.lay.seq) + b);
    q.groups = row_groups_of<PAIR>(P, (int)q.seq.y);
    return q;
}

// A warp looks up one unit: `pick` makes it of the number of all units, and where that lies goes to
// q (not if it is past the end).  Up to 32 sequences take one round of loads, their units
// summed over the lanes; more of them a search of the plan's prefix sums with 32 probes a
// round, or, where row groups make those sums useless, two passes over the sequences.
template <bool PAIR, typename F>
__device__ __forceinline__ long long look_up(const AParams &P, F pick, long long &total, Place &q)
{
    const long long *cum = reinterpret_cast<const long long *>(P.plan + P.lay.cum);
    const int lane = (int)threadIdx.x & 31;
    if (!PAIR && P.B > 32) {
        total = __ldg(cum + P.B) * P.Hkv;
        const long long u = pick(total);
        if (u >= total)
            return u;
        int lo = 0, len = P.B;
        while (len > 1) {
            const int step = (len + 31) / 32, at = lane * step;
            const bool below = at < len && __ldg(cum + lo + at) * P.Hkv <= u;
            const int last = 31 - __clz((int)__ballot_sync(0xffffffffu, below));
            lo += last * step;
            len = len - last * step < step ? len - last * step : step;
        }
        q = place_at<PAIR>(P, lo, __ldg(cum + lo) * P.Hkv);
        return u;
    }
    long long u = -1;
    for (int pass = 0; pass < 2; ++pass) {
        long long before = 0;
        for (int b0 = 0; b0 < P.B; b0 += 32) {
            long long v = 0;
            Place mine = {};
            if (b0 + lane < P.B) {
                mine = place_at<PAIR>(P, b0 + lane, 0);
                v = (long long)mine.tiles * mine.groups * P.Hkv;
            }
            long long sum = v;
            for (int d = 1; d < 32; d <<= 1) {
                const long long o = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d)
                    sum += o;
            }
            const long long all = __shfl_sync(0xffffffffu, sum, 31);
            if (P.B <= 32) {
                total = all;
                u = pick(total);
            }
            if (u >= before && u < before + all) {
                const uint32_t past = __ballot_sync(0xffffffffu, before + sum > u);
                const int at = __ffs((int)past) - 1;
                q.b = b0 + at;
                q.first = before + __shfl_sync(0xffffffffu, sum - v, at);
                q.tiles = __shfl_sync(0xffffffffu, mine.tiles, at);
                q.groups = __shfl_sync(0xffffffffu, mine.groups, at);
                q.seq.x = __shfl_sync(0xffffffffu, mine.seq.x, at);
                q.seq.y = __shfl_sync(0xffffffffu, mine.seq.y, at);
                q.seq.z = __shfl_sync(0xffffffffu, mine.seq.z, at);
                return u;
            }
            before += all;
        }
        if (P.B <= 32)
            return u;
        if (pass == 0) {
            total = before;
            u = pick(total);
            if (u >= total)
                return u;
        }
    }
    return u;
}

template <int N>
struct Int {
    static constexpr int value = N;
};
// Whether O(i) is reported as done by itself: where a group may look at it before
// its next scores, after tiles with new values and at the end of a piece.
__device__ __forceinline__ bool commits_done(int i, int plain, int step, int n)
{
    return i >= plain || i + step >= n;
}

struct Whole {
    static constexpr bool value = false;
};
struct Masked {
    static constexpr bool value = true;
};

// Keys of tile `jt` of an item: how many, and whether they are the cache's.
__device__ __forceinline__ int tile_keys(const Piece &p, int jt, bool &cached)
{
    const int cache_tiles = (p.len + KT - 1) / KT;
    cached = jt < cache_tiles;
    const int left = cached ? p.len - jt * KT : p.nn - (jt - cache_tiles) * KT;
    return left < KT ? left : KT;
}

// A CTA's share: `per` units for each of the slots that have any.  A share
// is at least 2 tiles, one for each softmax group.
__device__ __forceinline__ long long share(const AParams &P, long long total)
{
    const long long per = (total + P.slots - 1) / P.slots;
    return per < 2 ? 2 : per;
}

// The pieces of a CTA's share, one after the other (a warp's walk, all lanes alike).
template <bool PAIR>
struct Walk {
    Place q = {};
    long long u0, u1, u;
    int h = 0, rg = 0, tile = 0;

    __device__ __forceinline__ Walk(const AParams &P, int slot)
    {
        long long total = 0;
        u0 = look_up<PAIR>(P, [&](long long all) { return slot * share(P, all); }, total, q);
        const long long per = share(P, total);
        u1 = u0 + per < total ? u0 + per : total;
        u = u0;
        if (u < u1) {
            const long long at = u - q.first;
            const int item = (int)(at / q.tiles);
            tile = (int)(at - (long long)item * q.tiles);
            h = item / q.groups;
            rg = item - h * q.groups;
        }
    }
    __device__ __forceinline__ Piece piece() const
    {
        const long long left = u1 - u;
        Piece p;
        p.b = q.b;
        p.h = h;
        p.rt0 = rg * (PAIR ? 2 : 1);
        p.last = rg == q.groups - 1;
        p.tile0 = tile;
        p.n = left <= 0 ? 0 : q.tiles - tile < left ? q.tiles - tile : (int)left;
        p.tiles = q.tiles;
        p.len = (int)q.seq.x;
        p.nn = (int)q.seq.y;
        p.status = (int)q.seq.z;
        p.idle = p.nn <= 0;
        p.first = u - tile <= u0;
        return p;
    }
    __device__ __forceinline__ void go_on(const AParams &P, int n)
    {
        u += n;
        tile = 0;
        if (++rg == q.groups) {
            rg = 0;
            if (++h == P.Hkv) {
                h = 0;
                if (u < u1)
                    q = place_at<PAIR>(P, q.b + 1, u);
            }
        }
    }
};

// A CTA that has given up leaves NaN, not what memory held before: in the statistics of its
// pieces of split items, whose rows the join then makes NaN, and in the rows that it was to
// write itself.  By the softmax warps.
template <int NP, bool PAIR>
__device__ __noinline__ void void_share(const AParams &P, int slot, int tid)
{
    constexpr int TILES = Cfg<NP, PAIR>::Q_TILES;
    for (int i = tid; i < TILES * 2 * BM; i += SOFT_THREADS)
        P.part_ml[(size_t)slot * TILES * 2 * BM + i] = make_float2(NAN, NAN);
    Walk<PAIR> walk(P, slot);
    while (true) {
        const Piece p = walk.piece();
        if (p.n == 0)
            break;
        if (p.tile0 == 0) {
            const int from = p.idle ? 0 : p.rt0 * P.nodes_per_tile;
            const int to = p.idle || p.last ? P.N : min(P.N, (p.rt0 + TILES) * P.nodes_per_tile);
            for (int y = tid; y < (to - from) * P.G; y += SOFT_THREADS) {
                const int64_t row = ((int64_t)p.b * P.N + from + y / P.G) * P.Hq +
                                    (int64_t)p.h * P.G + y % P.G;
                for (int d = 0; d < P.D; d += 8)
                    *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(P.out) + row * P.D + d) =
                        make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
                if (P.lse)
                    P.lse[row] = NAN;
            }
        }
        walk.go_on(P, p.n);
    }
}

// Among each 8 lanes, chunk k of lane i and chunk i of lane k change places.
__device__ __forceinline__ void exchange8(uint4 (&u)[8], int lane)
{
#pragma unroll
    for (int m = 4; m; m >>= 1) {
        const bool up = (lane & m) != 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i & m)
                continue;
            uint4 &lo = u[i], &hi = u[i | m];
            const uint4 give = up ? lo : hi;
            uint4 got;
            got.x = __shfl_xor_sync(0xffffffffu, give.x, m);
            got.y = __shfl_xor_sync(0xffffffffu, give.y, m);
            got.z = __shfl_xor_sync(0xffffffffu, give.z, m);
            got.w = __shfl_xor_sync(0xffffffffu, give.w, m);
            if (up)
                lo = got;
            else
                hi = got;
        }
    }
}

template <int DT>
__device__ __forceinline__ void store8(const AParams &P, int64_t elem, const float (&v)[8])
{
    uint4 w;
    w.x = pack<DT>(v[0], v[1]);
    w.y = pack<DT>(v[2], v[3]);
    w.z = pack<DT>(v[4], v[5]);
    w.w = pack<DT>(v[6], v[7]);
    *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(P.out) + elem) = w;
}

// ln of a total of weights in units of 2^m; -inf for none
__device__ __forceinline__ float lse_of(float m, float l)
{
    return l == 0.0f ? -INFINITY : (m + log2f(l)) * (1.0f / LOG2E);
}

template <int NP, int DT, bool PAIR>
__global__ void __launch_bounds__(THREADS, 1)
    attention_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mkn,
                     const __grid_constant__ CUtensorMap mvn, const __grid_constant__ CUtensorMap mkc,
                     const __grid_constant__ CUtensorMap mvc, const __grid_constant__ AParams P)
{
    using C = Cfg<NP, PAIR>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t q_s = smem_addr(smem);
    const uint32_t k_s = q_s + C::Q_TILES * C::TILE, v_s = k_s + C::KST * C::TILE;
    uint8_t *v_p = smem + (size_t)C::TILE * (C::Q_TILES + C::KST);
    Tail &S = *reinterpret_cast<Tail *>(smem + (size_t)C::TILE * (C::Q_TILES + C::KST + C::VST));
    volatile int *abort_flag = &S.abort_flag;
    const int tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int slot = (int)blockIdx.x;

    if (tid == 0) {
        for (int i = 0; i < 6; ++i) {
            mbar_init(&S.kfull[i], 1);
            mbar_init(&S.kempty[i], 1);
            mbar_init(&S.vfull[i], 1);
            mbar_init(&S.vempty[i], 1);
        }
        mbar_init(&S.qfull, 1);
        mbar_init(&S.qempty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.sfull[i], 1);
            mbar_init(&S.pready[i], 4);
            mbar_init(&S.pvdone[i], 1);
            mbar_init(&S.noted[i], 4);
        }
        for (int i = 0; i < RING; ++i) {
            mbar_init(&S.pfull[i], 1);
            mbar_init(&S.pempty[i], 11);  // every warp but the one that writes
        }
        mbar_init(&S.join, 8);
        mbar_init(&S.drain, 1);
        S.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_shared();
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;"
                     :: "r"(smem_addr(&S.tmem_base)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem_base;
    wait_previous_kernel();
    allow_next_kernel();

    // Whether the CTA has given up, the same on every lane: lanes that each looked for
    // themselves could part, and wait for each other in the next test for good.  (The vote costs 1 %
    // of 32 chains of 5, 0.6 % of 4 trees of 256 nodes; one vote for flag and barrier, or
    // one sum, in the same instruction cost 1.5 and 4 % there.)
    auto given_up = [&]() -> bool { return __any_sync(0xffffffffu, *abort_flag != 0); };
    // A warp's wait: false on every lane once the CTA has given up.  (Kept this small: the
    // waits stand in every role's loop, and the loops share an instruction cache.)
    auto wait = [&](unsigned long long *bar, uint32_t parity) -> bool {
#pragma unroll 1
        for (int i = 0; i < WAIT_TRIES; ++i) {
            if (warp_try(bar, parity))
                return true;
            if (given_up())
                return false;
        }
        give_up(abort_flag, P.status);
        return false;
    };
    // the same for a warp that has time, with a limit of its own: it sleeps between its tests
    auto wait_idle = [&](unsigned long long *bar, uint32_t parity, int tries) -> bool {
#pragma unroll 1
        for (int i = 0; i < tries; ++i) {
            if (warp_try(bar, parity))
                return true;
            if (given_up())
                return false;
            __nanosleep(100);
        }
        give_up(abort_flag, P.status);
        return false;
    };
    // the next piece of the share: false when there is none or the CTA has given up
    uint32_t taken = 0;
    auto next = [&](Piece &p) -> bool {
        const int at = (int)(taken % RING);
        if (!wait(&S.pfull[at], (taken / RING) & 1u))
            return false;
        p = S.piece[at];
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&S.pempty[at]);
        ++taken;
        return p.n > 0;
    };

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(SOFT_REGS));
        // ---------------------------------------------------- softmax groups
        const int s = warp >> 2;                 // the group
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;       // row of the tile
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t t_s = tmem + lanes + (uint32_t)(s * KT);
        const uint32_t t_o = tmem + lanes + (uint32_t)(2 * KT + s * C::DP);
        const int local = r / P.G;               // node of the row, counted in the tile
        const int g = r - local * P.G;
        constexpr int STEP = PAIR ? 1 : 2;       // a group's next tile
        const int start = PAIR ? 0 : s;          // and its first
        const uint4 *masks = reinterpret_cast<const uint4 *>(P.plan + P.lay.mask);
        uint32_t cnt = 0, tv = 0, done = 0;      // the group's tiles, all tiles, reports of O
        uint32_t joins = 0, notes = 0;
        const unsigned long long c2 = f2(P.c, P.c);
        // a score x has weight 2^(x c + shift) under the maximum m
        auto shift_of = [&](float m) -> float {
            return m == -INFINITY ? 0.0f : fmaf(-m, P.c, lift<DT>());
        };
        // all softmax warps have come here
        auto join = [&]() -> bool {
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&S.join);
            return wait(&S.join, joins++ & 1u);
        };
        // this group's warps have come here
        auto group = [&]() -> bool {
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&S.noted[s]);
            return wait(&S.noted[s], notes++ & 1u);
        };
        // all warps that work on the group's tile
        auto tile_sync = [&]() -> bool { return PAIR ? join() : group(); };

        bool ok = true;
        Piece p = {};
        while (ok && next(p)) {
            const int node = (p.rt0 + (PAIR ? s : 0)) * P.nodes_per_tile + local;
            const bool row = local < P.nodes_per_tile && node < P.N;
            auto out_row = [&]() -> int64_t {
                return ((int64_t)p.b * P.N + node) * P.Hq + (int64_t)p.h * P.G + g;
            };
            if ((p.idle || p.last) && p.tile0 == 0) {
                // the head's rows of nodes that no row group has are 0, a bad sequence's NaN
                const int from =
                    p.idle ? 0 : min(P.N, (p.rt0 + C::Q_TILES) * P.nodes_per_tile);
                const float x = p.status ? NAN : 0.0f;
                const float v[8] = {x, x, x, x, x, x, x, x};
                for (int y = tid; y < (P.N - from) * P.G; y += SOFT_THREADS) {
                    const int64_t to = ((int64_t)p.b * P.N + from + y / P.G) * P.Hq +
                                       (int64_t)p.h * P.G + y % P.G;
                    for (int d = 0; d < P.D; d += 8)
                        store8<DT>(P, to * P.D + d, v);
                    if (P.lse)
                        P.lse[to] = p.status ? NAN : -INFINITY;
                }
            }
            if (p.idle)
                continue;
            const bool live = row && node < p.nn;
            const bool warp_live = __any_sync(0xffffffffu, live);
            const int cache_tiles = (p.len + KT - 1) / KT;
            const uint4 *mask = masks + ((size_t)p.b * P.N + node) * (P.lay.W / 4);
            uint4 see0 = make_uint4(0, 0, 0, 0);  // the first new tile's mask, loaded ahead
            if (live && p.tile0 <= cache_tiles && cache_tiles < p.tile0 + p.n)
                see0 = __ldg(mask);
            float m = -INFINITY, l = 0.0f;       // maximum of the raw scores, total
            const int plain = min(p.n, p.len / KT - p.tile0);
            // one tile of this group; `masked` tiles hold fewer than KT keys or new ones
            auto tile = [&](int i, auto kind) {
                constexpr bool masked = decltype(kind)::value;
                bool cached = true;
                const int jt = p.tile0 + i;
                const int keys = masked ? tile_keys(p, jt, cached) : KT;
                // what this row sees of the tile
                uint4 see = make_uint4(~0u, ~0u, ~0u, ~0u);
                if (!cached) {
                    see = see0;
                    if (live && jt > cache_tiles)
                        see = __ldg(mask + (jt - cache_tiles));
                }
                // the scores are there, and the group's product before is done
                ok = wait(&S.sfull[s], cnt & 1u);
                if (!ok)
                    return;
                tc_fence_after();
                uint32_t any_bad = 0;
                auto bad_keys = [&](int q) -> uint32_t {  // of keys 32 q on, after tile_sync
                    const volatile uint32_t(*f)[2][4] = S.bad;
                    const uint32_t own = f[s][cnt & 1u][q];
                    return PAIR ? own | f[s ^ 1][cnt & 1u][q] : own;
                };
                if (masked) {
                    // V: rows past the keys (up to the last product's 16) are zeroed; in new
                    // values, non-finite elements are noted and zeroed
                    const uint32_t t = tv + (uint32_t)i;
                    const int st = (int)(t % C::VST);
                    ok = wait(&S.vfull[st], (t / C::VST) & 1u);
                    if (!ok)
                        return;
                    uint8_t *vrow = v_p + (size_t)st * C::TILE + r * 128;
                    bool bad = false;
                    if (r >= keys && r < ((keys + 15) & ~15)) {
#pragma unroll
                        for (int x = 0; x < NP * 8; ++x)
                            *reinterpret_cast<uint4 *>(vrow + (x >> 3) * PANEL_BYTES +
                                                       (x & 7) * 16) = make_uint4(0, 0, 0, 0);
                    } else if (!cached && r < keys) {
                        // (two groups on one tile take a panel each)
#pragma unroll
                        for (int x = 0; x < NP * 8; ++x) {
                            if (PAIR && (x >> 3) != s)
                                continue;
                            uint4 *q = reinterpret_cast<uint4 *>(vrow + (x >> 3) * PANEL_BYTES +
                                                                 (x & 7) * 16);
                            uint4 w = *q;
                            const uint4 f = make_uint4(nonfinite<DT>(w.x), nonfinite<DT>(w.y),
                                                       nonfinite<DT>(w.z), nonfinite<DT>(w.w));
                            if (f.x | f.y | f.z | f.w) {
                                bad = true;
                                w.x &= ~f.x;
                                w.y &= ~f.y;
                                w.z &= ~f.z;
                                w.w &= ~f.w;
                                *q = w;
                            }
                        }
                    }
                    fence_async_shared();
                    if (!cached) {
                        const uint32_t ballot = __ballot_sync(0xffffffffu, bad);
                        if (lane == 0)
                            S.bad[s][cnt & 1u][quarter] = ballot;
                        ok = tile_sync();
                        if (!ok)
                            return;
                        any_bad = bad_keys(0) | bad_keys(1) | bad_keys(2) | bad_keys(3);
                    }
                }
                uint32_t zero_w[4] = {0, 0, 0, 0};  // keys whose weight is 0 (with any_bad only)
                // the row's new maximum `top`; O and l follow where it has grown far
                auto raise = [&](float top) {
                    if (i == start) {
                        m = top;
                        return;
                    }
                    const bool grown = (top - m) * P.c > growth<DT>();  // -inf to finite too
                    if (!__any_sync(0xffffffffu, grown))
                        return;
                    const float f = grown ? ex2((m - top) * P.c) : 1.0f;
                    l *= f;
                    if (grown)
                        m = top;
#pragma unroll 1
                    for (int d = 0; d < C::DP; d += 16) {
                        uint32_t o[16];
                        tmem_ld(t_o + d, o);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                        tmem_st(t_o + d, o);
                    }
                };
                unsigned long long sum[2] = {0ull, 0ull};
                // In a pair, whose products bound it, a tile's weights are made in one pass; the
                // other kernel is bound by its loads, where the small loop below did better
                // (2 % on 64 trees of 29 nodes)
                bool redo = !PAIR || masked || i == start;
                if (PAIR && warp_live && !redo) {
                    // in one pass: weights by the maximum so far, which serves as long as no
                    // score is far above it; the tile's own maximum is found on the way
                    const float shift = shift_of(m);
                    const unsigned long long shift2 = f2(shift, shift);
                    uint32_t x[32], y[32], pk[4][16];
                    __syncwarp();
                    tmem_ld_start(t_s, x);
                    tmem_ld_finish(x);
                    tmem_ld_start(t_s + 32, y);
                    float top = max32(x);
                    weigh<DT>(x, c2, shift2, sum, pk[0]);
                    tmem_ld_finish(y);
                    tmem_ld_start(t_s + 64, x);
                    top = fmaxf(top, max32(y));
                    weigh<DT>(y, c2, shift2, sum, pk[1]);
                    tmem_ld_finish(x);
                    tmem_ld_start(t_s + 96, y);
                    top = fmaxf(top, max32(x));
                    weigh<DT>(x, c2, shift2, sum, pk[2]);
                    tmem_ld_finish(y);
                    top = fmaxf(top, max32(y));
                    weigh<DT>(y, c2, shift2, sum, pk[3]);
                    redo = __any_sync(0xffffffffu,
                                      (top - m) * P.c > growth<DT>());  // -inf to finite too
                    if (!redo) {
#pragma unroll
                        for (int h = 0; h < 4; ++h)
                            tmem_st(t_s + h * 16, pk[h]);
                    } else {
                        sum[0] = sum[1] = 0ull;
                    }
                }
                if (warp_live && redo) {
                    // the maximum first: 32 keys at a time, and no more of them than the tile has
                    const int chunks = (keys + 31) / 32;
                    auto bits = [&](int h) -> uint32_t {
                        const uint32_t w = h == 0 ? see.x : h == 1 ? see.y : h == 2 ? see.z : see.w;
                        return keys - h * 32 >= 32 ? w : w & ((1u << (keys - h * 32)) - 1u);
                    };
                    float top = -INFINITY;
#pragma unroll 1
                    for (int h = 0; h < chunks; ++h) {
                        uint32_t x[32];
                        tmem_ld(t_s + h * 32, x);
                        if (masked)
                            hide(x, bits(h));
                        top = fmaxf(top, max32(x));
                    }
                    raise(top);
                    const float shift = shift_of(m);
                    const unsigned long long shift2 = f2(shift, shift);
#pragma unroll 1
                    for (int h = 0; h < chunks; ++h) {
                        uint32_t x[32], pk[16];
                        tmem_ld(t_s + h * 32, x);
                        if (masked)
                            hide(x, bits(h));
                        weigh<DT>(x, c2, shift2, sum, pk);
                        // weights 32 h on lie in columns 16 h on: over scores that were read
                        tmem_st(t_s + h * 16, pk);
                        if (any_bad) {
                            uint32_t z = 0;
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                z |= ((pk[j] & 0x7fffu) == 0 ? 1u : 0u) << (2 * j) |
                                     ((pk[j] & 0x7fff0000u) == 0 ? 2u : 0u) << (2 * j);
                            zero_w[0] = h == 0 ? z : zero_w[0];
                            zero_w[1] = h == 1 ? z : zero_w[1];
                            zero_w[2] = h == 2 ? z : zero_w[2];
                            zero_w[3] = h == 3 ? z : zero_w[3];
                        }
                    }
                }
                if (warp_live) {
                    float s0, s1;
                    f2_split(add2(sum[0], sum[1]), s0, s1);
                    l += s0 + s1;
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&S.pready[s]);
                if (any_bad) {
                    // what the zeroed elements give the rows that see them, once O(i) is done
                    ok = wait(&S.pvdone[s], done & 1u);
                    if (!ok)
                        return;
                    tc_fence_after();
                    const uint32_t w[4] = {see.x, see.y, see.z, see.w};
                    const int first = (jt - cache_tiles) * KT;
#pragma unroll 1
                    for (int d = 0; d < C::DP; d += 32) {
                        uint32_t o[32];
                        tmem_ld(t_o + d, o);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t left = bad_keys(q);
                            while (left) {
                                const int bit = __ffs((int)left) - 1;
                                left &= left - 1;
                                if (!((w[q] >> bit) & 1u))
                                    continue;
                                const uint16_t *src = reinterpret_cast<const uint16_t *>(P.v_new) +
                                    p.b * P.v_new_stride[0] +
                                    (first + q * 32 + bit) * P.v_new_stride[1] +
                                    p.h * P.v_new_stride[2];
                                const float z = (zero_w[q] >> bit) & 1u ? 0.0f : 1.0f;
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    if (d + j < P.D) {
                                        const uint32_t e = src[d + j];
                                        if (nonfinite<DT>(e) & 0xffffu)
                                            o[j] = __float_as_uint(__uint_as_float(o[j]) +
                                                                   z * unpack1<DT>(e));
                                    }
                            }
                        }
                        tmem_st(t_o + d, o);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    // the notes are written over only after every warp has read them
                    ok = tile_sync();
                }
                if (commits_done(i, plain, STEP, p.n))
                    ++done;
                ++cnt;
            };
            // whole tiles of the cache first, in a loop of their own: it stays small
            int i = start;
            for (; i < plain && ok; i += STEP)
                tile(i, Whole());
            for (; i < p.n && ok; i += STEP)
                tile(i, Masked());
            if (!ok)
                break;

            tv += (uint32_t)p.n;

            // each group writes one panel of the joined halves, or with a row tile of its own
            // all of it
            const bool mine = p.n > start;       // this group had a tile
            if (mine && !wait(&S.pvdone[s], (done - 1) & 1u))
                break;
            tc_fence_after();
            float top = mine && m != -INFINITY ? -shift_of(m) : -INFINITY;
            float sum = mine ? l : 0.0f;
            // a half that saw no key has no weight, whatever its O holds
            bool some0 = !(top == -INFINITY && sum == 0.0f), some1 = false;
            float w0 = 1.0f, w1 = 0.0f, base = top == -INFINITY ? 0.0f : top;
            if (!PAIR) {
                S.m[s][r] = top;
                S.l[s][r] = sum;
                tc_fence_before();
                if (!join())
                    break;
                tc_fence_after();
                const float m0 = S.m[0][r], m1 = S.m[1][r], l0 = S.l[0][r], l1 = S.l[1][r];
                top = fmaxf(m0, m1);
                base = top == -INFINITY ? 0.0f : top;
                some0 = !(m0 == -INFINITY && l0 == 0.0f);
                some1 = !(m1 == -INFINITY && l1 == 0.0f);
                w0 = some0 ? ex2(m0 - base) : 0.0f;
                w1 = some1 ? ex2(m1 - base) : 0.0f;
                sum = l0 * w0 + l1 * w1;
            }
            const bool whole = p.n == p.tiles;
            const bool two = !PAIR && p.n > 1;
            const bool writes = row && (whole || live);
            const int64_t orow = out_row();
            if (__any_sync(0xffffffffu, writes)) {
                const size_t at =
                    (((size_t)slot * C::Q_TILES + (PAIR ? s : 0)) * 2 + (p.first ? 0 : 1)) * BM;
                const float norm = sum != 0.0f ? 1.0f / sum : 0.0f;
                const uint32_t t_o0 = PAIR ? t_o : tmem + lanes + (uint32_t)(2 * KT);
#pragma unroll 1
                for (int panel = PAIR ? 0 : s; panel < NP; panel += STEP) {
                    uint4 u[8];
#pragma unroll
                    for (int d0 = 0; d0 < PANEL; d0 += 32) {
                        uint32_t a[32], b[32];
                        tmem_ld(t_o0 + (uint32_t)(panel * PANEL + d0), a);
                        if (two)
                            tmem_ld(t_o0 + (uint32_t)(C::DP + panel * PANEL + d0), b);
                        float v[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            v[j] = some0 ? __uint_as_float(a[j]) * w0 : 0.0f;
                            if (some1)
                                v[j] = fmaf(__uint_as_float(b[j]), w1, v[j]);
                        }
                        if (whole) {
#pragma unroll
                            for (int j = 0; j < 32; j += 8) {
                                const bool on = live && sum != 0.0f;
                                u[(d0 + j) / 8] = make_uint4(
                                    on ? pack<DT>(v[j] * norm, v[j + 1] * norm) : 0u,
                                    on ? pack<DT>(v[j + 2] * norm, v[j + 3] * norm) : 0u,
                                    on ? pack<DT>(v[j + 4] * norm, v[j + 5] * norm) : 0u,
                                    on ? pack<DT>(v[j + 6] * norm, v[j + 7] * norm) : 0u);
                            }
                        } else if (writes) {
                            // [column][row]: a warp's store is one line
                            float *o = P.part + at * C::DP + (panel * PANEL + d0) * BM + r;
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (panel * PANEL + d0 + j < P.D)
                                    o[j * BM] = v[j];
                        }
                    }
                    if (whole) {
                        // 8 lanes exchange so that each holds one 16-byte chunk of 8 rows: a
                        // store then covers 128 bytes of 4 rows, not 16 of 32 rows
                        exchange8(u, lane);
                        const int d = panel * PANEL + (lane & 7) * 8;
                        const uint32_t rows = __ballot_sync(0xffffffffu, writes);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int from = (lane & ~7) | k;
                            const int64_t at_row = __shfl_sync(0xffffffffu, orow, from);
                            if (((rows >> from) & 1u) && d < P.D)
                                *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(P.out) +
                                                           at_row * P.D + d) = u[k];
                        }
                    }
                }
                if ((PAIR || s == 0) && row) {
                    if (whole && P.lse)
                        P.lse[orow] = live ? lse_of(base, sum) : -INFINITY;
                    if (!whole && live)
                        P.part_ml[at + r] = make_float2(top, sum);
                }
            }
            tc_fence_before();
            if (!PAIR)
                ok = join();  // O and the exchanged statistics are free again
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(HELPER_REGS));
        if (warp == 8) {
            // ------------------------------------------------ TMA of K and V
            uint32_t t0 = 0;                     // tiles of earlier pieces
            uint32_t loaded_k = 0, loaded_v = 0; // tiles that a load was issued for
            bool ok = true;
            Piece p = {};
            // one tile's keys (side 0) or values (1): a box of rows per lane
            auto load = [&](int side, int i) {
                bool cached;
                const int jt = p.tile0 + i;
                const int keys = tile_keys(p, jt, cached);
                const int rows = cached ? P.page_rows : P.new_rows;
                const int at = lane * rows;
                const bool mine = at < keys;
                int y = (jt - (p.len + KT - 1) / KT) * KT + at, w = p.b;
                if (cached) {
                    y = jt * KT + at;
                    if (P.page_table && mine) {
                        const int e = y / P.page_size;
                        w = e < P.pages_per_seq
                            ? __ldg(P.page_table + (size_t)p.b * P.pages_per_seq + e) : -1;
                        y -= e * P.page_size;
                    }
                }
                const uint32_t n = t0 + (uint32_t)i, stages = side ? C::VST : C::KST;
                const int st = (int)(n % stages);
                ok = wait(side ? &S.vempty[st] : &S.kempty[st], ((n / stages) & 1u) ^ 1u);
                if (!ok)
                    return;
                unsigned long long *full = side ? &S.vfull[st] : &S.kfull[st];
                if (lane == 0)
                    mbar_arrive_expect_tx(
                        full, (uint32_t)(((keys + rows - 1) / rows) * rows * 128 * NP));
                __syncwarp();
                (side ? loaded_v : loaded_k) = n + 1;
                if (mine) {
                    const CUtensorMap *map = cached ? (side ? &mvc : &mkc) : (side ? &mvn : &mkn);
                    const uint32_t dst =
                        (side ? v_s : k_s) + (uint32_t)(st * C::TILE + at * 128);
#pragma unroll
                    for (int d = 0; d < NP; ++d)
                        tma_load_4d(dst + d * PANEL_BYTES, map, d * PANEL, y, p.h, w, full);
                }
                __syncwarp();
            };
            while (ok && next(p)) {
                if (p.idle)
                    continue;
                for (int i = 0; i < p.n && ok; ++i) {
                    load(0, i);
                    if (ok)
                        load(1, i);
                }
                t0 += (uint32_t)p.n;
            }
            if (lane == 0) {
                S.loaded[0] = loaded_k;
                S.loaded[1] = loaded_v;
            }
        } else if (warp == 9) {
            // -------------------------------------------- issuer of the products
            // The whole warp runs the loop and one elected lane issues: what the products
            // are given then stays in uniform registers (issued from under `lane == 0` each
            // product took about 120 clocks to issue, twice its time in the tensor pipe).
            uint32_t items = 0;
            bool ok = true;
            const int ksteps = (P.D + 15) / 16;
            const uint32_t id_o = idesc<DT>(ksteps * 16, true);
            Piece p = {};
            if constexpr (PAIR) {
                // A step of group G: O(i) += P V(i), then S = Q K(i + 1)^T.  Its own waits, commits
                // and addresses are what this warp's time goes into (1200 clocks of a step's 2000
                // when each was done by itself), so in the usual case one test covers both tiles
                // and one elected block issues all of it.
                int kst = 0, vst = 0;                // stages and phases of the next K and V tile
                uint32_t kph = 0, vph = 0, pph[2] = {0, 0};
                constexpr uint32_t id_s = idesc<DT>(KT, false);
                const uint64_t qd0 = desc_k(q_s), kd0 = desc_k(k_s), vd0 = desc_mn(v_s);
                constexpr uint64_t TILE16 = C::TILE >> 4;
                int plain = 0;                       // whole tiles of the cache come first
                auto next_k = [&]() {
                    kph ^= kst + 1 == C::KST ? 1u : 0u;
                    kst = kst + 1 == C::KST ? 0 : kst + 1;
                };
                auto next_v = [&]() {
                    vph ^= vst + 1 == C::VST ? 1u : 0u;
                    vst = vst + 1 == C::VST ? 0 : vst + 1;
                };
                // commits behind the scores of tile i
                auto scored = [&](int s, int i) {
                    if (s)
                        mma_commit(&S.kempty[kst]);
                    mma_commit(&S.sfull[s]);
                    if (i == p.n - 1 && s)
                        mma_commit(&S.qempty);
                };
                auto scores = [&](int s, int i) {    // S = Q K(i)^T by itself
                    bool cached;
                    const int keys = tile_keys(p, p.tile0 + i, cached);
                    ok = wait(&S.kfull[kst], kph);
                    if (!ok)
                        return;
                    tc_fence_after();
                    const uint32_t id = idesc<DT>((keys + 15) & ~15, false);
                    const uint32_t d = tmem + (uint32_t)(s * KT);
                    const uint64_t qd = qd0 + s * TILE16, kd = kd0 + kst * TILE16;
                    if (elect_one()) {
#pragma unroll 1
                        for (int x = 0; x < ksteps; ++x) {
                            const uint64_t off =
                                (uint64_t)(((x >> 2) * PANEL_BYTES + (x & 3) * 32) >> 4);
                            mma_ss(d, qd + off, kd + off, id, x ? 1u : 0u);
                        }
                        scored(s, i);
                    }
                    __syncwarp();
                    if (s)
                        next_k();
                };
                auto step = [&](auto group, int i) {
                    constexpr int G = decltype(group)::value;
                    const uint32_t t_s = tmem + (uint32_t)(G * KT);
                    const uint32_t t_o = tmem + (uint32_t)(2 * KT + G * C::DP);
                    const uint64_t vd = vd0 + vst * TILE16;
                    const uint32_t more = i >= 1 ? 1u : 0u;
                    const bool usual = i + 1 < plain && ksteps == NP * 4;
                    // (the second group of a pair finds the first one's tiles)
                    ok = wait(&S.pready[G], pph[G]);
                    if (!ok)
                        return;
                    const bool all = usual && (G ||
                                               warp_try2(&S.vfull[vst], vph, &S.kfull[kst], kph));
                    if (all) {
                        tc_fence_after();
                        const uint64_t qd = qd0 + G * TILE16, kd = kd0 + kst * TILE16;
                        if (elect_one()) {
                            // 16 keys a step: 8 columns of P, 2 KB of V
#pragma unroll
                            for (int x = 0; x < KT / 16; ++x)
                                mma_ts(t_o, t_s + (uint32_t)(x * 8), vd + (uint64_t)(x * (2048 >> 4)),
                                       id_o, x ? 1u : more);
                            if (G)
                                mma_commit(&S.vempty[vst]);
#pragma unroll
                            for (int x = 0; x < NP * 4; ++x) {
                                const uint64_t off =
                                    (uint64_t)(((x >> 2) * PANEL_BYTES + (x & 3) * 32) >> 4);
                                mma_ss(t_s, qd + off, kd + off, id_s, x ? 1u : 0u);
                            }
                            scored(G, i + 1);
                        }
                        __syncwarp();
                        if (G)
                            next_k();
                    } else {
                        bool cached;
                        const int keys = tile_keys(p, p.tile0 + i, cached);
                        ok = wait(&S.vfull[vst], vph);
                        if (!ok)
                            return;
                        tc_fence_after();
                        if (elect_one()) {
                            const int steps = (keys + 15) / 16;
#pragma unroll 1
                            for (int x = 0; x < steps; ++x)
                                mma_ts(t_o, t_s + (uint32_t)(x * 8), vd + (uint64_t)(x * (2048 >> 4)),
                                       id_o, x ? 1u : more);
                            if (G)
                                mma_commit(&S.vempty[vst]);
                            if (commits_done(i, plain, 1, p.n))
                                mma_commit(&S.pvdone[G]);
                        }
                        __syncwarp();
                        if (i + 1 < p.n)
                            scores(G, i + 1);
                    }
                    pph[G] ^= 1u;
                    if (G)
                        next_v();
                };
                while (ok && next(p)) {
                    if (p.idle)
                        continue;
                    plain = min(p.n, p.len / KT - p.tile0);
                    ok = wait(&S.qfull, items & 1u);
                    ++items;
                    if (ok)
                        scores(0, 0);
                    if (ok)
                        scores(1, 0);
                    for (int i = 0; i < p.n && ok; ++i) {
                        step(Int<0>(), i);
                        if (ok)
                            step(Int<1>(), i);
                    }
                }
            } else {
                uint32_t t0 = 0, cnt[2] = {0, 0};
                auto scores = [&](int j) {  // S = Q K(j)^T of group j & 1
                    bool cached;
                    const int keys = tile_keys(p, p.tile0 + j, cached);
                    const int s = j & 1;
                    const uint32_t t = t0 + (uint32_t)j;
                    const int st = (int)(t % C::KST);
                    ok = wait(&S.kfull[st], (t / C::KST) & 1u);
                    if (!ok)
                        return;
                    tc_fence_after();
                    const uint32_t id = idesc<DT>((keys + 15) & ~15, false);
                    const uint32_t d = tmem + (uint32_t)(s * KT);
                    const uint64_t qd = desc_k(q_s);
                    const uint64_t kd = desc_k(k_s + st * C::TILE);
                    if (elect_one()) {
                        if (ksteps == NP * 4) {
#pragma unroll
                            for (int x = 0; x < NP * 4; ++x) {
                                const uint64_t off =
                                    (uint64_t)(((x >> 2) * PANEL_BYTES + (x & 3) * 32) >> 4);
                                mma_ss(d, qd + off, kd + off, id, x ? 1u : 0u);
                            }
                        } else {
                            for (int x = 0; x < ksteps; ++x) {
                                const uint64_t off =
                                    (uint64_t)(((x >> 2) * PANEL_BYTES + (x & 3) * 32) >> 4);
                                mma_ss(d, qd + off, kd + off, id, x ? 1u : 0u);
                            }
                        }
                        mma_commit(&S.kempty[st]);
                        mma_commit(&S.sfull[s]);
                        if (j == p.n - 1)
                            mma_commit(&S.qempty);
                    }
                    __syncwarp();
                };
                while (ok && next(p)) {
                    if (p.idle)
                        continue;
                    const int plain = min(p.n, p.len / KT - p.tile0);
                    ok = wait(&S.qfull, items & 1u);
                    ++items;
                    for (int j = 0; j < 2 && j < p.n && ok; ++j)
                        scores(j);
                    for (int j = 0; j < p.n && ok; ++j) {
                        bool cached;
                        const int keys = tile_keys(p, p.tile0 + j, cached);
                        const int s = j & 1;
                        const uint32_t n = s ? cnt[1] : cnt[0];
                        const uint32_t t = t0 + (uint32_t)j;
                        const int st = (int)(t % C::VST);
                        ok = wait(&S.vfull[st], (t / C::VST) & 1u) && wait(&S.pready[s], n & 1u);
                        if (!ok)
                            break;
                        tc_fence_after();
                        const uint32_t d = tmem + (uint32_t)(2 * KT + s * C::DP);
                        const uint32_t a = tmem + (uint32_t)(s * KT);
                        const uint64_t vd = desc_mn(v_s + st * C::TILE);
                        // 16 keys a step: 8 columns of P, 2 KB of V
                        const int steps = (keys + 15) / 16;
                        const uint32_t more = j >= 2 ? 1u : 0u;
                        if (elect_one()) {
                            if (steps == KT / 16) {
#pragma unroll
                                for (int x = 0; x < KT / 16; ++x)
                                    mma_ts(d, a + (uint32_t)(x * 8), vd + (uint64_t)(x * (2048 >> 4)),
                                           id_o, x ? 1u : more);
                            } else {
                                for (int x = 0; x < steps; ++x)
                                    mma_ts(d, a + (uint32_t)(x * 8), vd + (uint64_t)(x * (2048 >> 4)),
                                           id_o, x ? 1u : more);
                            }
                            mma_commit(&S.vempty[st]);
                            if (commits_done(j, plain, 2, p.n))
                                mma_commit(&S.pvdone[s]);
                        }
                        __syncwarp();
                        if (s)
                            ++cnt[1];
                        else
                            ++cnt[0];
                        if (j + 2 < p.n)
                            scores(j + 2);
                    }
                    t0 += (uint32_t)p.n;
                }
            }
        } else if (warp == 10) {
            // ---------------------------------------------------- TMA of Q
            uint32_t items = 0;
            Piece p = {};
            while (next(p)) {
                if (p.idle)
                    continue;
                if (!wait_idle(&S.qempty, (items & 1u) ^ 1u, WAIT_TRIES))
                    break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&S.qfull,
                                          (uint32_t)(P.q_rows * 128 * NP * C::Q_TILES));
                    for (int i = 0; i < NP * C::Q_TILES; ++i)
                        tma_load_5d(q_s + i * PANEL_BYTES, &mq, (i % NP) * PANEL, 0,
                                    (p.rt0 + i / NP) * P.nodes_per_tile, p.h, p.b, &S.qfull);
                }
                __syncwarp();
                ++items;
            }
            if (lane == 0)
                S.loaded[2] = items;
        } else {
            // ------------------------------------------- the share's pieces
            Walk<PAIR> walk(P, slot);
            for (uint32_t k = 0;; ++k) {
                const int at = (int)(k % RING);
                // (the self-test: a wait for what nothing brings, with a small limit)
                const bool lose = slot == P.lose && (int)k == P.lose_after;
                if (!wait_idle(lose ? &S.drain : &S.pempty[at], lose ? 0u : ((k / RING) & 1u) ^ 1u,
                               lose ? LOSE_TRIES : WAIT_TRIES))
                    break;
                const Piece p = walk.piece();
                if (lane == 0) {
                    S.piece[at] = p;
                    mbar_arrive(&S.pfull[at]);
                }
                __syncwarp();
                if (p.n == 0)
                    break;
                walk.go_on(P, p.n);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // Every role has ended, some perhaps before the one that gave up: what they left in flight
        // lands first (bounded).  Each barrier's last phase that has a load, and the products.
        if (warp == 8) {
            for (int side = 0; side < 2; ++side) {
                const uint32_t stages = side ? C::VST : C::KST, n = S.loaded[side];
                for (uint32_t st = 0; st < stages && st < n; ++st)
                    (void)mbar_wait(side ? &S.vfull[st] : &S.kfull[st], ((n - 1 - st) / stages) & 1u);
            }
        } else if (warp == 9) {
            if (elect_one())
                mma_commit(&S.drain);
            __syncwarp();
            (void)mbar_wait(&S.drain, 0u);
        } else if (warp == 10 && S.loaded[2] > 0) {
            (void)mbar_wait(&S.qfull, (S.loaded[2] - 1) & 1u);
        } else if (warp < 8) {
            void_share<NP, PAIR>(P, slot, tid);
        }
        __syncthreads();
    }
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
    }
}

// ---------------------------------------------------------------- joining

constexpr int JOIN_WARPS = 8;
constexpr int JOIN_ROWS = 32;
constexpr int JOIN_UNROLL = 2;    // pieces whose sums a thread has in flight

// The running (log2 of the weights' unit, total, sums) of some pieces of one row.
template <int COLS>
struct Joined {
    float top = -INFINITY, sum = 0.0f;
    bool some = false;            // whether any piece saw a key
    float o[COLS];
    // scale of these sums under a new maximum `base` (finite)
    __device__ __forceinline__ float factor(float base) const
    {
        return some ? ex2(top - base) : 0.0f;
    }
};

// Joins the pieces of the items that lie across a share's end.  CTA x takes
// the item that the end of share x cuts (when no earlier end cuts it), 32 rows
// of one of its row tiles: a row per lane, an eighth of the columns per warp.
// Where there are fewer rows, the lanes left over take pieces of their own (a
// single token's item over 4096 positions has 17 of them, and one after the
// other they took most of the call's time).
template <int NP, int DT, bool PAIR>
__global__ void __launch_bounds__(JOIN_WARPS * 32, 4)
    join_kernel(const __grid_constant__ AParams P)
{
    using C = Cfg<NP, PAIR>;
    constexpr int COLS = C::DP / JOIN_WARPS;
    __shared__ __align__(16) uint16_t tile[JOIN_ROWS][C::DP + 8];
    const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
    const int mine = lane & (P.join_rows - 1), part = lane / P.join_rows;
    const int parts = 32 / P.join_rows;
    const int r = (int)blockIdx.z * JOIN_ROWS + mine;
    // the plan is complete: every CTA of the attention had waited for it before this grid began
    long long total = 0;
    Place q = {};
    const long long end = look_up<PAIR>(
        P, [&](long long all) { return ((long long)blockIdx.x + 1) * share(P, all); }, total, q);
    allow_next_kernel();
    wait_previous_kernel();
    const long long per = share(P, total);
    if (end >= total)
        return;
    const int index = (int)((end - q.first) / q.tiles);
    const long long item = q.first + (long long)index * q.tiles;  // its first unit
    const int nn = (int)q.seq.y;
    const int h = index / q.groups, rt = (index - h * q.groups) * C::Q_TILES + (int)blockIdx.y;
    if (item == end || item < end - per || nn <= 0)
        return;  // not cut here, or the previous end has it, or no node
    const int local = r / P.G, g = r - local * P.G;
    const int node = rt * P.nodes_per_tile + local;
    const bool row = local < P.nodes_per_tile && node < P.N;
    const bool live = row && node < nn;
    const int64_t orow = ((int64_t)q.b * P.N + node) * P.Hq + (int64_t)h * P.G + g;
    const int s0 = (int)blockIdx.x, n = (int)((item + q.tiles - 1) / per) - s0 + 1;
    // a share that starts with the item, or inside it, left its first piece; one that the item
    // starts inside of left its second
    auto at = [&](int k) -> size_t {
        const int which = (long long)(s0 + k) * per >= item ? 0 : 1;
        return (((size_t)(s0 + k) * C::Q_TILES + blockIdx.y) * 2 + which) * BM;
    };
    Joined<COLS> A;
#pragma unroll
    for (int j = 0; j < COLS; ++j)
        A.o[j] = 0.0f;
    if (live)
        for (int k0 = part; k0 < n; k0 += JOIN_UNROLL * parts) {
            float2 ml[JOIN_UNROLL];
            float x[JOIN_UNROLL][COLS];
#pragma unroll
            for (int u = 0; u < JOIN_UNROLL; ++u) {
                const int k = k0 + u * parts;
                ml[u] = make_float2(-INFINITY, 0.0f);
                if (k < n) {
                    ml[u] = __ldcg(&P.part_ml[at(k) + r]);
                    const float *v = P.part + at(k) * C::DP + (size_t)(warp * COLS) * BM + r;
#pragma unroll
                    for (int j = 0; j < COLS; ++j)
                        x[u][j] = warp * COLS + j < P.D ? __ldcg(v + j * BM) : 0.0f;
                }
            }
            float top = A.top;
#pragma unroll
            for (int u = 0; u < JOIN_UNROLL; ++u)
                top = fmaxf(top, ml[u].x);
            const float base = top == -INFINITY ? 0.0f : top;
            const float f = A.factor(base);
            A.sum *= f;
#pragma unroll
            for (int j = 0; j < COLS; ++j)
                A.o[j] *= f;
#pragma unroll
            for (int u = 0; u < JOIN_UNROLL; ++u) {
                if (ml[u].x == -INFINITY && ml[u].y == 0.0f)
                    continue;  // no key seen there
                const float w = ex2(ml[u].x - base);
                A.sum = fmaf(ml[u].y, w, A.sum);
#pragma unroll
                for (int j = 0; j < COLS; ++j)
                    A.o[j] = fmaf(x[u][j], w, A.o[j]);
                A.some = true;
            }
            A.top = top;
        }
    for (int d = P.join_rows; d < 32; d <<= 1) {
        const float top2 = __shfl_xor_sync(0xffffffffu, A.top, d);
        const float sum2 = __shfl_xor_sync(0xffffffffu, A.sum, d);
        const bool some2 = __shfl_xor_sync(0xffffffffu, A.some ? 1 : 0, d) != 0;
        const float top = fmaxf(A.top, top2), base = top == -INFINITY ? 0.0f : top;
        const float f = A.factor(base), f2 = some2 ? ex2(top2 - base) : 0.0f;
        A.sum = A.sum * f + sum2 * f2;
#pragma unroll
        for (int j = 0; j < COLS; ++j)
            A.o[j] = A.o[j] * f + __shfl_xor_sync(0xffffffffu, A.o[j], d) * f2;
        A.top = top;
        A.some |= some2;
    }
    const float norm = A.sum != 0.0f ? 1.0f / A.sum : 0.0f;
    if (part == 0) {
#pragma unroll
        for (int j = 0; j < COLS; j += 2)
            *reinterpret_cast<uint32_t *>(&tile[mine][warp * COLS + j]) =
                A.sum != 0.0f ? pack<DT>(A.o[j] * norm, A.o[j + 1] * norm) : 0u;
        if (warp == 0 && row && P.lse)
            P.lse[orow] = live ? lse_of(A.top == -INFINITY ? 0.0f : A.top, A.sum) : -INFINITY;
    }
    __syncthreads();
    const uint32_t rows = __ballot_sync(0xffffffffu, row && part == 0);
#pragma unroll
    for (int k = 0; k < JOIN_ROWS / JOIN_WARPS; ++k) {
        const int y = warp * (JOIN_ROWS / JOIN_WARPS) + k;
        const int64_t to = __shfl_sync(0xffffffffu, orow, y);
        const int d = lane * 4;
        if (((rows >> y) & 1u) && d < P.D)
            *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(P.out) + to * P.D + d) =
                *reinterpret_cast<const uint2 *>(&tile[y][d]);
    }
}

// ------------------------------------------------------------------- host

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool heads_ok(int32_t N, int32_t Hq, int32_t Hkv, int32_t D)
{
    return N >= 1 && N <= SPEC_ATTN_MAX_NODES && Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 &&
           Hq / Hkv <= BM && Hq <= 65535 && D >= 8 && D % 8 == 0 && D <= SPEC_ATTN_MAX_HEAD_DIM;
}

bool page_size_ok(int32_t s, bool paged)
{
    return s >= 1 && (!paged || s % KT == 0 || (s >= 8 && (s & (s - 1)) == 0));
}

bool strides_ok(const int64_t (&s)[3])
{
    for (int64_t x : s)
        if (x < 0 || x % 8 != 0 || x >= ((int64_t)1 << 38))
            return false;
    return true;
}

int row_tiles(int N, int G)
{
    const int per = BM / G;
    return (N + per - 1) / per;
}

struct WsLayout {
    size_t ml, part, total;
};

WsLayout ws_layout(int N, int G, int D)
{
    const size_t ctas = row_tiles(N, G) > 1 ? 2 * MAX_CTAS : MAX_CTAS;  // (row tiles of them)
    const size_t dp = D > PANEL ? 2 * PANEL : PANEL;
    WsLayout w;
    w.ml = 0;
    w.part = plan_align(w.ml + ctas * 2 * BM * sizeof(float2));
    w.total = plan_align(w.part + ctas * 2 * BM * dp * sizeof(float));
    return w;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static const EncodeTiledFn fn = []() -> EncodeTiledFn {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiledFn>(p);
        (void)cudaGetLastError();
        return nullptr;
    }();
    return fn;
}

// A tensor map of 64-element, 128-byte swizzled boxes; dims[0] is the head
// dimension, strides (elements) belong to dims 1 on.  What lies outside reads 0.
bool make_map(CUtensorMap *map, const void *base, int dtype, int rank, const uint64_t *dims,
              const int64_t *strides, const uint32_t *box)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn)
        return false;
    cuuint64_t d[5], s[4];
    cuuint32_t b[5], e[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        e[i] = 1;
        if (i > 0)  // a dimension of one entry is never stepped along: any stride will do
            s[i - 1] = (cuuint64_t)(dims[i] > 1 ? strides[i - 1] : (int64_t)dims[0] + 8) * 2 / 16 * 16;
    }
    return fn(map, dtype == SPEC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
              (cuuint32_t)rank, const_cast<void *>(base), d, s, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct DevInfo {
    std::atomic<int> sms;
    std::atomic<bool> attr[2][2][2];
};
DevInfo g_dev[64];

template <int NP, int DT, bool PAIR>
int launch(const CUtensorMap (&maps)[5], AParams &P, int sms, DevInfo &di, cudaStream_t st)
{
    if (!di.attr[NP - 1][DT - 1][PAIR].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(attention_kernel<NP, DT, PAIR>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem_bytes<NP, PAIR>()) != cudaSuccess) {
            (void)cudaGetLastError();
            return SPEC_ECUDA;
        }
        di.attr[NP - 1][DT - 1][PAIR].store(true, std::memory_order_release);
    }
    const int ctas = sms < MAX_CTAS ? sms : MAX_CTAS;
    P.slots = ctas;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned int)P.slots);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem_bytes<NP, PAIR>();
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, attention_kernel<NP, DT, PAIR>, maps[0], maps[1], maps[2], maps[3],
                           maps[4], P) != cudaSuccess) {
        (void)cudaGetLastError();
        return SPEC_ECUDA;
    }
    if (P.slots > 1) {
        const int rows = P.nodes_per_tile * P.G < P.N * P.G ? P.nodes_per_tile * P.G : P.N * P.G;
        P.join_rows = JOIN_ROWS;
        while (P.join_rows / 2 >= rows)
            P.join_rows /= 2;
        cfg.gridDim = dim3((unsigned int)(P.slots - 1), (unsigned int)(PAIR ? 2 : 1),
                           (unsigned int)((rows + JOIN_ROWS - 1) / JOIN_ROWS));
        cfg.blockDim = dim3(JOIN_WARPS * 32);
        cfg.dynamicSmemBytes = 0;
        if (cudaLaunchKernelEx(&cfg, join_kernel<NP, DT, PAIR>, P) != cudaSuccess) {
            (void)cudaGetLastError();
            return SPEC_ECUDA;
        }
    }
    return SPEC_OK;
}

}  // namespace

extern "C" {

size_t spec_tree_attention_workspace_size(int32_t N, int32_t Hq, int32_t Hkv, int32_t D)
{
    return heads_ok(N, Hq, Hkv, D) ? ws_layout(N, Hq / Hkv, D).total : 0;
}

static int32_t attend(const spec_tree_attention_args *args, void *workspace,
                      size_t workspace_bytes, int lose, int lose_after, void *stream)
{
    if (!args)
        return SPEC_EINVAL;
    const spec_tree_attention_args &a = *args;
    const bool paged = a.page_table != nullptr;
    if (!heads_ok(a.N, a.Hq, a.Hkv, a.D) || a.B < 0 || a.B > 65535 ||
        !page_size_ok(a.page_size, paged) || a.pages_per_seq < 1 || a.num_pages < 0 ||
        (long long)a.pages_per_seq * a.page_size > INT32_MAX - SPEC_ATTN_MAX_NODES ||
        (a.dtype != SPEC_BF16 && a.dtype != SPEC_F16) || !(a.scale > 0.0f) || isinf(a.scale))
        return SPEC_EINVAL;
    if (a.B == 0)
        return SPEC_OK;
    const void *bases[] = {a.q, a.k_new, a.v_new, a.k_cache, a.v_cache, a.out};
    for (const void *p : bases)
        if (!p || !aligned(p, 16))
            return SPEC_EINVAL;
    if (!strides_ok(a.q_stride) || !strides_ok(a.k_new_stride) || !strides_ok(a.v_new_stride) ||
        !strides_ok(a.k_cache_stride) || !strides_ok(a.v_cache_stride) || !a.plan ||
        !aligned(a.plan, 256) || !workspace || !aligned(workspace, 256) ||
        !aligned(a.page_table, 4) || !aligned(a.out_lse, 4) ||
        (!paged && (a.pages_per_seq != 1 || a.num_pages < a.B)))
        return SPEC_EINVAL;
    // TMA steps along a dimension by its stride: none may be 0 where there are two entries
    const int32_t G = a.Hq / a.Hkv;
    auto stepped = [](const int64_t (&s)[3], int64_t n0, int64_t n1, int64_t n2) {
        return (n0 < 2 || s[0] > 0) && (n1 < 2 || s[1] > 0) && (n2 < 2 || s[2] > 0);
    };
    if (!stepped(a.q_stride, a.B, a.N, a.Hq) || !stepped(a.k_new_stride, a.B, a.N, a.Hkv) ||
        !stepped(a.v_new_stride, a.B, a.N, a.Hkv) ||
        !stepped(a.k_cache_stride, a.num_pages, a.page_size, a.Hkv) ||
        !stepped(a.v_cache_stride, a.num_pages, a.page_size, a.Hkv))
        return SPEC_EINVAL;
    const WsLayout w = ws_layout(a.N, G, a.D);
    if (workspace_bytes < w.total)
        return SPEC_ENOSPACE;

    AParams P;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    P.plan = static_cast<const uint8_t *>(a.plan);
    P.lay = plan_layout(a.B, a.N);
    P.page_table = a.page_table;
    P.v_new = a.v_new;
    for (int i = 0; i < 3; ++i)
        P.v_new_stride[i] = a.v_new_stride[i];
    P.out = a.out;
    P.lse = a.out_lse;
    P.status = &reinterpret_cast<WsHeader *>(const_cast<void *>(a.plan))->status;
    P.part_ml = reinterpret_cast<float2 *>(ws + w.ml);
    P.part = reinterpret_cast<float *>(ws + w.part);
    P.c = a.scale * LOG2E;
    P.B = a.B;
    P.N = a.N;
    P.Hq = a.Hq;
    P.Hkv = a.Hkv;
    P.D = a.D;
    P.G = G;
    P.nodes_per_tile = BM / G;
    P.page_size = a.page_size;
    P.pages_per_seq = a.pages_per_seq;
    P.page_rows = paged && a.page_size < KT ? a.page_size : KT;
    P.new_rows = a.N < KT ? (a.N + 7) / 8 * 8 : KT;
    P.q_rows = P.nodes_per_tile * G;
    P.lose = lose;
    P.lose_after = lose_after;

    CUtensorMap maps[5];
    const uint64_t qd[5] = {(uint64_t)a.D, (uint64_t)G, (uint64_t)a.N, (uint64_t)a.Hkv,
                            (uint64_t)a.B};
    const int64_t qs[4] = {a.q_stride[2], a.q_stride[1], a.q_stride[2] * G, a.q_stride[0]};
    const uint32_t qb[5] = {PANEL, (uint32_t)G, (uint32_t)P.nodes_per_tile, 1, 1};
    const uint64_t nd[4] = {(uint64_t)a.D, (uint64_t)a.N, (uint64_t)a.Hkv, (uint64_t)a.B};
    const uint32_t nb[4] = {PANEL, (uint32_t)P.new_rows, 1, 1};
    const uint64_t cd[4] = {(uint64_t)a.D, (uint64_t)a.page_size, (uint64_t)a.Hkv,
                            (uint64_t)(a.num_pages > 0 ? a.num_pages : 1)};
    const uint32_t cb[4] = {PANEL, (uint32_t)P.page_rows, 1, 1};
    auto order = [](const int64_t (&s)[3], int64_t (&o)[3]) {  // (slot or node, head, page or sequence)
        o[0] = s[1];
        o[1] = s[2];
        o[2] = s[0];
    };
    int64_t kn[3], vn[3], kc[3], vc[3];
    order(a.k_new_stride, kn);
    order(a.v_new_stride, vn);
    order(a.k_cache_stride, kc);
    order(a.v_cache_stride, vc);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return SPEC_ECUDA;
    if (!make_map(&maps[0], a.q, a.dtype, 5, qd, qs, qb) ||
        !make_map(&maps[1], a.k_new, a.dtype, 4, nd, kn, nb) ||
        !make_map(&maps[2], a.v_new, a.dtype, 4, nd, vn, nb) ||
        !make_map(&maps[3], a.k_cache, a.dtype, 4, cd, kc, cb) ||
        !make_map(&maps[4], a.v_cache, a.dtype, 4, cd, vc, cb))
        return SPEC_ECUDA;
    DevInfo &di = g_dev[dev];
    int sms = di.sms.load(std::memory_order_relaxed);
    if (!sms) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            sms < 1)
            return SPEC_ECUDA;
        di.sms.store(sms, std::memory_order_relaxed);
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool wide = a.D > PANEL, pair = row_tiles(a.N, G) > 1;
    if (a.dtype == SPEC_BF16) {
        if (wide)
            return pair ? launch<2, SPEC_BF16, true>(maps, P, sms, di, st)
                        : launch<2, SPEC_BF16, false>(maps, P, sms, di, st);
        return pair ? launch<1, SPEC_BF16, true>(maps, P, sms, di, st)
                    : launch<1, SPEC_BF16, false>(maps, P, sms, di, st);
    }
    if (wide)
        return pair ? launch<2, SPEC_F16, true>(maps, P, sms, di, st)
                    : launch<2, SPEC_F16, false>(maps, P, sms, di, st);
    return pair ? launch<1, SPEC_F16, true>(maps, P, sms, di, st)
                : launch<1, SPEC_F16, false>(maps, P, sms, di, st);
}

int32_t spec_tree_attention(const spec_tree_attention_args *args, void *workspace,
                            size_t workspace_bytes, void *stream)
{
    return attend(args, workspace, workspace_bytes, -1, 0, stream);
}

int32_t spec_selftest_attention_timeout(const spec_tree_attention_args *args, void *workspace,
                                        size_t workspace_bytes, int32_t cta, int32_t after,
                                        void *stream)
{
    if (cta < 0 || after < 0)
        return SPEC_EINVAL;
    return attend(args, workspace, workspace_bytes, cta, after, stream);
}

}  // extern "C"
