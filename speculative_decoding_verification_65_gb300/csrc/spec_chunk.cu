// spec_chunk.cu -- causal attention of chunks of new tokens over a key/value cache on the
// tcgen05 tensor cores (include/spec_chunk.h).
//
// For one sequence and one key/value head the query rows are the new tokens times the G = Hq / Hkv
// heads of the group.  A CTA works on a row group: the 2 * floor(128 / G) tokens that fill two row
// tiles of 128, over the keys that any of them sees, 128 at a time: S = Q K^T, a running softmax
// per row, O += P V.  A step over 128 keys is four products of 128 x 128 x D, 2048 clocks of the
// tensor pipe at D = 128, for 64 KB of K and V from L2; that, and the 32768 exponentials beside it,
// is what bounds the kernel.
//
// Roles in a CTA (one per SM, 3 warpgroups; the third gives registers to the others):
//   warps 0-3, 4-7  a row tile each, one thread per row: while one tile's scores become weights
//                   (in TMEM, in the place of the scores, as the A operand of P V) the tensor
//                   cores work on the other's products
//   warp 8          TMA of the K and V tiles, each a ring of stages; pages
//                   smaller than a tile are boxes of one tile
//   warp 9          issues the products: S(0) of each tile, then O(i), S(i + 1) of the one and of
//                   the other; a commit behind S(i + 1) so also says that O(i) is done.  O(i) is
//                   issued in two halves of the keys, the first while the second's weights are made
//   warp 10         waits for the issuer's tiles
//   warp 11         walks the CTA's share, hands the pieces of it out through a small ring and loads
//                   their Q
// TMEM: S_0, S_1 (128 columns each), O_0, O_1 (up to 128 each).
//
// Measured, GPU time with plan, append and join, 128 columns bf16: 8 x up to 1024 tokens behind up to 4096
// positions, 32 heads on 8, 329 us, 1.17 PFLOP/s; 512 behind 96547, 40 on 8, 782 us, 1.46 PFLOP/s; 2 x
// up to 8192, 64 on 8, 1470 us, 1.34 PFLOP/s.  A step of both row tiles over 128 keys all of whose
// keys are seen takes 2470 to 2740 clocks, of which the tensor pipe is at work 2144; the products of S
// read 128 bytes of shared memory a clock, as many as there are, while TMA writes the next tiles.
// A piece's start and end add some 10000 clocks: its first maxima, its masked tile, its stores, and the
// instructions for them, which have left the caches in between.
//
// A row's sums are rescaled only when its maximum has grown by more than 2^8 (2^4 with fp16
// weights) since the last time, so most tiles leave O in TMEM alone.
//
// Work: the key tiles of all row groups and heads stand in a line and are dealt to the CTAs in
// equal runs.  An item (head, row group) that lies in one CTA's run is written by it; of a split
// item each CTA leaves its unnormalised sums with their maximum and total in the workspace, and a
// second kernel joins them in order, so repeats are bit-equal.  No CTA waits for another.
//
// What a row must not see: tiles that every row of the group sees whole come first and are not
// masked.  In the others, scores of hidden keys are replaced, not added to, so NaN keys have no
// effect.  A hidden key's value does enter P V with weight 0, and 0 * NaN is NaN: rows of V past
// the group's last position are zeroed in shared memory, and non-finite elements of values that
// only some of its rows see are taken out there and added back row by row.
//
// Every mbarrier wait is bounded; one that gives up sets SPEC_DEV_WAIT_TIMEOUT and the CTA's abort
// flag, after which no role waits or issues any more.  When all have ended, the loads and products
// in flight land (bounded again), the rows of the CTA's share become NaN, and TMEM is freed.
#include <cuda.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "spec_bench.h"
#include "spec_chunk.h"
#include "spec_verify.h"
#include "attn_common.cuh"
#include "chunk_plan.cuh"
#include "device_common.cuh"

namespace {

using namespace spec_dev;
using namespace spec_attn;

constexpr int SOFT_THREADS = 256;
constexpr int THREADS = SOFT_THREADS + 128;
// 384 threads launch with 168 registers each, 64512; a softmax thread holds a
// row's 128 scores: 256 * 208 + 128 * 88 = 64512
constexpr int SOFT_REGS = 208, HELPER_REGS = 88;
constexpr int MAX_CTAS = 192;     // the grid's and the workspace's bound
constexpr int RING = 4;           // pieces handed out ahead

template <int NP>
struct Cfg {
    static constexpr int KST = NP == 2 ? 3 : 4;
    static constexpr int VST = NP == 2 ? 2 : 4;
    static constexpr int TILE = NP * PANEL_BYTES;
    static constexpr int DP = NP * PANEL;  // columns of O
};
// Stages are taken in the order of the CTA's tiles.  A wait for a phase of a barrier tells it from
// the phase before only if that one is known to be over (parity).  The loader and the warp that waits
// for the issuer's tiles wait for all phases of a stage.  A softmax group waits only for the V of masked
// tiles, and before it waits for that tile's scores.  It has had the scores of tile c - 1 by then, which
// the products with V of tile c - 2 precede, or, in a piece's first tile, the last products of the
// piece before, with V of tile c - 1.  So V of tile c - 2 has landed, and a stage of V must not be
// taken again sooner than two tiles later.
static_assert(Cfg<1>::VST >= 2 && Cfg<2>::VST >= 2, "a group may wait for V two tiles ahead");

// A run of one item's key tiles inside a CTA's share.
struct Piece {
    int b, h;
    int row0, ntok;  // the group's rows
    int pos0;        // its first token's position
    int tile0, n;    // first tile and number of tiles (0: the share has ended)
    int tiles;       // of the whole item
    int idle;        // nothing to compute: a sequence in error
    int turn;        // the whole tiles are taken from this one on, and then from the first
    int first;       // 1 when the share starts inside the item or with it
};

struct Tail {
    unsigned long long kfull[4], kempty[4], vfull[4], vempty[4];
    unsigned long long qfull, qempty, sfull[2], halfdone[2], pvdone[2], vclean[2], drain;
    unsigned long long pfull[RING], pempty[RING];
    Piece piece[RING];
    uint32_t tmem_base;
    int abort_flag;
    uint32_t loaded[3];  // loads that were issued when their warp ended: tiles of K, of V, and Qs
    int issuer_out;      // the issuer has left
    int go[2][2];        // what the waits of a group came to, alternating
    uint16_t bad[4][8];     // keys of a masked tile with non-finite values, 16 for each warp that looked
};

template <int NP>
constexpr size_t smem_bytes()
{
    using C = Cfg<NP>;
    return (size_t)C::TILE * (2 + C::KST + C::VST) + sizeof(Tail);
}
static_assert(smem_bytes<2>() <= 232448 && smem_bytes<1>() <= 232448, "227 KB per CTA");

struct KParams {
    const uint8_t *plan;
    ChunkLayout lay;
    const int32_t *page_table;
    const void *v_cache;
    int64_t v_cache_stride[3];
    void *out;
    float *lse;
    int *status;
    float *part;     // [ctas][2 tiles][2][DP][BM] unnormalised sums of split items
    float2 *part_ml; // [ctas][2 tiles][2][BM] (log2 of the weights' unit, total)
    float c;         // scale * log2(e)
    int Hq, Hkv, D, G;
    int tokens_per_tile;
    int slots;       // CTAs
    int join_rows;   // rows of a join CTA: 32, or the least power of two that holds them
    int page_size, pages_per_seq;
    int page_rows;   // rows of a cache box: min(128, page_size) (contiguous: 128)
    int wide_rows;   // 1 where rows of out start on 32 bytes
    int lose, lose_after;  // the self-test's CTA (-1: none) and the pieces that it hands out first
};

// ------------------------------------------------------------------- work

// Where a unit (a key tile of an item) lies: its head, its row group, and the tile in it.
struct Place {
    int h, g, tile;
    int groups;
    long long total;  // units of one head
    ChunkGroup x;
    int status;
};

__device__ __forceinline__ void load_group(const KParams &P, Place &q)
{
    const int4 *at = reinterpret_cast<const int4 *>(P.plan + P.lay.group) + 2 * (size_t)q.g;
    const int4 a = __ldg(at), b = __ldg(at + 1);
    q.x.b = a.x;
    q.x.row0 = a.y;
    q.x.ntok = a.z;
    q.x.tiles = a.w;
    q.x.pos0 = b.x;
    q.x.bad = b.y;
    q.status = __ldg(reinterpret_cast<const int *>(P.plan + P.lay.status) + a.x);
}

// What a look-up begins with: the plan's totals, and, on its way beside them, each lane's first
// probe of the running sums (by the groups that there may be: how many there are is not known yet).
__device__ __forceinline__ Place empty_place(const KParams &P, long long &probe)
{
    const long long *cum = reinterpret_cast<const long long *>(P.plan + P.lay.cum);
    const int i = ((int)threadIdx.x & 31) * ((P.lay.most + 31) / 32);
    Place q = {};
    const int4 head = __ldg(reinterpret_cast<const int4 *>(P.plan));
    probe = i < P.lay.most ? __ldg(cum + i) : 0;
    q.groups = head.y;
    q.total = (long long)((unsigned long long)(unsigned int)head.w << 32 | (unsigned int)head.z);
    return q;
}

// A warp looks up unit u < total * Hkv: 32 probes of the plan's running sums a round, the last of them
// with the groups themselves.  (A chain of three loads up to 1024 groups, and the status.)
__device__ __forceinline__ void look_up(const KParams &P, long long u, long long probe, Place &q)
{
    const long long *cum = reinterpret_cast<const long long *>(P.plan + P.lay.cum);
    const int lane = (int)threadIdx.x & 31;
    q.h = (int)(u / q.total);
    const long long at = u - q.h * q.total;
    int step = (P.lay.most + 31) / 32, lo = 0, len = q.groups;
    bool below = lane * step < len && probe <= at;
    while (true) {
        const int last = 31 - __clz((int)__ballot_sync(0xffffffffu, below));
        lo += last * step;
        len = len - last * step < step ? len - last * step : step;
        if (len <= 32)
            break;
        step = (len + 31) / 32;
        below = lane * step < len && __ldg(cum + lo + lane * step) <= at;
    }
    long long before = 0;
    int4 a = {}, b = {};
    if (lane < len) {
        const int4 *group = reinterpret_cast<const int4 *>(P.plan + P.lay.group) + 2 * (size_t)(lo + lane);
        before = __ldg(cum + lo + lane);
        a = __ldg(group);
        b = __ldg(group + 1);
    }
    const int in = 31 - __clz((int)__ballot_sync(0xffffffffu, lane < len && before <= at));
    q.g = lo + in;
    q.tile = (int)(at - __shfl_sync(0xffffffffu, before, in));
    q.x.b = __shfl_sync(0xffffffffu, a.x, in);
    q.x.row0 = __shfl_sync(0xffffffffu, a.y, in);
    q.x.ntok = __shfl_sync(0xffffffffu, a.z, in);
    q.x.tiles = __shfl_sync(0xffffffffu, a.w, in);
    q.x.pos0 = __shfl_sync(0xffffffffu, b.x, in);
    q.x.bad = __shfl_sync(0xffffffffu, b.y, in);
    q.status = __ldg(reinterpret_cast<const int *>(P.plan + P.lay.status) + q.x.b);
}

// A CTA's share: `per` units for each of the slots that have any.
__device__ __forceinline__ long long share(const KParams &P, long long all)
{
    return (all + P.slots - 1) / P.slots;
}

// The pieces of a CTA's share, one after the other (a warp's walk, all lanes alike).
struct Walk {
    Place q;
    long long u0, u1, u, per;

    __device__ __forceinline__ Walk(const KParams &P, int slot)
    {
        long long probe;
        q = empty_place(P, probe);
        const long long all = q.total * P.Hkv;
        per = share(P, all);
        u0 = slot * per;
        u1 = u0 + per < all ? u0 + per : all;
        u = u0;
        if (u < u1)
            look_up(P, u, probe, q);
    }
    __device__ __forceinline__ Piece piece() const
    {
        const long long left = u1 - u;
        Piece p;
        p.b = q.x.b;
        p.h = q.h;
        p.row0 = q.x.row0;
        p.ntok = q.x.ntok;
        p.pos0 = q.x.pos0;
        p.tile0 = q.tile;
        p.tiles = q.x.tiles;
        p.n = left <= 0 ? 0 : p.tiles - q.tile < left ? p.tiles - q.tile : (int)left;
        p.idle = q.x.bad | (q.status != 0);
        p.first = u - q.tile <= u0;
        p.turn = piece_turn(u - u0, q.tile, p.tiles, per);
        return p;
    }
    // to the piece behind this one of n tiles
    __device__ __forceinline__ void go_on(const KParams &P, int n)
    {
        u += n;
        q.tile = 0;
        if (++q.g == q.groups) {
            q.g = 0;
            ++q.h;
        }
        if (u < u1)
            load_group(P, q);
    }
};

// The group's rows of one head become NaN, by the softmax warps.
__device__ __forceinline__ void void_rows(const KParams &P, int h, int row0, int ntok, int tid)
{
    for (int y = tid; y < ntok * P.G; y += SOFT_THREADS) {
        const int64_t row = ((int64_t)row0 + y / P.G) * P.Hq + (int64_t)h * P.G + y % P.G;
        for (int d = 0; d < P.D; d += 8)
            *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(P.out) + row * P.D + d) =
                make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
        if (P.lse)
            P.lse[row] = NAN;
    }
}

// A CTA that has given up leaves NaN, not what memory held before: in the statistics of its
// pieces of split items, whose rows the join then makes NaN, and in the rows that it was to
// write itself.
__device__ __noinline__ void void_share(const KParams &P, int slot, int tid)
{
    for (int i = tid; i < 2 * 2 * BM; i += SOFT_THREADS)
        P.part_ml[(size_t)slot * 2 * 2 * BM + i] = make_float2(NAN, NAN);
    Walk walk(P, slot);
    while (true) {
        const Piece p = walk.piece();
        if (p.n == 0)
            break;
        if (p.tile0 == 0)
            void_rows(P, p.h, p.row0, p.ntok, tid);
        walk.go_on(P, p.n);
    }
}

// Keys of tile `jt` of a group: those up to its last token's position.
__device__ __forceinline__ int tile_keys(const Piece &p, int jt)
{
    const int left = p.pos0 + p.ntok - jt * KT;
    return left < KT ? left : KT;
}

// Named barriers: a softmax group among itself; its weights of a tile's first and second half, for the
// issuer; the tiles of a step, for the issuer, one for each stage of V; a piece's first tiles.
enum { GROUP = 1, WEIGHTS = 3, TILES = 7, FIRST = 11 };

__device__ __forceinline__ void named_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void named_arrive(int id, int threads)
{
    __syncwarp();
    asm volatile("bar.arrive %0, %1;" :: "r"(id), "r"(threads) : "memory");
}

// 32 bytes to an address that they divide
__device__ __forceinline__ void store32(void *p, const uint32_t *w)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]),
                    "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Not 0 where one of a word's two elements is an infinity or NaN: its exponent, all ones, carries
// into the sign's place.
template <int DT>
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t w)
{
    constexpr uint32_t exponent = DT == SPEC_BF16 ? 0x7f807f80u : 0x7c007c00u;
    constexpr uint32_t one = DT == SPEC_BF16 ? 0x00800080u : 0x04000400u;
    return ((w & exponent) + one) & 0x80008000u;
}

template <int NP, int DT>
__global__ void __launch_bounds__(THREADS, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mkc,
                 const __grid_constant__ CUtensorMap mvc, const __grid_constant__ KParams P)
{
    using C = Cfg<NP>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t q_s = smem_addr(smem);
    const uint32_t k_s = q_s + 2 * C::TILE, v_s = k_s + C::KST * C::TILE;
    uint8_t *v_p = smem + (size_t)C::TILE * (2 + C::KST);
    Tail &S = *reinterpret_cast<Tail *>(smem + (size_t)C::TILE * (2 + C::KST + C::VST));
    volatile int *abort_flag = &S.abort_flag;
    const int tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int slot = (int)blockIdx.x;

    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&S.kfull[i], 1);
            mbar_init(&S.kempty[i], 1);
            mbar_init(&S.vfull[i], 1);
            mbar_init(&S.vempty[i], 1);
        }
        mbar_init(&S.qfull, 1);
        mbar_init(&S.qempty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.sfull[i], 1);
            mbar_init(&S.halfdone[i], 1);
            mbar_init(&S.pvdone[i], 1);
            mbar_init(&S.vclean[i], 8);
        }
        for (int i = 0; i < RING; ++i) {
            mbar_init(&S.pfull[i], 1);
            mbar_init(&S.pempty[i], 11);  // every warp but the one that writes
        }
        mbar_init(&S.drain, 1);
        S.abort_flag = 0;
        S.issuer_out = 0;
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
    // themselves could part, and wait for each other in the next test for good.
    auto given_up = [&]() -> bool { return __any_sync(0xffffffffu, *abort_flag != 0); };
    // A warp's wait: false on every lane once the CTA has given up.
    auto wait = [&](unsigned long long *bar, uint32_t parity) -> bool {
#pragma unroll 1
        for (int i = 0; i < WAIT_TRIES; ++i) {
            if (warp_try(bar, parity))
                return true;
            if ((i & 15) == 15 && given_up())
                return false;
        }
        give_up(abort_flag, P.status);
        return false;
    };
    // the same for a warp that has time: it sleeps between its tests
    auto wait_idle = [&](unsigned long long *bar, uint32_t parity, int tries = WAIT_TRIES) -> bool {
#pragma unroll 1
        for (int i = 0; i < tries; ++i) {
            if (warp_try(bar, parity))
                return true;
            if ((i & 15) == 15 && given_up())
                return false;
            __nanosleep(40);
        }
        give_up(abort_flag, P.status);
        return false;
    };
    // The next piece of the share, where it lies (the one before is given back with that): false
    // when there is none or the CTA has given up.
    uint32_t taken = 0;
    const Piece *piece = S.piece;
    auto next = [&](auto wait_for) -> bool {
        if (taken > 0 && lane == 0)
            mbar_arrive(&S.pempty[(taken - 1) % RING]);
        __syncwarp();
        const int at = (int)(taken % RING);
        if (!wait_for(&S.pfull[at], (taken / RING) & 1u))
            return false;
        piece = &S.piece[at];
        ++taken;
        return piece->n > 0;
    };
    // tiles of a piece that every row of the group sees whole
    auto plain_tiles = [](const Piece &p) -> int {
        const int whole = (p.pos0 + 1) / KT - p.tile0;
        return whole < 0 ? 0 : whole < p.n ? whole : p.n;
    };

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(SOFT_REGS));
        // ---------------------------------------------------- softmax groups
        const int s = warp >> 2;                 // the group, and its row tile
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;       // row of the tile
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t t_s = tmem + lanes + (uint32_t)(s * KT);
        const uint32_t t_o = tmem + lanes + (uint32_t)(2 * KT + s * C::DP);
        const int local = r / P.G;               // token of the row, counted in the tile
        const int g = r - local * P.G;
        const int tok = s * P.tokens_per_tile + local;  // and in the group
        uint32_t cnt = 0, hid = 0, pieces = 0;   // tiles, masked ones among them, pieces
        int vst = 0;                             // stage and phase of the next V tile
        uint32_t vph = 0;
        const unsigned long long c2 = f2(P.c, P.c);
        // a score x has weight 2^(x c + shift) under the maximum m
        auto shift_of = [&](float m) -> float {
            return m == -INFINITY ? 0.0f : fmaf(-m, P.c, lift<DT>());
        };
        // A group's wait: its first warp tests the barrier, the others are held without a
        // test at a named one (tests by all of them took half of the kernel's instructions, and
        // of the issue slots of the warps that had work).  The group leaves as one where the wait
        // has given up, so none is left at the named barrier.
        uint32_t waits = 0;
        auto wait_group = [&](unsigned long long *bar, uint32_t parity) -> bool {
            volatile int *go = &S.go[s][waits++ & 1u];
            if (quarter == 0) {
                const bool there = wait(bar, parity);
                if (lane == 0)
                    *go = there;
            }
            __syncwarp();
            named_sync(GROUP + s, 128);
            return *go != 0;
        };
        bool ok = true;
        while (ok && next(wait_group)) {
            const Piece &p = *piece;
            if (p.idle) {
                if (p.tile0 == 0)
                    void_rows(P, p.h, p.row0, p.ntok, tid);
                continue;
            }
            const bool live = local < P.tokens_per_tile && tok < p.ntok;
            const bool warp_live = __any_sync(0xffffffffu, live);
            float m = -INFINITY, l = 0.0f;       // maximum of the raw scores, total
            const int plain = plain_tiles(p);
            // keys 32 h on of tile jt that this row sees, as bits
            auto bits = [&](int jt, int h) -> uint32_t {
                const int left = min(tile_keys(p, jt), p.pos0 + tok + 1 - jt * KT) - h * 32;
                return left >= 32 ? ~0u : left <= 0 ? 0u : (1u << left) - 1u;
            };
            // What the zeroed elements of a masked tile's values give the rows that see them, once
            // its O is done.
            auto add_back = [&](int jt, uint32_t slot) {
                const volatile uint32_t *notes = reinterpret_cast<const uint32_t *>(S.bad[slot & 3u]);
                if ((notes[0] | notes[1] | notes[2] | notes[3]) == 0 || !warp_live)
                    return;
#pragma unroll 1
                for (int d = 0; d < C::DP; d += 32) {
                    uint32_t o[32];
                    tmem_ld(t_o + d, o);
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t left = live ? notes[q] & bits(jt, q) : 0u;
                        while (left) {
                            const int key = jt * KT + q * 32 + __ffs((int)left) - 1;
                            left &= left - 1;
                            const int e = key / P.page_size;
                            const int64_t page = P.page_table
                                ? __ldg(P.page_table + (size_t)p.b * P.pages_per_seq + e) : p.b;
                            const uint16_t *src = reinterpret_cast<const uint16_t *>(P.v_cache) +
                                page * P.v_cache_stride[0] +
                                (key - e * P.page_size) * P.v_cache_stride[1] +
                                p.h * P.v_cache_stride[2];
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (d + j < P.D) {
                                    const uint32_t v = src[d + j];
                                    if (nonfinite<DT>(v) & 0xffffu)
                                        o[j] = __float_as_uint(__uint_as_float(o[j]) + unpack1<DT>(v));
                                }
                        }
                    }
                    tmem_st(t_o + d, o);
                }
                tmem_wait_st();
            };
            // The tiles; in a masked one (the last ones) some keys are hidden from some rows.  What a
            // few tiles need beside the common way stands in small loops of its own: unrolled
            // variants of that way, run once in 30 tiles, took three times its time, most of it
            // for their instructions to arrive.
            for (int i = 0; i < p.n && ok; ++i) {
                const bool masked = i >= plain;
                const int jt = p.tile0 + i;
                if (masked) {
                    // V, while the scores are on their way: rows past the keys (up to the last
                    // product's 16) are zeroed; of keys that some row does not see, non-finite
                    // elements are noted and zeroed.  16 rows for each warp of both groups
                    ok = wait_group(&S.vfull[vst], vph);
                    if (!ok)
                        break;
                    const int keys = tile_keys(p, jt), r0 = warp * 16;
                    uint32_t found = 0;
                    uint8_t *at = v_p + (size_t)vst * C::TILE + (r0 + (lane >> 3)) * 128 +
                                  (lane & 7) * 16;
                    uint32_t any = 0;
#pragma unroll
                    for (int x = 0; x < NP * 4; ++x) {  // 4 rows of a panel, 8 lanes each
                        const int row = r0 + (x & 3) * 4 + (lane >> 3);
                        const uint4 w = *reinterpret_cast<const uint4 *>(at + (x >> 2) * PANEL_BYTES +
                                                                         (x & 3) * 512);
                        const uint32_t f = nonfinite_bits<DT>(w.x) | nonfinite_bits<DT>(w.y) |
                                           nonfinite_bits<DT>(w.z) | nonfinite_bits<DT>(w.w);
                        any |= row < keys && jt * KT + row > p.pos0 ? f : 0u;
                    }
                    // (seldom: one warp has rows past the keys, if any, and such values are rare)
                    if (__any_sync(0xffffffffu, any != 0) || (keys > r0 && keys < r0 + 16)) {
#pragma unroll 1
                        for (int x = 0; x < NP * 4; ++x) {
                            const int row = r0 + (x & 3) * 4 + (lane >> 3);
                            uint4 *v = reinterpret_cast<uint4 *>(at + (x >> 2) * PANEL_BYTES +
                                                                 (x & 3) * 512);
                            uint4 w = *v;
                            const uint4 f = make_uint4(nonfinite<DT>(w.x), nonfinite<DT>(w.y),
                                                       nonfinite<DT>(w.z), nonfinite<DT>(w.w));
                            const bool past = row >= keys && row < ((keys + 15) & ~15);
                            const bool bad = row < keys && jt * KT + row > p.pos0 &&
                                             (f.x | f.y | f.z | f.w) != 0;
                            if (past || bad)
                                *v = past ? make_uint4(0, 0, 0, 0)
                                          : make_uint4(w.x & ~f.x, w.y & ~f.y, w.z & ~f.z, w.w & ~f.w);
                            const uint32_t who = __ballot_sync(0xffffffffu, bad);
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                found |= ((who >> (8 * y)) & 0xffu ? 1u : 0u) << ((x & 3) * 4 + y);
                        }
                    }
                    if (lane == 0)
                        S.bad[hid & 3u][warp] = (uint16_t)found;
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&S.vclean[hid & 1u]);
                }
                // the scores are there, and the group's product before is done
                ok = wait_group(&S.sfull[s], cnt & 1u);
                if (!ok)
                    break;
                tc_fence_after();
                if (masked && i > plain)
                    add_back(jt - 1, hid - 1);
                if (warp_live) {
                    if (masked) {
#pragma unroll 1
                        for (int h = 0; h < 4; ++h) {
                            const uint32_t see = bits(jt, h);
                            if (__all_sync(0xffffffffu, see == ~0u))
                                continue;
                            uint32_t x[32];
                            tmem_ld(t_s + h * 32, x);
                            hide(x, see);
                            tmem_st(t_s + h * 32, x);
                        }
                        tmem_wait_st();
                    }
                    if (i == 0) {
                        m = -INFINITY;
#pragma unroll 1
                        for (int h = 0; h < 4; ++h) {
                            uint32_t x[32];
                            tmem_ld(t_s + h * 32, x);
                            m = fmaxf(m, max32(x));
                        }
                    }
                }
                // The tile in two halves, whose products begin one after the other: the first one's
                // runs while the second one's weights are made.  Each in one pass: weights by
                // the maximum so far, which serves as long as no score is far above it; the
                // half's own maximum is found on the way.  Weights 32 h on lie in columns 16 h on,
                // over scores that have been read.
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    if (warp_live) {
                        unsigned long long sum[2];
                        uint32_t x[32], y[32], pk[2][16];
                        while (true) {  // (twice at most: by the new maximum nothing has grown)
                            const float shift = shift_of(m);
                            const unsigned long long shift2 = f2(shift, shift);
                            sum[0] = sum[1] = 0ull;
                            __syncwarp();
                            tmem_ld_start(t_s + part * 64, x);
                            tmem_ld_finish(x);
                            tmem_ld_start(t_s + part * 64 + 32, y);
                            float top = max32(x);
                            weigh<DT>(x, c2, shift2, sum, pk[0]);
                            tmem_ld_finish(y);
                            top = fmaxf(top, max32(y));
                            weigh<DT>(y, c2, shift2, sum, pk[1]);
                            const bool grown = (top - m) * P.c > growth<DT>();  // -inf to finite too
                            if (!__any_sync(0xffffffffu, grown))
                                break;
                            // again, by the new maximum, which O and l follow (O when it has the
                            // first half; a wait that gives up ends the group's next one)
                            if (part) {
                                (void)wait(&S.halfdone[s], cnt & 1u);
                                tc_fence_after();
                            }
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
                        }
                        tmem_st(t_s + part * 32, pk[0]);
                        tmem_st(t_s + part * 32 + 16, pk[1]);
                        float s0, s1;
                        f2_split(add2(sum[0], sum[1]), s0, s1);
                        l += s0 + s1;
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    named_arrive(WEIGHTS + 2 * part + s, 160);
                }
                ++cnt;
                vph ^= vst + 1 == C::VST ? 1u : 0u;
                vst = vst + 1 == C::VST ? 0 : vst + 1;
                hid += masked ? 1u : 0u;
            }
            ok = ok && wait_group(&S.pvdone[s], pieces++ & 1u);
            if (!ok)
                break;
            tc_fence_after();
            if (p.n > plain)
                add_back(p.tile0 + p.n - 1, hid - 1);
            const float top = m != -INFINITY ? -shift_of(m) : -INFINITY;
            const float sum = l, base = top == -INFINITY ? 0.0f : top;
            // a row that saw no key has no weight, whatever its O holds
            const bool some = !(top == -INFINITY && sum == 0.0f);
            if (warp_live) {
                const bool whole = p.n == p.tiles;
                const int64_t orow = ((int64_t)p.row0 + tok) * P.Hq + (int64_t)p.h * P.G + g;
                const size_t at = (((size_t)slot * 2 + s) * 2 + (p.first ? 0 : 1)) * BM;
                const float norm = sum != 0.0f && some ? 1.0f / sum : 0.0f;
                uint16_t *to = reinterpret_cast<uint16_t *>(P.out) + orow * P.D;
#pragma unroll 1
                for (int d0 = 0; d0 < C::DP && d0 < P.D; d0 += 16) {
                    uint32_t a[16];
                    tmem_ld(t_o + (uint32_t)d0, a);
                    if (!live)
                        continue;
                    if (!whole) {
                        // [column][row]: a warp's store is one line (columns past D have their room)
                        float *o = P.part + at * C::DP + d0 * BM + r;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            o[j * BM] = some ? __uint_as_float(a[j]) : 0.0f;
                        continue;
                    }
                    uint32_t u[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        u[j] = norm != 0.0f ? pack<DT>(__uint_as_float(a[2 * j]) * norm,
                                                       __uint_as_float(a[2 * j + 1]) * norm) : 0u;
                    if (P.wide_rows) {
                        store32(to + d0, u);  // a lane's store is a whole sector of its row
                    } else {
                        *reinterpret_cast<uint4 *>(to + d0) = make_uint4(u[0], u[1], u[2], u[3]);
                        if (d0 + 8 < P.D)
                            *reinterpret_cast<uint4 *>(to + d0 + 8) = make_uint4(u[4], u[5], u[6], u[7]);
                    }
                }
                if (live) {
                    if (!whole)
                        P.part_ml[at + r] = make_float2(top, sum);
                    else if (P.lse)
                        P.lse[orow] = lse_of(base, sum);
                }
            }
            tc_fence_before();
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(HELPER_REGS));
        if (warp == 8) {
            // ------------------------------------------------ TMA of K and V
            // tiles that a load was issued for, and the next one's stage and phase: of K and of V
            uint32_t loaded[2] = {0, 0}, phase[2] = {1, 1};
            int stage[2] = {0, 0};
            bool ok = true;
            while (ok && next(wait_idle)) {
                const Piece &p = *piece;
                if (p.idle)
                    continue;
                const int rows = P.page_rows, at = lane * rows;  // a box of rows per lane
                const int plain = plain_tiles(p), turn = p.turn < plain ? p.turn : 0;
                for (int i = 0; i < p.n && ok; ++i) {
                    int jt = p.tile0 + i;
                    if (i < plain)
                        jt += i + turn < plain ? turn : turn - plain;
                    const int keys = tile_keys(p, jt);
                    const bool mine = at < keys;
                    int y = jt * KT + at, w = p.b;
                    if (P.page_table && mine) {
                        const int e = y / P.page_size;
                        w = __ldg(P.page_table + (size_t)p.b * P.pages_per_seq + e);
                        y -= e * P.page_size;
                    }
                    const uint32_t bytes = (uint32_t)(((keys + rows - 1) / rows) * rows * 128 * NP);
#pragma unroll
                    for (int side = 0; side < 2 && ok; ++side) {
                        const int st = stage[side];
                        unsigned long long *full = side ? &S.vfull[st] : &S.kfull[st];
                        ok = wait_idle(side ? &S.vempty[st] : &S.kempty[st], phase[side]);
                        if (!ok)
                            break;
                        if (lane == 0)
                            mbar_arrive_expect_tx(full, bytes);
                        __syncwarp();
                        if (mine) {
                            const uint32_t dst =
                                (side ? v_s : k_s) + (uint32_t)(st * C::TILE + at * 128);
#pragma unroll
                            for (int d = 0; d < NP; ++d)
                                tma_load_4d(dst + d * PANEL_BYTES, side ? &mvc : &mkc, d * PANEL, y,
                                            p.h, w, full);
                        }
                        __syncwarp();
                        ++loaded[side];
                        const bool last = st + 1 == (side ? C::VST : C::KST);
                        stage[side] = last ? 0 : st + 1;
                        phase[side] ^= last ? 1u : 0u;
                    }
                }
            }
            if (lane == 0) {
                S.loaded[0] = loaded[0];
                S.loaded[1] = loaded[1];
            }
        } else if (warp == 9) {
            // -------------------------------------------- issuer of the products
            // The whole warp runs the loop and one elected lane issues: what the products are
            // given then stays in uniform registers.  A step of group G: O(i) += P V(i), then
            // S = Q K(i + 1)^T.  It tests no mbarrier in its loop: a test of one that is ready takes
            // 100 to 200 clocks, in which the tensor pipe runs dry, a named barrier's sync
            // about 30.  The weights come by one from the softmax groups, the tiles by one from
            // the next warp, which tests theirs.  Where a CTA has given up that warp frees this one.
            bool ok = true;
            const int ksteps = (P.D + 15) / 16;
            const bool all_steps = ksteps == NP * 4;
            const uint32_t id_o = idesc<DT>(ksteps * 16, true);
            int kst = 0, vst = 0;                // stages of the next K and V tile
            constexpr uint32_t id_s = idesc<DT>(KT, false);
            const uint64_t qd0 = desc_k(q_s), kd0 = desc_k(k_s), vd0 = desc_mn(v_s);
            constexpr uint64_t TILE16 = C::TILE >> 4;
            // S = Q K^T of group s by the elected lane, and what it commits; `last` of the piece
            auto scores = [&](int s, uint32_t id, bool last) {
                const uint32_t d = tmem + (uint32_t)(s * KT);
                const uint64_t qd = qd0 + s * TILE16, kd = kd0 + kst * TILE16;
                if (all_steps) {
#pragma unroll
                    for (int x = 0; x < NP * 4; ++x) {
                        const uint64_t off = (uint64_t)(((x >> 2) * PANEL_BYTES + (x & 3) * 32) >> 4);
                        mma_ss(d, qd + off, kd + off, id, x ? 1u : 0u);
                    }
                } else {
#pragma unroll 1
                    for (int x = 0; x < ksteps; ++x) {
                        const uint64_t off = (uint64_t)(((x >> 2) * PANEL_BYTES + (x & 3) * 32) >> 4);
                        mma_ss(d, qd + off, kd + off, id, x ? 1u : 0u);
                    }
                }
                if (s)
                    mma_commit(&S.kempty[kst]);
                mma_commit(&S.sfull[s]);
                if (last && s)
                    mma_commit(&S.qempty);
            };
            while (ok && next(wait)) {
                const Piece &p = *piece;
                if (p.idle)
                    continue;
                const int n = p.n, plain = plain_tiles(p);
                // only a group's last tile can have fewer than KT keys
                const int tail = tile_keys(p, p.tile0 + n - 1);
                const uint32_t id_tail = idesc<DT>((tail + 15) & ~15, false);
                named_sync(FIRST, 64);
                ok = !given_up();
                if (!ok)
                    break;
                tc_fence_after();
                if (elect_one()) {
                    scores(0, n == 1 ? id_tail : id_s, n == 1);
                    scores(1, n == 1 ? id_tail : id_s, n == 1);
                }
                __syncwarp();
                kst = kst + 1 == C::KST ? 0 : kst + 1;
                auto step = [&](auto group, int i) {
                    constexpr int G = decltype(group)::value;
                    const uint32_t t_s = tmem + (uint32_t)(G * KT);
                    const uint32_t t_o = tmem + (uint32_t)(2 * KT + G * C::DP);
                    const uint64_t vd = vd0 + vst * TILE16;
                    const uint32_t more = i >= 1 ? 1u : 0u;
                    const bool end = i + 1 == n;
                    if (G == 0)  // (the second group finds the first one's tiles)
                        named_sync(TILES + vst, 64);
                    // 16 keys a product: 8 columns of P, 2 KB of V
                    auto products = [&](int from, int to) {
#pragma unroll 1
                        for (int x = from; x < to; ++x)
                            mma_ts(t_o, t_s + (uint32_t)(x * 8), vd + (uint64_t)(x * (2048 >> 4)),
                                   id_o, x ? 1u : more);
                    };
                    const bool full = !end || tail == KT;
                    const int some = (tail + 15) / 16;
                    named_sync(WEIGHTS + G, 160);
                    tc_fence_after();
                    if (elect_one()) {
                        if (full) {
#pragma unroll
                            for (int x = 0; x < KT / 32; ++x)
                                mma_ts(t_o, t_s + (uint32_t)(x * 8), vd + (uint64_t)(x * (2048 >> 4)),
                                       id_o, x ? 1u : more);
                        } else {
                            products(0, some < KT / 32 ? some : KT / 32);
                        }
                        mma_commit(&S.halfdone[G]);
                    }
                    __syncwarp();
                    named_sync(WEIGHTS + 2 + G, 160);
                    ok = !given_up();
                    if (!ok)
                        return;
                    tc_fence_after();
                    if (elect_one()) {
                        if (full) {
#pragma unroll
                            for (int x = KT / 32; x < KT / 16; ++x)
                                mma_ts(t_o, t_s + (uint32_t)(x * 8), vd + (uint64_t)(x * (2048 >> 4)),
                                       id_o, 1u);
                        } else {
                            products(KT / 32, some);
                        }
                        if (G)
                            mma_commit(&S.vempty[vst]);
                        if (end)
                            mma_commit(&S.pvdone[G]);
                        else
                            scores(G, i + 2 == n ? id_tail : id_s, i + 2 == n);
                    }
                    __syncwarp();
                    if (G) {
                        if (!end)
                            kst = kst + 1 == C::KST ? 0 : kst + 1;
                        vst = vst + 1 == C::VST ? 0 : vst + 1;
                    }
                };
                for (int i = 0; i < n && ok; ++i) {
                    step(Int<0>(), i);
                    if (ok)
                        step(Int<1>(), i);
                }
            }
            if (lane == 0)
                *(volatile int *)&S.issuer_out = 1;
        } else if (warp == 10) {
            // -------------------------------- waits for the issuer's tiles, some steps ahead of it
            // (A stage's barrier is come to again only when its V has been loaded again, so after the
            // issuer has been there; the first one when Q has been.)
            bool ok = true;
            int kst = 0, vst = 0;
            uint32_t kph = 0, vph = 0, items = 0, hid = 0;
            auto wait_k = [&]() -> bool {
                const bool there = wait(&S.kfull[kst], kph);
                kph ^= kst + 1 == C::KST ? 1u : 0u;
                kst = kst + 1 == C::KST ? 0 : kst + 1;
                return there;
            };
            while (ok && next(wait_idle)) {
                const Piece &p = *piece;
                if (p.idle)
                    continue;
                const int plain = plain_tiles(p);
                ok = wait(&S.qfull, items++ & 1u) && wait_k();
                if (ok)
                    named_arrive(FIRST, 64);
                for (int i = 0; i < p.n && ok; ++i) {
                    ok = wait(&S.vfull[vst], vph) && (i + 1 == p.n || wait_k());
                    if (ok && i >= plain) {
                        ok = wait(&S.vclean[hid & 1u], (hid >> 1) & 1u);
                        ++hid;
                    }
                    if (ok)
                        named_arrive(TILES + vst, 64);
                    vph ^= vst + 1 == C::VST ? 1u : 0u;
                    vst = vst + 1 == C::VST ? 0 : vst + 1;
                }
            }
            // The issuer's syncs have no limit of their own.  Once the CTA has given up, this warp comes
            // to all of them, again and again, until the issuer has left: whatever had come there
            // before, each fills up while the issuer waits at it.
            for (int i = 0; i < WAIT_TRIES; ++i) {
                if (__any_sync(0xffffffffu, *(volatile int *)&S.issuer_out != 0))
                    break;
                if (given_up()) {
                    for (int id = WEIGHTS; id < TILES; ++id)
                        named_arrive(id, 160);
                    for (int id = TILES; id <= FIRST; ++id)
                        named_arrive(id, 64);
                }
                __nanosleep(200);
            }
        } else {
            // ------------------------------- the share's pieces, and the TMA of their Q
            Walk walk(P, slot);
            uint32_t items = 0;
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
                if (!p.idle) {
                    if (!wait_idle(&S.qempty, (items & 1u) ^ 1u))
                        break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(
                            &S.qfull, (uint32_t)(P.tokens_per_tile * P.G * 128 * NP * 2));
                        for (int i = 0; i < NP * 2; ++i)
                            tma_load_4d(q_s + i * PANEL_BYTES, &mq, (i % NP) * PANEL, 0,
                                        p.row0 + (i / NP) * P.tokens_per_tile, p.h, &S.qfull);
                    }
                    __syncwarp();
                    ++items;
                }
                walk.go_on(P, p.n);
            }
            if (lane == 0)
                S.loaded[2] = items;
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
        } else if (warp == 11 && S.loaded[2] > 0) {
            (void)mbar_wait(&S.qfull, (S.loaded[2] - 1) & 1u);
        } else if (warp < 8) {
            void_share(P, slot, tid);
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

// Joins the pieces of the items that lie across a share's end.  CTA x takes the item that the end
// of share x cuts (when no earlier end cuts it), 32 rows of one of its row tiles: a row per lane,
// an eighth of the columns per warp.  Where there are fewer rows, the lanes left over take pieces
// of their own.  Bound by latency, 8 to 9 us cold for a few rows, and 14 us where every CTA left two
// pieces of 256 rows.
template <int NP, int DT>
__global__ void __launch_bounds__(JOIN_WARPS * 32, 4)
    chunk_join_kernel(const __grid_constant__ KParams P)
{
    using C = Cfg<NP>;
    constexpr int COLS = C::DP / JOIN_WARPS;
    __shared__ __align__(16) uint16_t tile[JOIN_ROWS][C::DP + 8];
    const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
    const int mine = lane & (P.join_rows - 1), part = lane / P.join_rows;
    const int parts = 32 / P.join_rows;
    const int r = (int)blockIdx.z * JOIN_ROWS + mine, s = (int)blockIdx.y;
    allow_next_kernel();
    // (the plan is complete: every CTA of the attention had waited for it before this grid began)
    long long probe;
    Place q = empty_place(P, probe);
    const long long all = q.total * P.Hkv, per = share(P, all);
    const long long end = ((long long)blockIdx.x + 1) * per;
    if (end < all)
        look_up(P, end, probe, q);
    wait_previous_kernel();
    if (end >= all)
        return;
    const long long item = end - q.tile;  // its first unit
    if (item == end || item < end - per || q.x.bad || q.status != 0)
        return;  // not cut here, or the previous end has it, or a sequence in error
    const int local = r / P.G, g = r - local * P.G;
    const int tok = s * P.tokens_per_tile + local;
    const bool live = local < P.tokens_per_tile && tok < q.x.ntok;
    const int64_t orow = ((int64_t)q.x.row0 + tok) * P.Hq + (int64_t)q.h * P.G + g;
    const int s0 = (int)blockIdx.x, n = (int)((item + q.x.tiles - 1) / per) - s0 + 1;
    // a share that starts with the item, or inside it, left its first piece; one that the item
    // starts inside of left its second
    auto at = [&](int k) -> size_t {
        const int which = (long long)(s0 + k) * per >= item ? 0 : 1;
        return (((size_t)(s0 + k) * 2 + s) * 2 + which) * BM;
    };
    float a_top = -INFINITY, a_sum = 0.0f, a_o[COLS];
    bool a_some = false;
#pragma unroll
    for (int j = 0; j < COLS; ++j)
        a_o[j] = 0.0f;
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
            float top = a_top;
#pragma unroll
            for (int u = 0; u < JOIN_UNROLL; ++u)
                top = fmaxf(top, ml[u].x);
            const float base = top == -INFINITY ? 0.0f : top;
            const float f = a_some ? ex2(a_top - base) : 0.0f;
            a_sum *= f;
#pragma unroll
            for (int j = 0; j < COLS; ++j)
                a_o[j] *= f;
#pragma unroll
            for (int u = 0; u < JOIN_UNROLL; ++u) {
                if (ml[u].x == -INFINITY && ml[u].y == 0.0f)
                    continue;  // no key seen there
                const float w = ex2(ml[u].x - base);
                a_sum = fmaf(ml[u].y, w, a_sum);
#pragma unroll
                for (int j = 0; j < COLS; ++j)
                    a_o[j] = fmaf(x[u][j], w, a_o[j]);
                a_some = true;
            }
            a_top = top;
        }
    for (int d = P.join_rows; d < 32; d <<= 1) {
        const float top2 = __shfl_xor_sync(0xffffffffu, a_top, d);
        const float sum2 = __shfl_xor_sync(0xffffffffu, a_sum, d);
        const bool some2 = __shfl_xor_sync(0xffffffffu, a_some ? 1 : 0, d) != 0;
        const float top = fmaxf(a_top, top2), base = top == -INFINITY ? 0.0f : top;
        const float f = a_some ? ex2(a_top - base) : 0.0f, f2 = some2 ? ex2(top2 - base) : 0.0f;
        a_sum = a_sum * f + sum2 * f2;
#pragma unroll
        for (int j = 0; j < COLS; ++j)
            a_o[j] = a_o[j] * f + __shfl_xor_sync(0xffffffffu, a_o[j], d) * f2;
        a_top = top;
        a_some |= some2;
    }
    const float norm = a_sum != 0.0f ? 1.0f / a_sum : 0.0f;
    if (part == 0) {
#pragma unroll
        for (int j = 0; j < COLS; j += 2)
            *reinterpret_cast<uint32_t *>(&tile[mine][warp * COLS + j]) =
                a_sum != 0.0f ? pack<DT>(a_o[j] * norm, a_o[j + 1] * norm) : 0u;
        if (warp == 0 && live && P.lse)
            P.lse[orow] = lse_of(a_top == -INFINITY ? 0.0f : a_top, a_sum);
    }
    __syncthreads();
    const uint32_t rows = __ballot_sync(0xffffffffu, live && part == 0);
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

bool heads_ok(int32_t Hq, int32_t Hkv, int32_t D)
{
    return Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 && Hq / Hkv <= BM && Hq <= 65535 && D >= 8 &&
           D % 8 == 0 && D <= SPEC_ATTN_MAX_HEAD_DIM;
}

struct WsLayout {
    size_t ml, part, total;
};

WsLayout ws_layout(int D)
{
    const size_t dp = D > PANEL ? 2 * PANEL : PANEL;
    WsLayout w;
    w.ml = 0;
    w.part = plan_align(w.ml + (size_t)MAX_CTAS * 2 * 2 * BM * sizeof(float2));
    w.total = plan_align(w.part + (size_t)MAX_CTAS * 2 * 2 * BM * dp * sizeof(float));
    return w;
}

struct DevInfo {
    std::atomic<int> sms;
    std::atomic<bool> attr[2][2];
};
DevInfo g_dev[64];

template <int NP, int DT>
int launch(const CUtensorMap (&maps)[3], KParams &P, int rows, int sms, DevInfo &di,
           cudaStream_t st)
{
    if (!di.attr[NP - 1][DT - 1].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(chunk_kernel<NP, DT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem_bytes<NP>()) != cudaSuccess) {
            (void)cudaGetLastError();
            return SPEC_ECUDA;
        }
        di.attr[NP - 1][DT - 1].store(true, std::memory_order_release);
    }
    P.slots = sms < MAX_CTAS ? sms : MAX_CTAS;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned int)P.slots);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem_bytes<NP>();
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, chunk_kernel<NP, DT>, maps[0], maps[1], maps[2], P) !=
        cudaSuccess) {
        (void)cudaGetLastError();
        return SPEC_ECUDA;
    }
    if (P.slots > 1) {
        const int most = P.tokens_per_tile < rows ? P.tokens_per_tile * P.G : rows * P.G;
        P.join_rows = JOIN_ROWS;
        while (P.join_rows / 2 >= most)
            P.join_rows /= 2;
        cfg.gridDim = dim3((unsigned int)(P.slots - 1), rows > P.tokens_per_tile ? 2u : 1u,
                           (unsigned int)((most + JOIN_ROWS - 1) / JOIN_ROWS));
        cfg.blockDim = dim3(JOIN_WARPS * 32);
        cfg.dynamicSmemBytes = 0;
        if (cudaLaunchKernelEx(&cfg, chunk_join_kernel<NP, DT>, P) != cudaSuccess) {
            (void)cudaGetLastError();
            return SPEC_ECUDA;
        }
    }
    return SPEC_OK;
}

}  // namespace

extern "C" {

size_t spec_chunk_attention_workspace_size(int32_t Hq, int32_t Hkv, int32_t D)
{
    return heads_ok(Hq, Hkv, D) ? ws_layout(D).total : 0;
}

// Whether an output shares memory with an input, by their extents, or with the other.  (out may be q
// itself: an item's queries are read by its own CTAs, which write its rows afterwards, the rows of split
// items by the join behind them all; what a box reads past a group's rows has no effect.)
static bool outputs_apart(const spec_chunk_attention_args &a, size_t plan_bytes)
{
    struct Span {
        const void *p;
        uint64_t bytes;
    };
    auto strided = [&](uint64_t n0, uint64_t s0, uint64_t n1, uint64_t s1, uint64_t n2, uint64_t s2) {
        return 2 * ((n0 - 1) * s0 + (n1 - 1) * s1 + (n2 - 1) * s2 + (uint64_t)a.D);
    };
    auto cache = [&](const int64_t (&s)[3]) -> uint64_t {
        return a.num_pages < 1 ? 0 : strided(a.num_pages, s[0], a.page_size, s[1], a.Hkv, s[2]);
    };
    auto apart = [](const Span &x, const Span &y) {
        const uintptr_t i = reinterpret_cast<uintptr_t>(x.p), j = reinterpret_cast<uintptr_t>(y.p);
        return !x.p || !y.p || i >= j + y.bytes || j >= i + x.bytes;
    };
    const bool in_place = a.out == a.q && (a.rows == 1 || a.q_stride[0] == (int64_t)a.Hq * a.D) &&
                          (a.Hq == 1 || a.q_stride[1] == a.D);
    const Span in[] = {
        {a.q, in_place ? 0 : strided(a.rows, a.q_stride[0], a.Hq, a.q_stride[1], 1, 0)},
        {a.k_cache, cache(a.k_cache_stride)}, {a.v_cache, cache(a.v_cache_stride)},
        {a.plan, plan_bytes}, {a.page_table, (uint64_t)a.B * a.pages_per_seq * 4}};
    const uint64_t heads = (uint64_t)a.rows * a.Hq;
    const Span out = {a.out, heads * a.D * 2}, lse = {a.out_lse, heads * 4};
    for (const Span &x : in)
        if (!apart(out, x) || !apart(lse, x))
            return false;
    return apart(out, lse);
}

static int32_t attend(const spec_chunk_attention_args *args, void *workspace,
                      size_t workspace_bytes, int lose, int lose_after, void *stream)
{
    if (!args)
        return SPEC_EINVAL;
    const spec_chunk_attention_args &a = *args;
    const bool paged = a.page_table != nullptr;
    if (!heads_ok(a.Hq, a.Hkv, a.D) || a.B < 0 || a.B > 65535 || a.rows < 0 ||
        a.rows > SPEC_CHUNK_MAX_ROWS || !page_size_ok(a.page_size, paged) || a.pages_per_seq < 1 ||
        a.num_pages < 0 ||
        (long long)a.pages_per_seq * a.page_size > INT32_MAX - SPEC_CHUNK_MAX_ROWS ||
        (a.dtype != SPEC_BF16 && a.dtype != SPEC_F16) || !(a.scale > 0.0f) || isinf(a.scale))
        return SPEC_EINVAL;
    if (a.B == 0 || a.rows == 0)
        return SPEC_OK;
    const void *bases[] = {a.q, a.k_cache, a.v_cache, a.out};
    for (const void *p : bases)
        if (!p || !aligned(p, 16))
            return SPEC_EINVAL;
    const int64_t qs3[3] = {a.q_stride[0], a.q_stride[1], 0};
    if (!strides_ok(qs3) || !strides_ok(a.k_cache_stride) || !strides_ok(a.v_cache_stride) ||
        !a.plan || !aligned(a.plan, 256) || !workspace || !aligned(workspace, 256) ||
        !aligned(a.page_table, 4) || !aligned(a.out_lse, 4) ||
        (!paged && (a.pages_per_seq != 1 || a.num_pages < a.B)))
        return SPEC_EINVAL;
    // TMA steps along a dimension by its stride: none may be 0 where there are two entries
    auto stepped = [&](const int64_t (&s)[3]) {
        return (a.num_pages < 2 || s[0] > 0) && (a.page_size < 2 || s[1] > 0) &&
               (a.Hkv < 2 || s[2] > 0);
    };
    if (!stepped(a.k_cache_stride) || !stepped(a.v_cache_stride) ||
        (a.rows > 1 && a.q_stride[0] == 0) || (a.Hq > 1 && a.q_stride[1] == 0))
        return SPEC_EINVAL;
    const WsLayout w = ws_layout(a.D);
    if (workspace_bytes < w.total)
        return SPEC_ENOSPACE;
    const int32_t G = a.Hq / a.Hkv;
    if (!outputs_apart(a, chunk_layout(a.B, a.rows, G).total))
        return SPEC_EINVAL;

    KParams P;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    P.plan = static_cast<const uint8_t *>(a.plan);
    P.lay = chunk_layout(a.B, a.rows, G);
    P.page_table = a.page_table;
    P.v_cache = a.v_cache;
    for (int i = 0; i < 3; ++i)
        P.v_cache_stride[i] = a.v_cache_stride[i];
    P.out = a.out;
    P.lse = a.out_lse;
    P.status = &reinterpret_cast<ChunkHeader *>(const_cast<void *>(a.plan))->status;
    P.part_ml = reinterpret_cast<float2 *>(ws + w.ml);
    P.part = reinterpret_cast<float *>(ws + w.part);
    P.c = a.scale * LOG2E;
    P.Hq = a.Hq;
    P.Hkv = a.Hkv;
    P.D = a.D;
    P.G = G;
    P.tokens_per_tile = BM / G;
    P.page_size = a.page_size;
    P.pages_per_seq = a.pages_per_seq;
    P.wide_rows = a.D % 16 == 0 && aligned(a.out, 32);
    P.lose = lose;
    P.lose_after = lose_after;
    P.page_rows = paged && a.page_size < KT ? a.page_size : KT;

    CUtensorMap maps[3];
    const uint64_t qd[4] = {(uint64_t)a.D, (uint64_t)G, (uint64_t)a.rows, (uint64_t)a.Hkv};
    const int64_t qs[3] = {a.q_stride[1], a.q_stride[0], a.q_stride[1] * G};
    const uint32_t qb[4] = {PANEL, (uint32_t)G, (uint32_t)P.tokens_per_tile, 1};
    const uint64_t cd[4] = {(uint64_t)a.D, (uint64_t)a.page_size, (uint64_t)a.Hkv,
                            (uint64_t)(a.num_pages > 0 ? a.num_pages : 1)};
    const uint32_t cb[4] = {PANEL, (uint32_t)P.page_rows, 1, 1};
    const int64_t kc[3] = {a.k_cache_stride[1], a.k_cache_stride[2], a.k_cache_stride[0]};
    const int64_t vc[3] = {a.v_cache_stride[1], a.v_cache_stride[2], a.v_cache_stride[0]};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return SPEC_ECUDA;
    if (!make_map(&maps[0], a.q, a.dtype, 4, qd, qs, qb) ||
        !make_map(&maps[1], a.k_cache, a.dtype, 4, cd, kc, cb) ||
        !make_map(&maps[2], a.v_cache, a.dtype, 4, cd, vc, cb))
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
    if (a.dtype == SPEC_BF16)
        return a.D > PANEL ? launch<2, SPEC_BF16>(maps, P, a.rows, sms, di, st)
                           : launch<1, SPEC_BF16>(maps, P, a.rows, sms, di, st);
    return a.D > PANEL ? launch<2, SPEC_F16>(maps, P, a.rows, sms, di, st)
                       : launch<1, SPEC_F16>(maps, P, a.rows, sms, di, st);
}

int32_t spec_chunk_attention(const spec_chunk_attention_args *args, void *workspace,
                             size_t workspace_bytes, void *stream)
{
    return attend(args, workspace, workspace_bytes, -1, 0, stream);
}

int32_t spec_selftest_chunk_timeout(const spec_chunk_attention_args *args, void *workspace,
                                    size_t workspace_bytes, int32_t cta, int32_t after,
                                    void *stream)
{
    if (cta < 0 || after < 0)
        return SPEC_EINVAL;
    return attend(args, workspace, workspace_bytes, cta, after, stream);
}

}  // extern "C"
