// attn_common.cuh -- what the attention kernels share: wrappers of the tcgen05, TMA and
// mbarrier instructions, the descriptors of their operands, the steps of a row's softmax, and
// the tensor maps on the host.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "spec_attn.h"
#include "spec_verify.h"
#include "attn_plan.cuh"
#include "device_common.cuh"

namespace spec_attn {

using namespace spec_dev;

constexpr int BM = 128;           // rows of a tile (TMEM lanes)
constexpr int PANEL = 64;         // elements of a 128-byte swizzled row
constexpr int PANEL_BYTES = 128 * 128;  // 128 rows (or keys) of one panel
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

// ln of a total of weights in units of 2^m; -inf for none
__device__ __forceinline__ float lse_of(float m, float l)
{
    return l == 0.0f ? -INFINITY : (m + log2f(l)) * (1.0f / LOG2E);
}

// ------------------------------------------------------------------- host

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool page_size_ok(int32_t s, bool paged)
{
    return s >= 1 && (!paged || s % KT == 0 || (s >= 8 && (s & (s - 1)) == 0));
}

inline bool strides_ok(const int64_t (&s)[3])
{
    for (int64_t x : s)
        if (x < 0 || x % 8 != 0 || x >= ((int64_t)1 << 38))
            return false;
    return true;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn()
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
inline bool make_map(CUtensorMap *map, const void *base, int dtype, int rank, const uint64_t *dims,
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

}  // namespace spec_attn
