// spec_attn.cu -- tree attention over a key/value cache (include/spec_attn.h).
//
// One CTA of 128 threads per (tree node, query head).  Keys go by in tiles of
// 128, one per thread: the thread's score, the tile's maximum and the running
// (maximum, sum, weighted sum) of the softmax; then thread d adds the tile's
// weighted values of element d.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "spec_attn.h"
#include "spec_verify.h"
#include "attn_plan.cuh"
#include "device_common.cuh"

namespace {

using namespace spec_dev;
using namespace spec_attn;

struct AParams {
    spec_tree_attention_args a;
    PlanLayout lay;
    int G;
};

template <int DT>
__device__ __forceinline__ float elem(const void *p, int64_t i)
{
    if (DT == SPEC_BF16)
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
    return __half2float(reinterpret_cast<const __half *>(p)[i]);
}

template <int DT>
__device__ __forceinline__ void store(void *p, int64_t i, float x)
{
    if (DT == SPEC_BF16)
        reinterpret_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
    else
        reinterpret_cast<__half *>(p)[i] = __float2half_rn(x);
}

template <int DT>
__global__ void __launch_bounds__(KT) attention_kernel(const AParams P)
{
    const spec_tree_attention_args &A = P.a;
    __shared__ float qs[SPEC_ATTN_MAX_HEAD_DIM];
    __shared__ float w[KT];
    __shared__ float red[4];
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = (int)(blockIdx.x / A.N), n = (int)(blockIdx.x % A.N);
    const int h = (int)blockIdx.y, kvh = h / P.G;
    wait_previous_kernel();
    const uint8_t *plan = static_cast<const uint8_t *>(A.plan);
    const PlanSeq S = reinterpret_cast<const PlanSeq *>(plan + P.lay.seq)[b];
    const uint32_t *mask = reinterpret_cast<const uint32_t *>(plan + P.lay.mask) +
                           ((size_t)b * A.N + n) * P.lay.W;
    const int64_t orow = ((int64_t)b * A.N + n) * A.Hq + h;
    if (n >= S.n_nodes) {
        if (tid < A.D)
            store<DT>(A.out, orow * A.D + tid, S.status ? NAN : 0.0f);
        if (tid == 0 && A.out_lse)
            A.out_lse[orow] = S.status ? NAN : -INFINITY;
        return;
    }
    if (tid < A.D)
        qs[tid] = elem<DT>(A.q, b * A.q_stride[0] + n * A.q_stride[1] + h * A.q_stride[2] + tid);
    __syncthreads();
    auto row_of = [&](int j, const int64_t *cs, const int64_t *ns, bool &cached) -> int64_t {
        cached = j < S.cache_len;
        if (cached) {
            const int pg = A.page_table
                ? A.page_table[(size_t)b * A.pages_per_seq + j / A.page_size] : b;
            return pg * cs[0] + (j % A.page_size) * cs[1] + kvh * cs[2];
        }
        return b * ns[0] + (j - S.cache_len) * ns[1] + kvh * ns[2];
    };
    float m = -INFINITY, l = 0.0f, o = 0.0f;
    const int total = S.cache_len + S.n_nodes;
    const float c = A.scale * LOG2E;
    for (int j0 = 0; j0 < total; j0 += KT) {
        const int j = j0 + tid, t = j - S.cache_len;
        const bool on = j < total && (t < 0 || ((mask[t >> 5] >> (t & 31)) & 1u));
        float s = -INFINITY;
        if (on) {
            bool cached;
            const int64_t r = row_of(j, A.k_cache_stride, A.k_new_stride, cached);
            const void *base = cached ? A.k_cache : A.k_new;
            s = 0.0f;
            for (int d = 0; d < A.D; ++d)
                s = fmaf(qs[d], elem<DT>(base, r + d), s);
            s *= c;
        }
        float mx = s;
        for (int d = 16; d; d >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        if (lane == 0)
            red[warp] = mx;
        __syncthreads();
        const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        const float ms = mn == -INFINITY ? 0.0f : mn;
        w[tid] = on ? ex2(s - ms) : -1.0f;  // -1: not seen
        const float f = m == -INFINITY ? 0.0f : ex2(m - ms);
        l *= f;
        if (f != 1.0f)
            o = m == -INFINITY ? 0.0f : o * f;
        m = mn;
        __syncthreads();
        const int cnt = min(KT, total - j0);
        for (int i = 0; i < cnt; ++i) {
            const float p = w[i];
            if (p == -1.0f)
                continue;
            l += p;
            if (tid < A.D) {
                bool cached;
                const int64_t r = row_of(j0 + i, A.v_cache_stride, A.v_new_stride, cached);
                o = fmaf(p, elem<DT>(cached ? A.v_cache : A.v_new, r + tid), o);
            }
        }
        __syncthreads();
    }
    if (tid < A.D)
        store<DT>(A.out, orow * A.D + tid, l == 0.0f ? 0.0f : o / l);
    if (tid == 0 && A.out_lse)
        A.out_lse[orow] = l == 0.0f ? -INFINITY : (m + log2f(l)) / LOG2E;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool heads_ok(int32_t N, int32_t Hq, int32_t Hkv, int32_t D)
{
    return N >= 1 && N <= SPEC_ATTN_MAX_NODES && Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 &&
           Hq / Hkv <= 128 && Hq <= 65535 && D >= 8 && D % 8 == 0 && D <= SPEC_ATTN_MAX_HEAD_DIM;
}

bool page_size_ok(int32_t s, bool paged)
{
    return s >= 1 && (!paged || s % 128 == 0 || (s >= 8 && (s & (s - 1)) == 0));
}

bool strides_ok(const int64_t (&s)[3])
{
    for (int64_t x : s)
        if (x < 0 || x % 8 != 0 || x > ((int64_t)1 << 38))
            return false;
    return true;
}

}  // namespace

extern "C" {

size_t spec_tree_attention_workspace_size(int32_t N, int32_t Hq, int32_t Hkv, int32_t D)
{
    return heads_ok(N, Hq, Hkv, D) ? 256 : 0;
}

int32_t spec_tree_attention(const spec_tree_attention_args *args, void *workspace,
                            size_t workspace_bytes, void *stream)
{
    if (!args)
        return SPEC_EINVAL;
    const spec_tree_attention_args &a = *args;
    if (!heads_ok(a.N, a.Hq, a.Hkv, a.D) || a.B < 0 || a.B > 65535 ||
        !page_size_ok(a.page_size, a.page_table != nullptr) || a.pages_per_seq < 1 ||
        a.num_pages < 0 ||
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
        (!a.page_table && (a.pages_per_seq != 1 || a.num_pages < a.B)))
        return SPEC_EINVAL;
    if (workspace_bytes < spec_tree_attention_workspace_size(a.N, a.Hq, a.Hkv, a.D))
        return SPEC_ENOSPACE;
    AParams P;
    P.a = a;
    P.lay = plan_layout(a.B, a.N);
    P.G = a.Hq / a.Hkv;
    const dim3 grid((unsigned int)a.B * (unsigned int)a.N, (unsigned int)a.Hq);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (a.dtype == SPEC_BF16)
        attention_kernel<SPEC_BF16><<<grid, KT, 0, st>>>(P);
    else
        attention_kernel<SPEC_F16><<<grid, KT, 0, st>>>(P);
    if (cudaPeekAtLastError() != cudaSuccess) {
        (void)cudaGetLastError();
        return SPEC_ECUDA;
    }
    return SPEC_OK;
}

}  // extern "C"
