// attn_plan.cuh -- the layout of the plan that spec_tree_plan makes and the
// attention kernels read (include/spec_attn.h).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace spec_attn {

constexpr int KT = 128;  // keys per tile of the attention, the plan's unit of work

// What the attention reads of one sequence: lengths that the plan has checked
// (both 0 where status is not 0).
struct PlanSeq {
    int cache_len;
    int n_nodes;
    int status;
    int pad;
};

// header (the device status word of the attention calls that read the plan) |
// sequences [B] | tile prefix sums [B + 1] | positions [B][N] |
// status [B] | mask [B][N][W]
struct PlanLayout {
    size_t seq, cum, positions, status, mask, total;
    int W;  // mask words per node: a multiple of 4, so rows are 16-byte aligned
};

__host__ __device__ inline size_t plan_align(size_t x) { return (x + 255) / 256 * 256; }

__host__ __device__ inline PlanLayout plan_layout(int B, int N)
{
    PlanLayout p;
    p.W = (N + KT - 1) / KT * 4;
    p.seq = 256;
    p.cum = plan_align(p.seq + (size_t)B * sizeof(PlanSeq));
    p.positions = plan_align(p.cum + ((size_t)B + 1) * sizeof(long long));
    p.status = plan_align(p.positions + (size_t)B * N * 4);
    p.mask = plan_align(p.status + (size_t)B * 4);
    p.total = plan_align(p.mask + (size_t)B * N * p.W * 4);
    return p;
}

// Key tiles of one sequence: its cache's, then its new tokens'.  At least one,
// so that every sequence has a tile that writes its rows.
__host__ __device__ inline int plan_tiles(int cache_len, int n_nodes)
{
    if (n_nodes <= 0)
        return 1;
    return (cache_len + KT - 1) / KT + (n_nodes + KT - 1) / KT;
}

}  // namespace spec_attn
