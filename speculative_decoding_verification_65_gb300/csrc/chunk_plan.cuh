// chunk_plan.cuh -- the layout of the plan that spec_chunk_plan makes and the
// chunk attention's kernels read (include/spec_chunk.h).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "attn_plan.cuh"

namespace spec_attn {

// A row group: the tokens of one sequence that a CTA has at a time, two row
// tiles of 128 rows (tokens times the heads that share a key head).
struct alignas(16) ChunkGroup {
    int b;
    int row0;   // its first token's row
    int ntok;
    int tiles;  // key tiles that any of its tokens sees (1 in an error)
    int pos0;   // its first token's position
    int bad;    // lengths or rows in error (pages: the sequence's status)
    int pad[2];
};

struct alignas(16) ChunkHeader {
    int status;       // device status word of the attention calls that read the plan
    int groups;
    long long tiles;  // key tiles of all groups
    int pad[60];
};
static_assert(sizeof(ChunkHeader) == 256, "header is 256 bytes");

// header | status [B] | groups [most] | key tiles before a group [most + 1]
struct ChunkLayout {
    size_t status, group, cum, total;
    int tokens;  // of a row group
    int most;    // row groups
};

__host__ __device__ inline int chunk_tokens(int group) { return 2 * (128 / group); }

__host__ __device__ inline ChunkLayout chunk_layout(int B, int rows, int group)
{
    ChunkLayout p;
    p.tokens = chunk_tokens(group);
    p.most = rows / p.tokens + B;  // each sequence has one that is not full, at most
    p.status = 256;
    p.group = plan_align(p.status + (size_t)B * 4);
    p.cum = plan_align(p.group + (size_t)p.most * sizeof(ChunkGroup));
    p.total = plan_align(p.cum + ((size_t)p.most + 1) * sizeof(long long));
    return p;
}

// Where an item's tiles are those of more than one share, whole tiles are taken in an order by the
// time: tile t of the item when the CTA has taken t more than a multiple of a share's tiles.  CTAs
// that read the same keys for other rows then read them at one time, once from DRAM: from the first
// tile on, each at a place of its own, 512 tokens behind 131072 positions read 11 times the cache, as
// fast as DRAM gives it.  The first of them for a piece that begins at tile `tile` of `tiles` when
// the CTA has taken `taken` units; `per` units are a share, none where no sequence has rows.
__host__ __device__ inline int piece_turn(long long taken, int tile, int tiles, long long per)
{
    if (per <= 0 || tiles < per)
        return 0;
    const long long turn = (taken - tile) % per;
    return (int)(turn < 0 ? turn + per : turn);
}

}  // namespace spec_attn
