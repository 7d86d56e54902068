// attention.cuh -- what the cross attention kernels share: the division of the
// work over the SMs, and the masked keys' compaction.
//
// Work.  A tile is a block of rows that one accumulator holds, an iteration one
// step of its contraction (128 keys, or 128 queries of one head for the key
// gradients).  All iterations of all tiles form one line, tiles of one item and
// key head next to each other, and block c of n takes the c-th n-th of it.  A
// tile that lies in one block's share is finished there; a tile cut by shares'
// ends leaves partial results, two per block at most, which a second kernel
// joins in the order of the line.  So every SM gets the same work for any
// lengths and any number of tiles, one long row of keys or thousands of short
// ones, and results do not depend on timing.
#pragma once

#include "tensor.cuh"

namespace gsr {

constexpr int kKeyTile = 128;

struct Schedule {
    int batch;
    int tiles;               // tiles per item
    int inner;               // iterations per step of the item's length (query heads x query tiles), or 1
    const int32_t *lengths;  // device [batch] or NULL
    int length;              // of every item when lengths is NULL, and their limit
};

struct Segment {
    int item, tile;          // tile within the item
    int begin, end;          // iterations of the tile
    int total;               // iterations the tile has
    int length;              // the item's length
    __device__ bool whole() const { return begin == 0 && end == total; }
};

__device__ __forceinline__ int item_length(const int32_t *lengths, int limit, int item)
{
    return lengths ? max(0, min(lengths[item], limit)) : limit;
}

// Walks tiles whose iterations are the item's key tiles (queries as rows).
// An item without keys has one iteration per tile, which writes its zeros.
struct QueryWalk {
    const Schedule &s;
    int64_t at, stop;        // position on the line, end of the share
    int64_t base = 0;        // line position of the current item
    int item = 0, length = 0, steps = 0;

    __device__ static int steps_of(int length) { return max(1, (length + kKeyTile - 1) / kKeyTile); }
    __device__ static int64_t line(const Schedule &s)
    {
        if (!s.lengths) return (int64_t)s.batch * s.tiles * steps_of(s.length);
        int64_t n = 0;
        for (int b = 0; b < s.batch; ++b) n += (int64_t)s.tiles * steps_of(item_length(s.lengths, s.length, b));
        return n;
    }
    __device__ QueryWalk(const Schedule &sched, int64_t begin, int64_t end) : s(sched), at(begin), stop(end)
    {
        if (!s.lengths) {
            length = s.length;
            steps = steps_of(length);
            item = (int)(at / ((int64_t)s.tiles * steps));
            base = (int64_t)item * s.tiles * steps;
        } else {
            length = item_length(s.lengths, s.length, 0);
            steps = steps_of(length);
        }
    }
    __device__ bool next(Segment &g)
    {
        if (at >= stop) return false;
        while (at >= base + (int64_t)s.tiles * steps) {
            base += (int64_t)s.tiles * steps;
            ++item;
            if (s.lengths) {
                length = item_length(s.lengths, s.length, item);
                steps = steps_of(length);
            }
        }
        const int64_t in = at - base;
        g.item = item;
        g.tile = (int)(in / steps);
        g.begin = (int)(in - (int64_t)g.tile * steps);
        g.end = (int)min((int64_t)steps, g.begin + (stop - at));
        g.total = steps;
        g.length = length;
        at += g.end - g.begin;
        return true;
    }
};

__device__ __forceinline__ int64_t share_begin(int64_t line, int block, int blocks)
{
    return line / blocks * block + line % blocks * block / blocks;
}

// Blocks with a share (the grid is sized for full lengths; the line may be shorter).
__device__ __forceinline__ int busy_blocks(int64_t line, int grid) { return (int)min((int64_t)grid, line); }

// Partial results of a block: slot 2 c for a tile cut at its start by the block's
// share, 2 c + 1 for one cut at its end alone.
__device__ __forceinline__ int partial_slot(const Segment &g, int block) { return 2 * block + (g.begin > 0 ? 0 : 1); }

// Masked keys packed to the front: rows [item][key head][token][dim] of k and v,
// their original indices and the items' counts.
struct Packed {
    gsr_heads k, v;
    int32_t *counts;         // [batch]
    int32_t *index;          // [batch, kv_len]
};

size_t packed_bytes(const gsr_attention &d);
cudaError_t pack_keys(gsr_ctx *ctx, const gsr_attention &d, const gsr_heads &k, const gsr_heads &v, void *work,
                      Packed *out, cudaStream_t stream);

}  // namespace gsr
