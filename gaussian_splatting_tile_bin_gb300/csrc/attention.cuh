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
    int tiles;               // tiles per item (queries as rows) or per item and key head (keys as rows)
    int heads;               // key heads (keys as rows)
    int inner;               // iterations of a tile of keys: query heads of a group x query tiles
    const int32_t *lengths;  // device [batch] or NULL
    int length;              // of every item when lengths is NULL, and their limit
};

struct Segment {
    int item, head, tile;    // head: key head (keys as rows)
    int begin, end;          // iterations of the tile
    int total;               // iterations the tile has
    int length;              // the item's length
    __device__ bool whole() const { return begin == 0 && end == total; }
};

__device__ __forceinline__ int item_length(const int32_t *lengths, int limit, int item)
{
    return lengths ? max(0, min(lengths[item], limit)) : limit;
}

// Tiles of queries; their iterations are the item's key tiles.  An item without
// keys has one iteration per tile, which writes its zeros.
struct QueryLine {
    __device__ static int steps(int length) { return max(1, (length + kKeyTile - 1) / kKeyTile); }
    __device__ static int64_t of_item(const Schedule &s, int length) { return (int64_t)s.tiles * steps(length); }
    __device__ static void at(const Schedule &s, int length, int64_t in, Segment &g)
    {
        g.total = steps(length);
        g.head = 0;
        g.tile = (int)(in / g.total);
        g.begin = (int)(in - (int64_t)g.tile * g.total);
    }
};

// Tiles of keys; their iterations are the query tiles of every head of the group.
// A tile behind the item's length has one, which writes its zeros.
struct KeyLine {
    __device__ static int full(int length) { return (length + kKeyTile - 1) / kKeyTile; }
    __device__ static int64_t of_head(const Schedule &s, int length)
    {
        const int n = full(length);
        return (int64_t)n * s.inner + (s.tiles - n);
    }
    __device__ static int64_t of_item(const Schedule &s, int length) { return s.heads * of_head(s, length); }
    __device__ static void at(const Schedule &s, int length, int64_t in, Segment &g)
    {
        const int64_t span = of_head(s, length), some = (int64_t)full(length) * s.inner;
        g.head = (int)(in / span);
        in -= g.head * span;
        if (in < some) {
            g.total = s.inner;
            g.tile = (int)(in / s.inner);
            g.begin = (int)(in - (int64_t)g.tile * s.inner);
        } else {
            g.total = 1;
            g.tile = full(length) + (int)(in - some);
            g.begin = 0;
        }
    }
};

template <typename Line>
__device__ int64_t line_length(const Schedule &s)
{
    if (!s.lengths) return s.batch * Line::of_item(s, s.length);
    int64_t n = 0;
    for (int b = 0; b < s.batch; ++b) n += Line::of_item(s, item_length(s.lengths, s.length, b));
    return n;
}

// The segments of [at, stop) on the line, one per tile.
template <typename Line>
struct Walk {
    const Schedule &s;
    int64_t at, stop;
    int64_t base = 0, span = 0;   // the current item's place on the line
    int item = 0, length = 0;

    __device__ Walk(const Schedule &sched, int64_t begin, int64_t end) : s(sched), at(begin), stop(end)
    {
        length = item_length(s.lengths, s.length, 0);
        span = Line::of_item(s, length);
        if (!s.lengths) {
            item = (int)(at / span);
            base = item * span;
        }
    }
    __device__ bool next(Segment &g)
    {
        if (at >= stop) return false;
        while (at >= base + span) {
            base += span;
            ++item;
            if (s.lengths) {
                length = item_length(s.lengths, s.length, item);
                span = Line::of_item(s, length);
            }
        }
        Line::at(s, length, at - base, g);
        g.item = item;
        g.length = length;
        g.end = (int)min((int64_t)g.total, g.begin + (stop - at));
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

// This block's share.
template <typename Line>
__device__ Walk<Line> walk_share(const Schedule &s)
{
    const int64_t line = line_length<Line>(s);
    const int blocks = busy_blocks(line, gridDim.x), block = min((int)blockIdx.x, blocks);
    return Walk<Line>(s, share_begin(line, block, blocks), block < blocks ? share_begin(line, block + 1, blocks) : line);
}

// Partial results of a block: slot 2 c for a tile cut at its start by the block's
// share, 2 c + 1 for one cut at its end alone.
__device__ __forceinline__ int partial_slot(const Segment &g, int block) { return 2 * block + (g.begin > 0 ? 0 : 1); }

// The tile that the start of share `first` cuts, if that is the first share that
// starts inside the tile: its parts are slot 2 first - 1 and slots 2 b of the
// blocks b = first .. last.
template <typename Line>
__device__ bool cut_tile(const Schedule &s, int grid, int first, Segment &g, int &last)
{
    const int64_t line = line_length<Line>(s);
    const int blocks = busy_blocks(line, grid);
    if (first >= blocks) return false;
    const int64_t cut = share_begin(line, first, blocks);
    Walk<Line> walk(s, cut, line);
    walk.next(g);
    const int64_t start = cut - g.begin, stop = start + g.total;
    if (g.begin == 0 || share_begin(line, first - 1, blocks) > start) return false;
    last = first;
    while (last + 1 < blocks && share_begin(line, last + 1, blocks) < stop) ++last;
    return true;
}

// Masked keys packed to the front: rows [item][key head][token][dim] of k and v,
// their original indices and the items' counts.
struct Packed {
    gsr_heads k, v;
    int32_t *counts;         // [batch]
    int32_t *index;          // [batch, kv_len]
};

// Query rows that the kernel for few rows takes (attention_few.cu): the tokens of
// all query heads of a key head.
constexpr int kFewRows = 16;
int few_rows_forward(gsr_ctx *ctx, const gsr_attention &d, const gsr_heads &q, const gsr_heads &k, const gsr_heads &v,
                     const gsr_heads &out, float *lse, cudaStream_t stream);

size_t packed_bytes(const gsr_attention &d);
cudaError_t pack_keys(gsr_ctx *ctx, const gsr_attention &d, const gsr_heads &k, const gsr_heads &v, void *work,
                      Packed *out, cudaStream_t stream);

}  // namespace gsr
