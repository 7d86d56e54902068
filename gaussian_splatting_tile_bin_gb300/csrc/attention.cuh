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
// ones, and results do not depend on timing.  The line has fewer than 2^31
// iterations (checked with the arguments), so its arithmetic is in 32 bits:
// 64-bit divisions cost each tile half a microsecond.
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
    __device__ static uint32_t steps(int length) { return (uint32_t)max(1, (length + kKeyTile - 1) / kKeyTile); }
    __device__ static uint32_t of_item(const Schedule &s, int length) { return s.tiles * steps(length); }
    __device__ static void at(const Schedule &s, int length, uint32_t in, Segment &g)
    {
        const uint32_t total = steps(length), tile = in / total;
        g.total = (int)total;
        g.head = 0;
        g.tile = (int)tile;
        g.begin = (int)(in - tile * total);
    }
};

// Tiles of keys; their iterations are the query tiles of every head of the group.
// A tile behind the item's length has one, which writes its zeros.
struct KeyLine {
    __device__ static uint32_t full(int length) { return (uint32_t)(length + kKeyTile - 1) / kKeyTile; }
    __device__ static uint32_t of_head(const Schedule &s, int length)
    {
        const uint32_t n = full(length);
        return n * s.inner + (s.tiles - n);
    }
    __device__ static uint32_t of_item(const Schedule &s, int length) { return s.heads * of_head(s, length); }
    __device__ static void at(const Schedule &s, int length, uint32_t in, Segment &g)
    {
        const uint32_t span = of_head(s, length), some = full(length) * s.inner, head = in / span;
        g.head = (int)head;
        in -= head * span;
        if (in < some) {
            const uint32_t tile = in / s.inner;
            g.total = (int)s.inner;
            g.tile = (int)tile;
            g.begin = (int)(in - tile * s.inner);
        } else {
            g.total = 1;
            g.tile = (int)(full(length) + (in - some));
            g.begin = 0;
        }
    }
};

// The iterations of 32 items, or what is left of the batch; a whole warp's call.
template <typename Line>
__device__ __forceinline__ uint32_t items_length(const Schedule &s, int item)
{
    const int mine = item + (int)(threadIdx.x % 32);
    return __reduce_add_sync(~0u, mine < s.batch ? Line::of_item(s, item_length(s.lengths, s.length, mine)) : 0u);
}

template <typename Line>
__device__ uint32_t line_length(const Schedule &s)
{
    if (!s.lengths) return s.batch * Line::of_item(s, s.length);
    uint32_t n = 0;
    for (int b = 0; b < s.batch; b += 32) n += items_length<Line>(s, b);
    return n;
}

// The segments of [at, stop) on the line, one per tile.  Made by whole warps.
template <typename Line>
struct Walk {
    const Schedule &s;
    uint32_t at, stop;
    uint32_t base = 0, span = 0;   // the current item's place on the line
    int item = 0, length = 0;

    __device__ Walk(const Schedule &sched, uint32_t begin, uint32_t end) : s(sched), at(begin), stop(end)
    {
        if (s.lengths) {
            while (item + 32 < s.batch) {
                const uint32_t some = items_length<Line>(s, item);
                if (at < base + some) break;
                base += some;
                item += 32;
            }
        }
        length = item_length(s.lengths, s.length, item);
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
        g.end = (int)min((uint32_t)g.total, g.begin + (stop - at));
        at += g.end - g.begin;
        return true;
    }
};

__device__ __forceinline__ uint32_t share_begin(uint32_t line, uint32_t block, uint32_t blocks)
{
    return line / blocks * block + line % blocks * block / blocks;
}

// Blocks with a share (the grid is sized for full lengths; the line may be shorter).
__device__ __forceinline__ int busy_blocks(uint32_t line, int grid) { return (int)min((uint32_t)grid, line); }

// This block's share.
template <typename Line>
__device__ Walk<Line> walk_share(const Schedule &s)
{
    const uint32_t line = line_length<Line>(s);
    const int blocks = busy_blocks(line, gridDim.x), block = min((int)blockIdx.x, blocks);
    return Walk<Line>(s, share_begin(line, block, blocks), block < blocks ? share_begin(line, block + 1, blocks) : line);
}

// The value of lane 0 of a whole warp, which lets the compiler keep what follows
// from it in registers that the warp shares.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(~0u, x, 0); }

// The next segment, for a whole warp.  (Products issue from such registers: as
// long as the warps' own numbers and segments looked different from lane to lane,
// moving each product's operands there made the forward 8% and the backward 10%
// slower.)
template <typename Line>
__device__ __forceinline__ bool next_uniform(Walk<Line> &walk, Segment &g)
{
    if (!uniform(walk.next(g))) return false;
    g.begin = uniform(g.begin);
    g.end = uniform(g.end);
    g.total = uniform(g.total);
    g.length = uniform(g.length);
    g.tile = uniform(g.tile);
    return true;
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
    const uint32_t line = line_length<Line>(s);
    const int blocks = busy_blocks(line, grid);
    if (first >= blocks) return false;
    const uint32_t cut = share_begin(line, first, blocks);
    Walk<Line> walk(s, cut, line);
    walk.next(g);
    const uint32_t start = cut - g.begin, stop = start + g.total;
    if (g.begin == 0 || share_begin(line, first - 1, blocks) > start) return false;
    last = first;
    while (last + 1 < blocks && share_begin(line, last + 1, blocks) < stop) ++last;
    return true;
}

// Keys of a tile's last step whose scores are computed, `valid` of which take part.
__device__ __forceinline__ int round_keys(int valid) { return min(kKeyTile, (valid + 15) & ~15); }

// Zeros in a key tile's rows from `valid` on: what they hold must not meet zero
// factors as infinities or NaN.  `row`: the calling thread's, of 128.
template <int BLOCKS>
__device__ __forceinline__ void clear_tail(unsigned char *tile, int row, int valid)
{
    if (row >= valid)
        for (int b = 0; b < BLOCKS; ++b)
            for (int e = 0; e < 8; ++e)   // lanes start at different banks
                *(uint4 *)(tile + b * kBlockBytes + row * 128 + ((e + row) & 7) * 16) = make_uint4(0, 0, 0, 0);
    fence_async();
}

// 32 bytes at an address aligned to them.
__device__ __forceinline__ void store32(void *p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f,
                                        uint32_t g, uint32_t h)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a), "r"(b), "r"(c), "r"(d),
                 "r"(e), "r"(f), "r"(g), "r"(h)
                 : "memory");
}

// An average of v whose weights P were rounded to 16 bits may come out above the
// largest v by 2^-11 of it, which beside f16's largest number is infinity.
template <typename T>
__device__ __forceinline__ float within_range(float x)
{
    if constexpr (std::is_same<T, __half>::value) return fabsf(x) < 65600.0f ? fminf(fmaxf(x, -65504.0f), 65504.0f) : x;
    return x;
}

// Two averages as a 16-bit pair.
template <typename T>
__device__ __forceinline__ uint32_t pack_average(float lo, float hi)
{
    return pack2<T>(within_range<T>(lo), within_range<T>(hi));
}

// Up to 32 results of a row (AVERAGE: averages of v), `left` of them there, to their
// place (whole) or to the partial results.  A thread holds a row, so its
// neighbours' stores fall into other lines: the wider each is the fewer there are.
// `wide`: out's rows and `left` are multiples of 32 bytes.
template <typename T, bool AVERAGE = false>
__device__ __forceinline__ void store_results(T *out, float *partial, bool whole, bool wide, int left, const float (&f)[32])
{
    if (!whole) {
#pragma unroll
        for (int y = 0; y < 32; y += 8)
            if (y < left)
                store32(partial + y, __float_as_uint(f[y]), __float_as_uint(f[y + 1]), __float_as_uint(f[y + 2]),
                        __float_as_uint(f[y + 3]), __float_as_uint(f[y + 4]), __float_as_uint(f[y + 5]),
                        __float_as_uint(f[y + 6]), __float_as_uint(f[y + 7]));
        return;
    }
    uint32_t w[16];
#pragma unroll
    for (int y = 0; y < 16; ++y) w[y] = pack2<T>(f[2 * y], f[2 * y + 1]);
    if constexpr (AVERAGE && std::is_same<T, __half>::value) {
        __half2 top = __habs2(*(const __half2 *)&w[0]);
#pragma unroll
        for (int y = 1; y < 16; ++y) top = __hmax2(top, __habs2(*(const __half2 *)&w[y]));
        if (__hisinf(__low2half(top)) || __hisinf(__high2half(top))) {
#pragma unroll
            for (int y = 0; y < 16; ++y) w[y] = pack_average<T>(f[2 * y], f[2 * y + 1]);
        }
    }
    if (wide) {
#pragma unroll
        for (int y = 0; y < 16; y += 8)
            if (2 * y < left) store32(out + 2 * y, w[y], w[y + 1], w[y + 2], w[y + 3], w[y + 4], w[y + 5], w[y + 6], w[y + 7]);
    } else {
#pragma unroll
        for (int y = 0; y < 16; y += 4)
            if (2 * y < left) *(uint4 *)(out + 2 * y) = make_uint4(w[y], w[y + 1], w[y + 2], w[y + 3]);
    }
}

// Whether an array's rows take 32-byte stores.
inline bool rows_of_32_bytes(const gsr_heads &t, int dim)
{
    return dim % 16 == 0 && (uintptr_t)t.data % 32 == 0 && t.batch_stride % 16 == 0 && t.token_stride % 16 == 0 &&
           t.head_stride % 16 == 0;
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
