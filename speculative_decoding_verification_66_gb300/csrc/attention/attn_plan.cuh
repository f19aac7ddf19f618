// attn_plan.cuh -- how the tile kernel's work is laid out and shared among its
// thread blocks.
//
// The query rows of one sequence that read one key/value head, T tokens times G
// heads, are taken in blocks of R rows (row r is token r / G, head r % G of the
// group). An item is such a block with the range of 128-key tiles that its rows
// see. All items' tiles, in the order sequence, head, row block, tile, form one
// line of U units, and block c of n takes the units [c U / n, (c + 1) U / n):
// every block gets the same number of tiles whatever the lengths are, a block
// meets at most two items that it shares with others, and nothing has to be
// known on the host. Blocks find their start by summing the sequences' units,
// B at a time over the block's threads.
#pragma once

#include "attn_common.cuh"

namespace sva {

constexpr int kTile = 128;  // keys to a tile
constexpr int kTileShift = 7;

// What a block left for the joining kernel.
struct Share {
    int32_t leads;  // this block began an item that it did not finish
    int32_t b, h, row0, rows;
    int32_t q0;     // first packed row of the sequence
    int32_t last;   // the block that finished it
    int64_t units;  // U
};

struct Range {
    int32_t lo, hi;  // tiles [lo, hi)
};

// The tiles seen by rows [r0, r1) of a sequence.
__device__ __forceinline__ Range row_tiles(const Attn& a, int64_t cached, int r0, int r1)
{
    const int64_t first = first_key(a, cached + r0 / a.G);
    const int64_t last = cached + (r1 - 1) / a.G;
    return Range{static_cast<int32_t>(first >> kTileShift),
                 static_cast<int32_t>(last >> kTileShift) + 1};
}

// Units of one head of a sequence.
template <int R>
__device__ __forceinline__ int64_t head_units(const Attn& a, const Seq& q)
{
    if (q.bad) return 0;
    const int rows = q.count * a.G;
    int64_t n = 0;
    for (int r = 0; r < rows; r += R) {
        const Range t = row_tiles(a, q.cached, r, min(r + R, rows));
        n += t.hi - t.lo;
    }
    return n;
}

// a / b, b > 0, a >= 0: a 64-bit division is a long routine, and most of these
// numbers are small.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    if (static_cast<uint64_t>(a | b) >> 32 == 0)
        return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}
__device__ __forceinline__ int64_t share_begin(int64_t U, int c, int n) { return quotient(U * c, n); }

// Where a block starts.
struct Start {
    int64_t u0, u1, U;
    int64_t off;  // units into sequence b
    int32_t b;
};

// A block's part of one item.
struct Segment {
    int32_t b, h, q0, row0, rows;
    int64_t cached;
    Range item;  // the item's tiles
    Range t;     // this block's
};

// Walks a block's segments. Every warp of the block walks for itself.
template <int R>
struct Walk {
    const Attn& a;
    int64_t left;
    Seq q;
    int64_t skip;
    int32_t b, h, row0;

    __device__ Walk(const Attn& args, const Start& s) : a(args), left(s.u1 - s.u0)
    {
        b = s.b;
        h = row0 = 0;
        skip = s.off;
        if (left <= 0) return;
        q = seq_of(a.c, b, a.tokens, a.max_chunk);
        const int64_t n = head_units<R>(a, q);
        h = static_cast<int32_t>(quotient(skip, n));
        skip -= h * n;
    }

    __device__ bool next(Segment* s)
    {
        while (left > 0) {
            const int rows = q.bad ? 0 : q.count * a.G;
            if (row0 >= rows) {
                row0 = 0;
                if (rows == 0 || ++h == a.c.Hkv) {
                    h = 0;
                    ++b;
                    if (b >= a.c.B) return false;  // (not reached: the units end first)
                    q = seq_of(a.c, b, a.tokens, a.max_chunk);
                }
                continue;
            }
            const int r1 = min(row0 + R, rows);
            const Range t = row_tiles(a, q.cached, row0, r1);
            const int n = t.hi - t.lo;
            if (skip >= n) {
                skip -= n;
                row0 += R;
                continue;
            }
            s->b = b;
            s->h = h;
            s->q0 = q.start;
            s->row0 = row0;
            s->rows = r1 - row0;
            s->cached = q.cached;
            s->item = t;
            s->t.lo = t.lo + static_cast<int32_t>(skip);
            s->t.hi = static_cast<int32_t>(left < t.hi - s->t.lo ? s->t.lo + left : t.hi);
            skip = 0;
            left -= s->t.hi - s->t.lo;
            row0 += R;
            return true;
        }
        return false;
    }
};

}  // namespace sva
