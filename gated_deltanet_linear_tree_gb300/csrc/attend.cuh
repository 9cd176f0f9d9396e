// Attention of new rows over a paged cache: what its kernels share.
//
// Row i of a sequence (new token i, at position ctx + depth_i, depth_i = i
// without a tree) sees the cache's ctx tokens and its own root path.  The rows
// of a sequence are worked on in tiles of rt tokens, each with the g query heads
// of one key head (rows of a tile: token-major, head fastest), against tiles of
// kt keys, the units of the work.  A plan lists the row tiles of all sequences and the
// running sum of their units over all key heads; CTA c of G takes units
// [c U / G, (c + 1) U / G) of that line, so that every CTA has the same work
// whatever the sequences' lengths.  A (row tile, key head) whose units fall to
// several CTAs is merged by the one that finishes last, in the pieces' order.
#pragma once

#include "common.cuh"

namespace canopy {
namespace att {

constexpr int kMaskWords = kMaxT / 32;
constexpr int kNoWindow = 0x7FFFFFFF;

struct Tile {
    int b, row;              // sequence; first row of q and o
    int t0, ntok;            // its index in the sequence; rows (tokens) of the tile
    int ctx, n;              // tokens in the cache before the sequence's new ones; new ones
    int sink_end, near, hi;  // keys [0, sink_end) and [near, hi) are seen by some row
    int sink_tiles, first;   // key tiles [0, sink_tiles) and from `first` on
    int units;               // how many key tiles
};

struct Args {
    const void *q, *kc, *vc;
    void* o;
    const int32_t *table, *context, *starts, *parent, *lengths;
    int N, B, T, HQ, HKV, g;
    int pages, log_page, max_pages;
    int window, sinks;
    float scale2;  // scale * log2(e): weights are powers of two
    int rt, log_kt, ctas, max_tiles;
    int slot_rows;  // rows of a slot
    // workspace
    int32_t* err;
    int4* seqs;       // [B]: first row, rows, ctx, first tile
    Tile* tiles;      // [max_tiles]
    int64_t* line;    // [max_tiles + 1]
    int* first_tile;  // [ctas]: the tile that CTA c begins in
    int* total;       // number of tiles
    uint32_t* mask;   // trees: [N][kMaskWords], the nodes of a row's path that it sees
    int32_t* depth;   // trees: [N]
    int32_t* done;    // [2 ctas]: pieces finished of the item that begins in CTA c (by halves of its rows)
    float* part;      // [2 ctas] slots
};

// ---------------------------------------------------------------------------
// Which keys a row sees.  t: the row's index in its sequence, depth its depth (t
// without a tree), mask its path (null without a tree).
__device__ inline bool sees(const Args& a, const Tile& tile, int depth, const uint32_t* mask, int key) {
    const int p = key - tile.ctx;
    if (mask && p >= 0) return p < tile.n && ((mask[p >> 5] >> (p & 31)) & 1u);
    const int pos = tile.ctx + depth;
    return key <= pos && (pos - key < a.window || key < a.sinks);
}
// Whether every row of the tile sees keys [key, key + kt).
__device__ inline bool all_see(const Args& a, const Tile& tile, int key, int kt) {
    const int last = key + kt - 1;
    if (last >= tile.ctx + (a.parent ? 0 : tile.t0 + 1)) return false;
    return last < a.sinks || tile.ctx + (a.parent ? tile.n : tile.t0 + tile.ntok) - 1 - key < a.window;
}
// Whether some row of the tile may see the key (the others' pages may be gone).
__device__ inline bool in_reach(const Tile& tile, int key) {
    return key < tile.sink_end || (key >= tile.near && key < tile.hi);
}
__device__ inline int key_tile(const Tile& tile, int u) {
    return u < tile.sink_tiles ? u : tile.first + u - tile.sink_tiles;
}

// ---------------------------------------------------------------------------
// The line of units and its division.

__device__ inline int64_t cta_begin(int64_t units, int ctas, int c) { return units * c / ctas; }
// The CTA whose part holds unit u: the largest c with floor(c U / G) <= u.
__device__ inline int cta_of(int64_t units, int ctas, int64_t u) {
    return int(((u + 1) * ctas + units - 1) / units) - 1;
}

// Inclusive scan over the block's threads, and the total.
template <int NT, typename V, typename Op>
__device__ inline V block_scan(V x, Op op, V* warps, V& total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int s = 1; s < 32; s *= 2) {
        const V y = __shfl_up_sync(0xffffffffu, x, s);
        if (lane >= s) x = op(y, x);
    }
    if (lane == 31) warps[w] = x;
    __syncthreads();
    total = warps[0];
#pragma unroll
    for (int i = 1; i < NT / 32; ++i) {
        if (i == w) x = op(total, x);
        total = op(total, warps[i]);
    }
    __syncthreads();
    return x;
}

__device__ inline Tile make_tile(const Args& a, int b, const int4& s, int t) {
    Tile r;
    r.b = b;
    r.t0 = t * a.rt;
    r.row = s.x + r.t0;
    r.ntok = min(a.rt, s.y - r.t0);
    r.n = s.y;
    r.ctx = s.z;
    r.hi = r.ctx + (a.parent ? r.n : r.t0 + r.ntok);
    const int64_t near = int64_t(r.ctx) + (a.parent ? 0 : r.t0) - a.window + 1;
    r.near = near > 0 ? int(near) : 0;
    r.sink_end = min(a.sinks, r.near);
    const int kt = 1 << a.log_kt;
    r.first = r.near >> a.log_kt;
    r.sink_tiles = min((r.sink_end + kt - 1) >> a.log_kt, r.first);
    r.units = r.sink_tiles + ((r.hi + kt - 1) >> a.log_kt) - r.first;
    return r;
}

// The plan, by a whole block of NT threads: a.seqs, a.tiles, a.line, and the
// number of tiles (returned).  Starts out of order or range are read as their
// running maximum, lengths and contexts as the nearest that fit; these set bits
// in *bad.
template <int NT>
__device__ inline int make_plan(const Args& a, int* bad) {
    __shared__ int wi[NT / 32];
    __shared__ int64_t wl[NT / 32];
    const auto most = [](int x, int y) { return max(x, y); };
    const auto sum = [](int64_t x, int64_t y) { return x + y; };
    const auto isum = [](int x, int y) { return x + y; };
    const int tid = threadIdx.x;
    int carry_lo = 0, carry_hi = 0, carry = 0, total;
    if (a.starts) carry_lo = carry_hi = start_in_range(a.starts, 0, a.N);
    for (int b0 = 0; b0 < a.B; b0 += NT) {
        const int b = b0 + tid;
        int lo = b * a.T, n = a.T;
        if (a.starts) {
            const int s = b < a.B ? start_in_range(a.starts, b, a.N) : 0;
            const int e = b < a.B ? start_in_range(a.starts, b + 1, a.N) : 0;
            lo = max(carry_lo, block_scan<NT>(s, most, wi, total));
            carry_lo = max(carry_lo, total);
            const int hi = max(carry_hi, block_scan<NT>(e, most, wi, total));
            carry_hi = max(carry_hi, total);
            n = hi - lo;
            if (b < a.B && (a.starts[b] != lo || a.starts[b + 1] != hi)) *bad |= CANOPY_DEVERR_LENGTH;
        }
        int ctx = 0;
        if (b < a.B) {
            n = min(n, stream_len(a.lengths, b, a.T, bad));
            ctx = a.context[b];
            if (ctx < 0) {
                ctx = 0;
                *bad |= CANOPY_DEVERR_LENGTH;
            }
            const int room = a.max_pages << a.log_page;
            if (n > room || ctx > room - n) {
                *bad |= CANOPY_DEVERR_PAGE;
                n = min(n, room);
                ctx = min(ctx, room - n);
            }
        } else {
            n = 0;
        }
        const int nt = (n + a.rt - 1) / a.rt;
        const int upto = carry + block_scan<NT>(nt, isum, wi, total);
        if (b < a.B) a.seqs[b] = make_int4(lo, n, ctx, upto - nt);
        carry += total;
    }
    __syncthreads();
    const int ntiles = carry;
    int64_t line = 0, ltotal;
    for (int i0 = 0; i0 < ntiles; i0 += NT) {
        const int i = i0 + tid;
        int64_t units = 0;
        if (i < ntiles) {
            int b = 0, e = a.B;  // the last sequence whose first tile is not behind i
            while (e - b > 1) {
                const int m = (b + e) >> 1;
                if (a.seqs[m].w <= i) b = m; else e = m;
            }
            const int4 s = a.seqs[b];
            const Tile t = make_tile(a, b, s, i - s.w);
            a.tiles[i] = t;
            units = int64_t(t.units) * a.HKV;
        }
        const int64_t upto = line + block_scan<NT>(units, sum, wl, ltotal);
        if (i < ntiles) a.line[i] = upto - units;
        line += ltotal;
    }
    if (tid == 0) a.line[ntiles] = line;
    __syncthreads();
    return ntiles;
}

// How many CTAs share the work: no part is shorter than `least` units.
__device__ inline int parts(const Args& a, int64_t units, int least) {
    const int64_t most = units / least;
    return int(most < 1 ? 1 : most < a.ctas ? most : a.ctas);
}

// The last tile that begins at or before unit u.
__device__ inline int tile_at(const int64_t* line, int ntiles, int64_t u) {
    int lo = 0, hi = ntiles;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (line[m] <= u) lo = m; else hi = m;
    }
    return lo;
}

// One CTA's part of a (row tile, key head): units [u0, u1) of `tile`.
struct Piece {
    Tile tile;
    int h, u0, u1;
    int slot;           // where an unfinished piece goes
    int first, pieces;  // the CTA that the item begins in; CTAs that have a piece of it
};

// Walks a CTA's pieces.
struct Walk {
    int64_t units, at, end;
    int ctas, tile;
    __device__ bool next(const Args& a, Piece& p) {
        if (at >= end) return false;
        while (a.line[tile + 1] <= at) ++tile;
        p.tile = a.tiles[tile];
        const int64_t rel = at - a.line[tile];
        p.h = int(rel / p.tile.units);
        p.u0 = int(rel - int64_t(p.h) * p.tile.units);
        p.u1 = int(min(int64_t(p.tile.units), p.u0 + (end - at)));
        const int64_t begin = at - p.u0;
        p.first = p.u0 == 0 ? int(blockIdx.x) : cta_of(units, ctas, begin);
        p.pieces = p.u1 == p.tile.units && p.u0 == 0 ? 1 : cta_of(units, ctas, begin + p.tile.units - 1) - p.first + 1;
        p.slot = 2 * int(blockIdx.x) + (p.u0 == 0);
        at += p.u1 - p.u0;
        return true;
    }
};
// Slot of piece i of an item that begins in CTA `first`.
__device__ inline int slot_of(int first, int i) { return 2 * (first + i) + (i == 0); }

}  // namespace att
}  // namespace canopy
