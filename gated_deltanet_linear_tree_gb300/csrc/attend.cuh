// Attention of new rows over a paged cache: what its kernels share.
//
// Row i of a sequence (new token i, at position ctx + depth_i, depth_i = i
// without a tree) sees the cache's ctx tokens and its own root path.  The rows
// of a sequence are worked on in tiles of rt tokens, each with the g query heads
// of one key head (rows of a tile: token-major, head fastest), against tiles of
// kt keys, the units of the work.  A plan lists the row tiles of all sequences and the
// running sum of their units over all key heads; CTA c of G takes units
// [c U / G, (c + 1) U / G) of that line, so that every CTA has the same work
// whatever the sequences' lengths.  The pieces of a (row tile, key head) whose
// units fall to several CTAs go to the workspace, and a second launch joins them in
// order.
#pragma once

#include "common.cuh"

namespace canopy {

bool make_bf16_box_map(CUtensorMap* m, const void* base, const uint64_t (&dim)[3], const uint64_t (&stride)[2],
                       const uint32_t (&size)[3]);  // verify_tc.cu

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
    int sink_full, full_from, full_to;  // key tiles [0, sink_full) and [full_from, full_to) are seen whole by all rows
};

struct Args {
    const void *q, *kc, *vc;
    void* o;
    const int32_t *table, *context, *starts, *parent, *lengths;
    int N, B, T, HQ, HKV, g;
    int pages, log_page, max_pages;
    int window, sinks;
    float scale2;  // scale * log2(e): weights are powers of two
    int rt, kt, ctas, least;      // tokens of a row tile, keys of a unit, CTAs at most, units of a CTA at least
    int slot_rows;                // rows of a slot
    // workspace
    int32_t* err;
    int4* seqs;       // [B + 1]: first row, rows, ctx, first tile (of the last: the number of tiles)
    int64_t* line;    // [number of tiles + 1]: units before the tile, of all key heads
    int2* first_tile;  // [ctas]: the tile that CTA c begins in, and its sequence
    int4* joins;      // [ctas - 1]: of the item first cut behind CTA c its first row, tokens, key head, and
                      // pieces (0: none is)
    uint32_t* mask;   // trees: [N][kMaskWords], the nodes of a row's path that it sees
    int32_t* depth;   // trees: [N]
    float* part;      // [2 ctas] slots
};

// ---------------------------------------------------------------------------
// Whether every row of the tile sees all of a key tile.
__device__ inline bool all_see(const Tile& tile, int key_tile) {
    return key_tile < tile.sink_full || (key_tile >= tile.full_from && key_tile < tile.full_to);
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
    r.first = r.near / a.kt;
    r.sink_tiles = min((r.sink_end + a.kt - 1) / a.kt, r.first);
    r.units = r.sink_tiles + (r.hi + a.kt - 1) / a.kt - r.first;
    // all rows see the keys before the first row's new ones, as far back as the last row's window
    const int lim = r.ctx + (a.parent ? 0 : r.t0 + 1);
    const int64_t low = int64_t(r.ctx) + (a.parent ? r.n : r.t0 + r.ntok) - a.window;
    r.sink_full = min(a.sinks, lim) / a.kt;
    r.full_from = low > 0 ? int((low + a.kt - 1) / a.kt) : 0;
    r.full_to = lim / a.kt;
    return r;
}

// The sequence that tile i belongs to: the last whose first tile is not behind it.
__device__ inline int sequence_at(const int4* seqs, int B, int i) {
    int b = 0, e = B;
    while (e - b > 1) {
        const int m = (b + e) >> 1;
        if (seqs[m].w <= i) b = m; else e = m;
    }
    return b;
}

// Rows and context of a sequence brought into what its page table has room for.
__device__ inline void fit(const Args& a, int& n, int& ctx, int* bad) {
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
}

// The plan, by a whole block of NT threads: seqs, line, and the number of tiles
// (returned).  Starts out of order or range are read as their
// running maximum, lengths and contexts as the nearest that fit; these set bits
// in *bad.
template <int NT>
__device__ inline int make_plan(const Args& a, int4* seqs, int64_t* line_of, int* bad) {
    __shared__ int wi[NT / 32];
    __shared__ int64_t wl[NT / 32];
    const auto most = [](int x, int y) { return max(x, y); };
    const auto sum = [](int64_t x, int64_t y) { return x + y; };
    const auto isum = [](int x, int y) { return x + y; };
    const int tid = threadIdx.x;
    if (!a.starts && a.B <= 32 && a.T <= a.rt) {  // a tile a stream at most: one warp, no meetings on the way
        if (tid < 32) {
            const bool stream = tid < a.B;
            int n = stream ? min(a.T, stream_len(a.lengths, tid, a.T, bad)) : 0;
            int ctx = n > 0 ? a.context[tid] : 0;
            fit(a, n, ctx, bad);
            const uint32_t filled = __ballot_sync(0xffffffffu, n > 0);
            const int tile = __popc(filled & ((1u << tid) - 1)), ntiles = __popc(filled);
            const int4 s = make_int4(tid * a.T, n, ctx, tile);
            const int64_t units = n > 0 ? int64_t(make_tile(a, tid, s, 0).units) * a.HKV : 0;
            int64_t upto = units;
#pragma unroll
            for (int x = 1; x < 32; x *= 2) {
                const int64_t y = __shfl_up_sync(0xffffffffu, upto, x);
                if (tid >= x) upto += y;
            }
            if (stream) seqs[tid] = s;
            if (n > 0) line_of[tile] = upto - units;
            if (tid == 31) {
                seqs[a.B] = make_int4(a.N, 0, 0, ntiles);
                line_of[ntiles] = upto;
            }
        }
        __syncthreads();
        return seqs[a.B].w;
    }
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
            ctx = n > 0 ? a.context[b] : 0;
            fit(a, n, ctx, bad);
        } else {
            n = 0;
        }
        const int nt = (n + a.rt - 1) / a.rt;
        const int upto = carry + block_scan<NT>(nt, isum, wi, total);
        if (b < a.B) seqs[b] = make_int4(lo, n, ctx, upto - nt);
        carry += total;
    }
    const int ntiles = carry;
    if (tid == 0) seqs[a.B] = make_int4(a.N, 0, 0, ntiles);
    __syncthreads();
    int64_t line = 0, ltotal;
    for (int i0 = 0; i0 < ntiles; i0 += NT) {
        const int i = i0 + tid;
        int64_t units = 0;
        if (i < ntiles) {
            const int b = sequence_at(seqs, a.B, i);
            const int4 s = seqs[b];
            units = int64_t(make_tile(a, b, s, i - s.w).units) * a.HKV;
        }
        const int64_t upto = line + block_scan<NT>(units, sum, wl, ltotal);
        if (i < ntiles) line_of[i] = upto - units;
        line += ltotal;
    }
    if (tid == 0) line_of[ntiles] = line;
    __syncthreads();
    return ntiles;
}

// How many CTAs share the work: no part is shorter than `least` units.
__device__ inline int parts(const Args& a, int64_t units) {
    const int64_t most = units / a.least;
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
    bool whole;
    int slot;  // where it goes if it is not the whole
};

// Walks a CTA's pieces.
struct Walk {
    const int4* seqs;
    const int64_t* line;
    int64_t units, at, end;
    int ctas, tile, b;
    // CTA c's part of the plan.
    __device__ Walk(const Args& a, const int4* seqs, const int64_t* line, int c, const int2* first_tile)
        : seqs(seqs), line(line), units(0), at(0), end(0), ctas(1), tile(0), b(0) {
        const int ntiles = seqs[a.B].w;
        units = line[ntiles];
        ctas = parts(a, units);
        if (c >= ctas || units == 0) return;
        at = cta_begin(units, ctas, c);
        end = cta_begin(units, ctas, c + 1);
        if (first_tile) {
            tile = first_tile[c].x;
            b = first_tile[c].y;
        } else {
            tile = tile_at(line, ntiles, at);
            b = sequence_at(seqs, a.B, tile);
        }
    }
    __device__ bool next(const Args& a, Piece& p) {
        if (at >= end) return false;
        while (line[tile + 1] <= at) ++tile;
        while (seqs[b + 1].w <= tile) ++b;
        const int4 s = seqs[b];
        p.tile = make_tile(a, b, s, tile - s.w);
        const int64_t rel = at - line[tile];
        p.h = int(rel / p.tile.units);
        p.u0 = int(rel - int64_t(p.h) * p.tile.units);
        p.u1 = int(min(int64_t(p.tile.units), p.u0 + (end - at)));
        p.whole = p.u0 == 0 && p.u1 == p.tile.units;
        p.slot = 2 * int(blockIdx.x) + (p.u0 == 0);
        at += p.u1 - p.u0;
        return true;
    }
};
// Slot of piece i of an item that begins in CTA `first`.
__device__ inline int slot_of(int first, int i) { return 2 * (first + i) + (i == 0); }

// ---------------------------------------------------------------------------
// What the two kernels on the tensor cores share.

__device__ inline void prefetch_map(const CUtensorMap* m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

constexpr float kGrow = 8.f;  // a row's maximum is kept until it grows by this, in powers of two

__device__ inline float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ inline uint32_t pack_bf16(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// The first and the second of a pair of bf16 values.
__device__ inline float first_of(uint32_t x) { return __uint_as_float(x << 16); }
__device__ inline float second_of(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

// Bits [a, b) of a word.
__device__ inline uint32_t range_bits(int a, int b) {
    a = min(max(a, 0), 32);
    b = min(max(b, a), 32);
    return uint32_t((1ull << b) - (1ull << a));
}
// Which of the keys [base, base + 32) a row sees, by its depth (its index in the
// sequence without a tree) and its path (mask, null without a tree).  The row is at
// position t = ctx + depth.  Key j is a new one of a tree if j >= ctx there: it is seen
// if node j - ctx is in the mask (those out of the window are not).  Any other is seen
// if j <= t, and t - j < window or j < sinks.
__device__ inline uint32_t seen_bits(const Args& a, const Tile& tile, int depth, const uint32_t* mask, int base) {
    const int pos = tile.ctx + depth;
    const int end = (mask ? min(pos, tile.ctx - 1) : pos) + 1;  // past the last one in the cache, or in all
    const int64_t near = int64_t(pos) - a.window + 1 - base;
    uint32_t bits = range_bits(int(near > 0 ? near : 0), end - base) | range_bits(0, min(a.sinks, end) - base);
    const int p = base - tile.ctx;
    if (mask && p > -32 && p < kMaxT) {
        if (p < 0) {
            bits |= mask[0] << -p;
        } else {
            const uint32_t lo = mask[p >> 5], hi = (p >> 5) + 1 < kMaskWords ? mask[(p >> 5) + 1] : 0u;
            bits |= __funnelshift_r(lo, hi, p & 31);
        }
    }
    return bits;
}

// Of a pair of bf16 values: whether both are finite, and the pair with those that are not as zeros.
__device__ inline bool finite_pair(uint32_t x) {
    return (x & 0x7F80u) != 0x7F80u && (x & 0x7F800000u) != 0x7F800000u;
}
__device__ inline uint32_t finite_part(uint32_t x) {
    return x & (((x & 0x7F80u) != 0x7F80u ? 0x0000FFFFu : 0u) | ((x & 0x7F800000u) != 0x7F800000u ? 0xFFFF0000u : 0u));
}

// What the products leave out for a row that sees it: the values that are not
// finite, in the tiles of [u0, u1) whose keys the tile's rows see in part.  They go
// to the row's sums behind the last product, add(c, x, y) for column pair c, read
// from the pages again: a row that sees such a value is rare.  A thread has Words
// first, first + step, ... of a row, of W pairs each.
template <typename Words, typename Add>
__device__ inline void add_not_finite(const Args& a, const Piece& p, int depth, const uint32_t* mask, int d, int first,
                                      int step, Add add) {
    constexpr int W = sizeof(Words) / 4;
    const int words = d / (2 * W);
#pragma unroll 1
    for (int c = first; c < words; c += step) {
        float sum[2 * W] = {};
        bool more = true;  // some column may still change
#pragma unroll 1
        for (int u = p.u0; more && u < p.u1; ++u) {
            const int kt = key_tile(p.tile, u), end = (kt + 1) * a.kt;
            if (all_see(p.tile, kt)) continue;
#pragma unroll 1
            for (int base = kt * a.kt; more && base < end; base += 32) {
                uint32_t seen = seen_bits(a, p.tile, depth, mask, base) & range_bits(0, end - base);
#pragma unroll 1
                for (; seen; seen &= seen - 1) {
                    const int key = base + __ffs(seen) - 1;
                    const int page = a.table[size_t(p.tile.b) * a.max_pages + (key >> a.log_page)];
                    if (page < 0 || page >= a.pages) continue;
                    const size_t row = (((size_t(page) * a.HKV + p.h) << a.log_page) + (key & ((1 << a.log_page) - 1)));
                    const Words x = static_cast<const Words*>(a.vc)[row * words + c];
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        const uint32_t y = reinterpret_cast<const uint32_t*>(&x)[i], bad = y ^ finite_part(y);
                        sum[2 * i] += first_of(bad);
                        sum[2 * i + 1] += second_of(bad);
                    }
                }
                more = false;
#pragma unroll
                for (int i = 0; i < 2 * W; ++i) more |= sum[i] == sum[i];
            }
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (sum[2 * i] != 0.f || sum[2 * i + 1] != 0.f) add(W * c + i, sum[2 * i], sum[2 * i + 1]);
    }
}

// A wait of a whole warp, which goes on or gives up together.
__device__ inline bool warp_wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}
// Waits for a barrier's phases in turn.
struct Phase {
    uint32_t bit = 0;
    __device__ bool wait(uint64_t* bar) {
        const bool ok = warp_wait(bar, bit);
        bit ^= 1;
        return ok;
    }
};
// A place in the ring of stages.
template <int STAGES>
struct Ring {
    int at = 0;
    uint32_t phase = 0;
    __device__ void step() {
        if (++at == STAGES) {
            at = 0;
            phase ^= 1;
        }
    }
    __device__ void back() {
        if (at-- == 0) {
            at = STAGES - 1;
            phase ^= 1;
        }
    }
};

}  // namespace att
}  // namespace canopy
