// Attention of many new rows over a paged cache on the tensor cores (bf16).
//
// A CTA works on up to 256 rows of one (sequence, key head): two halves of 128
// lanes, each of 128 / g tokens with the g query heads that share the key head,
// against tiles of KT keys.  Per half and key tile
//     S = Q K^T            (128 x KT x d, Q and K in shared memory)
//     P = 2^(scale2 S - m) (four warps, a row a thread; rounded to bf16)
//     O += P V             (128 x d x KT, P from tensor memory)
// with S, P and O of both halves in the 512 columns of tensor memory.  KT is what
// leaves P a place of its own (80 for d = 128, 128 for d = 64): as soon as the
// softmax has S in registers the next tile's S is formed, and one thread a half
// issues both products.  Tiles of 128 with P over S were as fast only with the
// halves half a tile apart (a chunk of 4,096 tokens behind 28,672, 32/8 heads: 1,594
// us; 1,460 to 1,587 this way, 1.3 PFLOP/s, and a window of 1,024 292 and 187 us);
// tiles of 64 with two P took 1,976 us.  The softmax's warps hold it: 2,300 cycles a tile of
// 80 keys, where the products take 1,280 (tensor pipe 0.6 of active cycles).  They
// spill 64 bytes of stores and 108 of loads (d = 64: 132 and 224) at 168 registers.
//
// m is the running maximum as of the last time that it grew by more than 2^8:
// until then the weights are merely larger than 1, by less than 2^8, and neither
// sums nor roundings know the difference; when it does grow, the row's thread
// scales O.  The weights are rounded to bf16 for the second product (their sum
// is of the unrounded ones): off by up to 2^-8 each, which averages out over the
// keys.
//
// Key tiles come by TMA, one box per page (or 16 keys, where tiles and pages
// cut each other) and 64 columns, into a ring of stages that K and V tiles take
// in turns.  A page that no row sees is read at a coordinate outside the cache, as
// zeros.  Where not every row sees every key of a tile, the softmax's warps look
// through its V first: what no row sees, and what is not finite, becomes zero (0
// times it would reach every row's sum), and a row that sees such a value has it
// added to its sum behind the last product.  (A warp of its own for the look took
// 246 us for the window case.)
#include "attend.cuh"

namespace canopy {
namespace att {
namespace tcg {

constexpr int NT = 384;
constexpr uint32_t kCols = 512;

template <int D>
struct Shape {
    static constexpr int KT = D == 128 ? 80 : 128;  // keys of a tile
    static constexpr int COLS = 256 - D;            // tensor memory of a half's S and P
    static constexpr int PCOL = KT;                 // P's place in it
    static_assert(KT + KT / 2 <= COLS, "S and P");
    static constexpr int FIRST = (KT / 16 + 1) / 2;  // the 16-key steps of a tile's P that are handed over first
    static constexpr int QTILE = 128 * D * 2;        // a half's Q: [d / 64][128 rows][128 bytes]
    static constexpr int TILE = KT * D * 2;          // K or V: [d / 64][KT rows][128 bytes]
    static constexpr int STAGES = (D == 128 ? 163840 : 131072) / TILE;
    static constexpr int Q = 0, KV = 2 * QTILE, BARS = KV + STAGES * TILE;
    // barriers: Q full, Q read; per stage full, empty, and V looked through; per half S full, S read, P there (in two
    // parts), O done, and all done
    static constexpr int NBAR = 2 + 3 * STAGES + 12;
    static_assert(STAGES % 2 == 0, "K tiles in even stages, V tiles in odd ones");
    // [STAGES][8]: keys with a value that is not finite, by the warp that found them
    static constexpr int POISON = (BARS + 8 * NBAR + 15) / 16 * 16;
    static constexpr int MISC = POISON + 32 * STAGES;  // tensor memory's address
    static constexpr int TOTAL = MISC + 16;
};
static_assert(Shape<128>::TOTAL + 1024 <= 232448 && Shape<64>::TOTAL + 1024 <= 232448, "shared memory");

__device__ inline float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Keys of a box at most: tiles and pages may cut each other anywhere but at multiples of 16 keys.
__host__ __device__ constexpr int box_keys(int d) { return d == 128 ? 16 : 128; }

template <int D>
__global__ void __launch_bounds__(NT, 1)
    attend_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                  const __grid_constant__ CUtensorMap mapV, const Args a) {
    using Sh = Shape<D>;
    constexpr int HALVES = D / 64, KT = Sh::KT, STAGES = Sh::STAGES;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Sh::BARS);
    uint64_t *q_full = bars, *q_read = bars + 1, *full = bars + 2, *empty = full + STAGES, *looked = empty + STAGES,
             *s_full = looked + STAGES, *s_read = s_full + 2, *p_there = s_read + 2, *o_done = p_there + 4,
             *drained = o_done + 2;
    uint32_t* poison = reinterpret_cast<uint32_t*>(sm + Sh::POISON);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + Sh::MISC);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 8) {
        tmem_alloc(tmem_slot, kCols);
        tmem_relinquish();
    }
    if (warp == 9 && lane == 0) {
        prefetch_map(&mapQ);
        prefetch_map(&mapK);
        prefetch_map(&mapV);
    }
    if (warp == 10 && lane == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_read, 2);
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 2);  // both halves' products
            mbar_init(looked + i, 256);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(s_read + i, 128);
            mbar_init(p_there + 2 * i, 128);
            mbar_init(p_there + 2 * i + 1, 128);
            mbar_init(o_done + i, 1);
            mbar_init(drained + i, 1);
        }
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_trigger();  // after the wait: the next launch may rely on everything before this one

    Walk walk(a, a.seqs, a.line, blockIdx.x, a.first_tile);
    const int half_tok = a.rt / 2;  // tokens of a half
    bool ok = true;
    Piece p;

    // 200 registers for the softmax's warps, 104 for the others: all of the 64,512 that the block was launched with
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        if (warp >= 10) {
            // ---- loads: Q and K tiles by one warp, V tiles by the other -----------------------
            // (the issue of a box takes 85 cycles and more, one lane after the other)
            const bool keys = warp == 10;
            Ring<STAGES> ring;
            if (!keys) ring.step();  // K tiles are the even stages, V tiles the odd ones
            uint32_t q_phase = 1;  // the first Q needs nothing read
            int q_loads = 0, loads = 0;
            const int box = min(1 << a.log_page, box_keys(D)), boxes = KT / box;  // keys of a box, boxes of a tile
            const int i = lane / HALVES, part = lane % HALVES;                    // a lane's box
            int bad = 0;
            while (ok && walk.next(a, p)) {
                const Tile& tile = p.tile;
                const bool two = tile.ntok > half_tok;
                if (keys) {
                    ok = warp_wait(q_read, q_phase);
                    q_phase ^= 1;
                    if (!ok) break;
                    ++q_loads;
                    if (lane == 0) {
                        mbar_expect_tx(q_full, (two ? 2 : 1) * HALVES * half_tok * a.g * 128);
                        for (int h = 0; h < (two ? 2 : 1); ++h)
                            for (int c = 0; c < HALVES; ++c)
                                tma_load_3d(sm + Sh::Q + h * Sh::QTILE + c * 16384, &mapQ, q_full, 64 * c, p.h * a.g,
                                            tile.row + h * half_tok);
                    }
                }
                for (int u = p.u0; ok && u < p.u1; ++u) {
                    const int key = key_tile(tile, u) * KT + i * box;
                    int z = a.pages * a.HKV;  // outside: zeros
                    if (i < boxes && (key < tile.sink_end || (key + box > tile.near && key < tile.hi))) {
                        const int page = a.table[size_t(tile.b) * a.max_pages + (key >> a.log_page)];
                        if (page < 0 || page >= a.pages) bad = CANOPY_DEVERR_PAGE;
                        else z = page * a.HKV + p.h;
                    }
                    ok = warp_wait(empty + ring.at, ring.phase ^ 1);
                    if (!ok) break;
                    ++loads;
                    if (lane == 0) mbar_expect_tx(full + ring.at, Sh::TILE);
                    __syncwarp();
                    if (i < boxes)
                        tma_load_3d(sm + Sh::KV + ring.at * Sh::TILE + part * (KT * 128) + i * box * 128,
                                    keys ? &mapK : &mapV, full + ring.at, 64 * part, key & ((1 << a.log_page) - 1), z);
                    ring.step();
                    ring.step();
                }
            }
            if (bad) raise_err(a.err, bad);
            // no copy is left in flight, should another warp have given up
            if (q_loads) warp_wait(q_full, (q_loads - 1) & 1);
            for (int i = min(loads, STAGES / 2); i > 0; --i) {
                ring.back();
                ring.back();
                warp_wait(full + ring.at, ring.phase);
            }
        } else {
            // ---- products: of one half, by one thread ----------------------------------------
            if (lane == 0) {
                const int h = warp - 8;
                Ring<STAGES> ring, look;
                uint32_t q_phase = 0, s_phase = 1, p_phase = 0;
                // (descriptors hold addresses in units of 16 bytes: a step is an addition)
                const uint64_t q = sdesc_sw128(smem_u32(sm + Sh::Q) + h * Sh::QTILE);
                const uint32_t kv = smem_u32(sm + Sh::KV), S = tmem + Sh::COLS * h, P = S + Sh::PCOL,
                               O = tmem + 2 * Sh::COLS + D * h;
                // S of the key tile in the ring's next stage, once the one before is in registers
                auto scores = [&](bool last) {
                    if (!mbar_wait(full + ring.at, ring.phase) || !mbar_wait(s_read + h, s_phase)) return false;
                    s_phase ^= 1;
                    tc_fence_after();
                    const uint64_t k = sdesc_sw128(kv + ring.at * Sh::TILE);
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
                        mma_bf16_ss(S, q + (i >> 2) * 1024 + (i & 3) * 2, k + (i >> 2) * (KT * 8) + (i & 3) * 2,
                                    idesc_bf16(128, KT), i > 0);
                    mma_commit(s_full + h);
                    mma_commit(empty + ring.at);
                    if (last) mma_commit(q_read);
                    ring.step();
                    return true;
                };
                while (ok && walk.next(a, p)) {
                    const Tile& tile = p.tile;
                    const bool mine = h == 0 || tile.ntok > half_tok;
                    ok = mbar_wait(q_full, q_phase);
                    q_phase ^= 1;
                    if (!ok) break;
                    if (!mine) {  // the stages pass by
                        mbar_arrive(q_read);
                        for (int u = p.u0; ok && u < p.u1; ++u) {
                            for (int i = 0; ok && i < 2; ++i) {
                                ok = mbar_wait(full + ring.at, ring.phase);
                                mbar_arrive(empty + ring.at);
                                ring.step();
                            }
                            if (!all_see(tile, key_tile(tile, u))) look.step();
                        }
                        continue;
                    }
                    ok = scores(p.u0 + 1 == p.u1);
                    for (int u = p.u0; ok && u < p.u1; ++u) {
                        const bool all = all_see(tile, key_tile(tile, u));
                        const Ring<STAGES> v = ring;
                        ring.step();
                        if (u + 1 < p.u1) ok = scores(u + 2 == p.u1);
                        ok = ok && mbar_wait(full + v.at, v.phase);
                        if (ok && !all) {
                            ok = mbar_wait(looked + look.at, look.phase);
                            look.step();
                        }
                        const uint64_t vd = sdesc_sw128_mn(kv + v.at * Sh::TILE, KT * 128);
#pragma unroll
                        for (int part = 0; part < 2; ++part) {
                            ok = ok && mbar_wait(p_there + 2 * h + part, p_phase);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll
                            for (int i = part * Sh::FIRST; i < (part ? KT / 16 : Sh::FIRST); ++i)
                                mma_bf16_ts(O, P + 8 * i, vd + i * 128, idesc_bf16(128, D) | kIdescBMnMajor,
                                            u > p.u0 || i > 0);
                        }
                        if (!ok) break;
                        p_phase ^= 1;
                        mma_commit(o_done + h);
                        mma_commit(empty + v.at);
                    }
                }
                mma_commit(drained + h);
                mbar_wait(drained + h, 0);
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ---- softmax ------------------------------------------------------------------
        const int h = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = tmem + (uint32_t((warp & 3) * 32) << 16), S = lanes + Sh::COLS * h, P = S + Sh::PCOL,
                       O = lanes + 2 * Sh::COLS + D * h;
        Ring<STAGES> look, ring;
        ring.step();  // the stage of the unit's V
        Phase scores_ready, added;
        const int tok_in_half = r / a.g, head = r % a.g;
        while (ok && walk.next(a, p)) {
            const Tile& tile = p.tile;
            const bool two = tile.ntok > half_tok, mine = h == 0 || two;  // this half has rows
            const int tok = h * half_tok + tok_in_half;
            const bool valid = tok_in_half < half_tok && tok < tile.ntok;
            const int row = tile.row + min(tok, tile.ntok - 1);
            const int depth = a.parent ? (mine ? a.depth[row] : 0) : tile.t0 + tok;
            const uint32_t* mask = a.parent ? a.mask + size_t(row) * kMaskWords : nullptr;
            float m = -INFINITY, base = 0.f;  // the maximum that the weights are relative to, scaled
            float l = 0.f;
            bool left_out = false;  // the row sees a value that its products leave out
            for (int u = p.u0; u < p.u1; ++u) {
                const int kt = key_tile(tile, u), key = kt * KT;
                const bool all = all_see(tile, kt);
                const Ring<STAGES> v = look, stage = ring;
                if (!all) look.step();
                ring.step();
                ring.step();
                if (!mine) continue;
                ok = scores_ready.wait(s_full + h);
                if (!ok) break;
                tc_fence_after();
                uint32_t s[KT];
#pragma unroll
                for (int c = 0; c + 32 <= KT; c += 32) tmem_ld32(S + c, s + c);
                if (KT % 32) tmem_ld16(S + KT / 32 * 32, *reinterpret_cast<uint32_t(*)[16]>(s + KT / 32 * 32));
                tmem_wait_ld();
                tc_fence_before();
                mbar_arrive(s_read + h);
                if (!all) {
                    constexpr int W = (KT + 31) / 32;
                    uint32_t seen[W];
#pragma unroll
                    for (int c = 0; c < W; ++c) seen[c] = seen_bits(a, tile, depth, mask, key + 32 * c);
#pragma unroll
                    for (int j = 0; j < KT; ++j)
                        if (!((seen[j >> 5] >> (j & 31)) & 1u)) s[j] = 0xFF800000u;
                    // this warp's eighth of V (of one half's four warps two)
                    ok = warp_wait(full + stage.at, stage.phase);
                    if (!ok) break;
                    constexpr int ROWS = KT / 8, CHUNKS = ROWS * HALVES * 8 / 32;  // keys, 16 bytes a lane
                    uint32_t* found = poison + 8 * v.at;
                    for (int w = warp; w < 8; w += two ? 8 : 4) {
                        uint4* tile_v = reinterpret_cast<uint4*>(sm + Sh::KV + stage.at * Sh::TILE);
                        uint32_t bad = 0;
#pragma unroll
                        for (int e = 0; e < CHUNKS; ++e) {
                            const int id = 32 * e + lane, j = (id >> 3) % ROWS;
                            uint4* at = tile_v + ((id >> 3) / ROWS * KT + ROWS * w + j) * 8 + (id & 7);
                            const uint4 x = *at;
                            const bool there = in_reach(tile, key + ROWS * w + j);
                            if (there && finite_pair(x.x) && finite_pair(x.y) && finite_pair(x.z) && finite_pair(x.w))
                                continue;
                            *at = there ? make_uint4(finite_part(x.x), finite_part(x.y), finite_part(x.z), finite_part(x.w))
                                        : make_uint4(0, 0, 0, 0);
                            if (there) bad |= 1u << j;
                        }
                        bad = __reduce_or_sync(0xffffffffu, bad);
                        if (lane == 0) found[w] = bad;
                        fence_proxy_async_smem();
                        mbar_arrive(looked + v.at);
                    }
                    ok = warp_wait(looked + v.at, v.phase);
                    if (!ok) break;
                    const uint4 f0 = *reinterpret_cast<uint4*>(found), f1 = *reinterpret_cast<uint4*>(found + 4);
                    if (f0.x | f0.y | f0.z | f0.w | f1.x | f1.y | f1.z | f1.w)
                        for (int j = 0; j < KT; ++j)
                            if (((seen[j >> 5] >> (j & 31)) & 1u) && ((found[j / ROWS] >> (j % ROWS)) & 1u)) left_out = true;
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < KT; j += 8)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        top[c] = max3(top[c], __uint_as_float(s[j + 2 * c]), __uint_as_float(s[j + 2 * c + 1]));
                const float t = a.scale2 * fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                const bool grow = t > m + kGrow;  // (the first finite one too)
                if (u > p.u0) {  // the product before has read P and added to O
                    ok = added.wait(o_done + h);
                    if (!ok) break;
                    tc_fence_after();
                }
                if (__any_sync(0xffffffffu, grow)) {
                    const float keep = grow ? exp2_approx(m - t) : 1.f;
                    if (grow) {
                        m = t;
                        base = t;
                    }
                    l *= keep;
                    if (u > p.u0) {
#pragma unroll
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(O + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * keep);
                            tmem_st16(O + c, o);
                        }
                    }
                }
                const uint64_t sc = pack2(a.scale2, a.scale2), mb = pack2(-base, -base);
                uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
                for (int c = 0; c < KT / 16; ++c) {
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float x, y;
                        unpack2(fma2(pack2(__uint_as_float(s[16 * c + 2 * j]), __uint_as_float(s[16 * c + 2 * j + 1])),
                                     sc, mb),
                                x, y);
                        x = exp2_approx(x);
                        y = exp2_approx(y);
                        if (j & 1) sum1 = add2(sum1, pack2(x, y));
                        else sum0 = add2(sum0, pack2(x, y));
                        w[j] = pack_bf16(x, y);
                    }
                    tmem_st8(P + 8 * c, w);
                    if (c == Sh::FIRST - 1 || c == KT / 16 - 1) {
                        tmem_wait_st();
                        tc_fence_before();
                        mbar_arrive(p_there + 2 * h + (c != Sh::FIRST - 1));
                    }
                }
                float x, y;
                unpack2(add2(sum0, sum1), x, y);
                l += x + y;
            }
            if (!ok) break;
            if (!mine) continue;
            ok = added.wait(o_done + h);
            if (!ok) break;
            tc_fence_after();
            if (p.whole) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o) + (size_t(row) * a.HQ + p.h * a.g + head) * D;
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(O + c, o);
                    tmem_wait_ld();
                    if (valid)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint4 w;
                            w.x = pack_bf16(__uint_as_float(o[8 * j]) * inv, __uint_as_float(o[8 * j + 1]) * inv);
                            w.y = pack_bf16(__uint_as_float(o[8 * j + 2]) * inv, __uint_as_float(o[8 * j + 3]) * inv);
                            w.z = pack_bf16(__uint_as_float(o[8 * j + 4]) * inv, __uint_as_float(o[8 * j + 5]) * inv);
                            w.w = pack_bf16(__uint_as_float(o[8 * j + 6]) * inv, __uint_as_float(o[8 * j + 7]) * inv);
                            *reinterpret_cast<uint4*>(out + c + 8 * j) = w;
                        }
                }
                if (valid && left_out)
                    add_not_finite<uint4>(a, p, depth, mask, D, 0, 1, [&](int c, float x, float y) {
                        uint32_t& pair = reinterpret_cast<uint32_t*>(out)[c];
                        pair = pack_bf16(first_of(pair) + x, second_of(pair) + y);
                    });
                __syncwarp();
                continue;
            }
            // a slot: per half [D / 4][rows] float4, then the rows' m and l
            const int hr = min(a.slot_rows, 128);
            const size_t half = size_t(hr) * (D + 2);
            float* slot = a.part + (size_t(p.slot) * (a.slot_rows / hr) + h) * half;
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32(O + c, o);
                tmem_wait_ld();
                if (r < hr)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        reinterpret_cast<uint4*>(slot)[(c / 4 + j) * hr + r] =
                            make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            }
            if (r < hr) {
                slot[hr * D + r] = m;
                slot[hr * D + hr + r] = l;
            }
            if (valid && left_out)
                add_not_finite<uint4>(a, p, depth, mask, D, 0, 1, [&](int c, float x, float y) {
                    float* at = slot + (c / 2 * hr + r) * 4 + 2 * (c % 2);
                    at[0] += x;
                    at[1] += y;
                });
            __syncwarp();
        }
    }
    if (!ok && lane == 0) raise_err(a.err, CANOPY_DEVERR_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

// Joins the pieces of an item that is cut: block (c, e) rows 32 e .. 32 e + 31 of the
// one whose first cut is between CTA c and c + 1.  A thread has four columns of
// four of the rows, eight threads side by side eight rows (128 bytes of a piece).
template <int D>
__global__ void __launch_bounds__(2 * D) join_kernel(const Args a) {
    // The plan is older than the launch that this one waits for.  Every block waits, one without a cut too: the
    // launch behind this one relies on the one before it through this one's end.
    const int c = blockIdx.x;
    const int4 join = a.joins[c];
    const int row = join.x, ntok = join.y, h = join.z, pieces = join.w;
    const int hr = min(a.slot_rows, 128), col = threadIdx.x >> 3;
    const size_t size = size_t(hr) * (D + 2), next = a.slot_rows / hr * size;
    pdl_wait();
    pdl_trigger();
    if (pieces == 0) return;
    // four rows a thread, whose reads of two pieces are all on their way at a time
    const float* part[4];
    float top[4], sum[4];
    float4 x[4];
    int lanes[4], out_row[4];
    bool there[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int r = 32 * blockIdx.y + 8 * e + (threadIdx.x & 7), half = r >> 7, lane = r & 127;
        const int tok = half * (a.rt / 2) + lane / a.g;
        there[e] = r < a.slot_rows && lane / a.g < a.rt / 2 && tok < ntok;
        out_row[e] = (row + tok) * a.HQ + h * a.g + lane % a.g;
        part[e] = a.part + half * size;
        lanes[e] = lane;
        top[e] = -INFINITY;
        sum[e] = 0.f;
        x[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int i0 = 0; i0 < pieces; i0 += 2) {
        float m[4][2], l[4][2];
        float4 y[4][2];
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[e][i] = -INFINITY;
                l[e][i] = 0.f;
                y[e][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (!there[e] || i0 + i >= pieces) continue;
                const float* in = part[e] + slot_of(c, i0 + i) * next;
                m[e][i] = in[hr * D + lanes[e]];
                l[e][i] = in[hr * D + hr + lanes[e]];
                y[e][i] = reinterpret_cast<const float4*>(in)[col * hr + lanes[e]];
            }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float before = top[e];
            top[e] = fmaxf(top[e], fmaxf(m[e][0], m[e][1]));
            const float from = top[e] == -INFINITY ? 0.f : top[e], keep = exp2_approx(before - from);
            const float f0 = exp2_approx(m[e][0] - from), f1 = exp2_approx(m[e][1] - from);
            sum[e] = sum[e] * keep + f0 * l[e][0] + f1 * l[e][1];
            x[e].x = x[e].x * keep + f0 * y[e][0].x + f1 * y[e][1].x;
            x[e].y = x[e].y * keep + f0 * y[e][0].y + f1 * y[e][1].y;
            x[e].z = x[e].z * keep + f0 * y[e][0].z + f1 * y[e][1].z;
            x[e].w = x[e].w * keep + f0 * y[e][0].w + f1 * y[e][1].w;
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (!there[e]) continue;
        const float f = sum[e] == 0.f ? 0.f : 1.f / sum[e];
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + size_t(out_row[e]) * D + 4 * col) =
            make_uint2(pack_bf16(x[e].x * f, x[e].y * f), pack_bf16(x[e].z * f, x[e].w * f));
    }
}

}  // namespace tcg

// Rows of a tile are 2 (128 / g) tokens of g heads.
int tc_tile_tokens(int g) { return 2 * (128 / g); }
int tc_tile_keys(int d) { return d == 128 ? tcg::Shape<128>::KT : tcg::Shape<64>::KT; }

template <int D>
static cudaError_t launch_tc_d(const Args& a, cudaStream_t st) {
    CUtensorMap mq, mk, mv;
    const uint64_t row = D * 2, page = uint64_t(1) << a.log_page;
    const uint32_t keys = uint32_t(page < tcg::box_keys(D) ? page : tcg::box_keys(D));
    if (!make_bf16_box_map(&mq, a.q, {D, uint64_t(a.HQ), uint64_t(a.N)}, {row, a.HQ * row},
                           {64, uint32_t(a.g), uint32_t(a.rt / 2)}) ||
        !make_bf16_box_map(&mk, a.kc, {D, page, uint64_t(a.pages) * a.HKV}, {row, page * row}, {64, keys, 1}) ||
        !make_bf16_box_map(&mv, a.vc, {D, page, uint64_t(a.pages) * a.HKV}, {row, page * row}, {64, keys, 1}))
        return cudaErrorInvalidValue;
    const int smem = tcg::Shape<D>::TOTAL + 1024;
    static OncePerDevice once;
    cudaError_t e = once([=] { return allow_smem(tcg::attend_kernel<D>, smem); });
    if (e != cudaSuccess) return e;
    e = launch_pdl(tcg::attend_kernel<D>, dim3(a.ctas), dim3(tcg::NT), smem, st, mq, mk, mv, a);
    if (e != cudaSuccess) return e;
    if (a.ctas == 1) return cudaSuccess;  // nothing is cut
    return launch_pdl(tcg::join_kernel<D>, dim3(a.ctas - 1, (a.slot_rows + 31) / 32), dim3(2 * D), 0, st, a);
}

cudaError_t launch_tc(const Args& a, int d, cudaStream_t st) {
    return d == 128 ? launch_tc_d<128>(a, st) : launch_tc_d<64>(a, st);
}

}  // namespace att
}  // namespace canopy
