// Attention of new rows over a paged cache: the plan, the trees' masks, and the
// fp32 path on CUDA cores.
//
// For row i: o_i = sum_j p_ij v_j / sum_j p_ij, p_ij = 2^(s_ij - m_i), s_ij =
// scale log2(e) q_i.k_j over the keys that i sees, m_i the running maximum.
#include "attend.cuh"

#include <type_traits>

namespace canopy {
namespace att {

// Block 0 plans; block 1 + b, with trees, lists the paths of stream b.
__global__ void __launch_bounds__(256) plan_kernel(const Args a) {
    pdl_wait();
    pdl_trigger();  // after the wait: the next launch may rely on everything before this one
    if (blockIdx.x == 0) {
        int bad = 0;
        const int ntiles = make_plan<256>(a, a.seqs, a.line, &bad);
        if (bad) raise_err(a.err, bad);
        const int64_t units = a.line[ntiles];
        const int ctas = parts(a, units);
        for (int c = threadIdx.x; c < a.ctas; c += 256) {
            int4 join = make_int4(0, 0, 0, 0);
            if (c < ctas && ntiles) {
                const int64_t at = cta_begin(units, ctas, c);
                const int tile = tile_at(a.line, ntiles, at), b = sequence_at(a.seqs, a.B, tile);
                a.first_tile[c] = make_int2(tile, b);
                // whether the item that CTA c begins in was begun by the CTA before, and by no earlier one
                const int64_t line = a.line[tile];
                const int per = int((a.line[tile + 1] - line) / a.HKV), h = int((at - line) / per);
                const int64_t begin = line + int64_t(h) * per;
                if (begin != at && cta_of(units, ctas, begin) == c - 1) {
                    const Tile t = make_tile(a, b, a.seqs[b], tile - a.seqs[b].w);
                    join = make_int4(t.row, t.ntok, h, cta_of(units, ctas, begin + per - 1) - c + 2);
                }
            }
            if (c) a.joins[c - 1] = join;
        }
        return;
    }
    __shared__ int sPtr[kMaxT], sLen[kMaxT];
    __shared__ float sS[kMaxT];
    __shared__ uint64_t sM[kMaxT * 4];
    const int b = blockIdx.x - 1, i = threadIdx.x;
    int bad = 0;
    const int T = stream_len(a.lengths, b, a.T, &bad);
    const size_t row = size_t(b) * a.T + i;
    if (i < T) {
        int par = a.parent[row];
        if (i == 0 ? par != -1 : (par < 0 || par >= i)) {
            bad |= CANOPY_DEVERR_TREE;
            par = i == 0 ? -1 : 0;
        }
        sPtr[i] = par;
        sS[i] = 0.f;
    }
    if (bad) raise_err(a.err, bad);
    __syncthreads();
    jump_paths<4>(T, sPtr, sLen, sS, sM);
    if (i >= T) return;
    const int depth = sLen[i] - 1;
    a.depth[row] = depth;
    const int ctx = a.context[b];
    for (int w = 0; w < kMaskWords; ++w) {
        uint32_t m = uint32_t(sM[i * 4 + (w >> 1)] >> (32 * (w & 1)));
        if (depth >= a.window)  // the path's far nodes are out of the window
            for (uint32_t left = m; left; left &= left - 1) {
                const int j = 32 * w + __ffs(left) - 1, up = sLen[j] - 1;
                if (depth - up >= a.window && int64_t(ctx) + up >= a.sinks) m &= ~(1u << (j & 31));
            }
        a.mask[row * kMaskWords + w] = m;
    }
}

// ---------------------------------------------------------------------------
// fp32 on CUDA cores.  256 threads on R rows x 64 keys: thread (ty, tx) forms the
// scores of R / 16 rows with keys tx + 16 j, and D / 16 columns of those rows'
// outputs; a row's statistics stay with its 16 threads.  Rows and keys come by
// asynchronous copies, the next unit's while one is worked on.
namespace simt {

constexpr int KT = 64, NT = 256;

template <int D, int R>
struct Smem {
    static constexpr int LD = D + 4, LP = KT + 4;  // float4 reads of neighbouring rows on other banks
    float q[R * LD], kv[2][2][KT * LD], p[R * LP];
};

// 16 bytes to shared memory, or zeros (src is not read then).
__device__ inline void copy16(float* dst, const float* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ inline void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ inline void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D, int R>
__global__ void __launch_bounds__(NT) attend_kernel(const Args a) {
    constexpr int RR = R / 16, C4 = D / 64, LD = Smem<D, R>::LD, LP = Smem<D, R>::LP;
    extern __shared__ __align__(16) uint8_t raw[];
    Smem<D, R>& sm = *reinterpret_cast<Smem<D, R>*>(raw);
    pdl_wait();
    pdl_trigger();  // after the wait: the next launch may rely on everything before this one
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const float *q = static_cast<const float*>(a.q), *kc = static_cast<const float*>(a.kc),
                *vc = static_cast<const float*>(a.vc);
    Walk walk(a, a.seqs, a.line, blockIdx.x, a.first_tile);
    int bad = 0;
    Piece p;
    while (walk.next(a, p)) {
        const Tile& tile = p.tile;
        const int rows = tile.ntok * a.g;
        auto stage = [&](int u) {
            float *k = sm.kv[(u - p.u0) & 1][0], *v = sm.kv[(u - p.u0) & 1][1];
            for (int e = tid; e < KT * (D / 4); e += NT) {
                const int j = e / (D / 4), c = 4 * (e % (D / 4)), key = key_tile(tile, u) * KT + j;
                size_t from = 0;
                bool there = in_reach(tile, key);
                if (there) {
                    const int page = a.table[size_t(tile.b) * a.max_pages + (key >> a.log_page)];
                    there = page >= 0 && page < a.pages;
                    if (there)
                        from = (((size_t(page) * a.HKV + p.h) << a.log_page) + (key & ((1 << a.log_page) - 1))) * D + c;
                    else
                        bad = CANOPY_DEVERR_PAGE;
                }
                copy16(k + j * LD + c, kc + from, there);
                copy16(v + j * LD + c, vc + from, there);
            }
        };
        __syncthreads();
        for (int e = tid; e < R * (D / 4); e += NT) {
            const int r = e / (D / 4), c = 4 * (e % (D / 4)), i = min(r, rows - 1);
            copy16(sm.q + r * LD + c, q + (size_t(tile.row + i / a.g) * a.HQ + p.h * a.g + i % a.g) * D + c, r < rows);
        }
        stage(p.u0);
        copies_end();
        float m[RR], l[RR];
        float4 o[RR][C4];
        int depth[RR];
        const uint32_t* mask[RR];
#pragma unroll
        for (int r = 0; r < RR; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int c = 0; c < C4; ++c) o[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
            const int i = min((ty * RR + r) / a.g, tile.ntok - 1);
            depth[r] = a.parent ? a.depth[tile.row + i] : tile.t0 + i;
            mask[r] = a.parent ? a.mask + size_t(tile.row + i) * kMaskWords : nullptr;
        }
        for (int u = p.u0; u < p.u1; ++u) {
            if (u + 1 < p.u1) stage(u + 1);
            copies_end();
            copies_wait<1>();
            __syncthreads();
            const float *k = sm.kv[(u - p.u0) & 1][0], *v = sm.kv[(u - p.u0) & 1][1];
            const int kt = key_tile(tile, u);
            const bool all = all_see(tile, kt);
            float s[RR][4] = {};
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                float4 k4[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) k4[j] = *reinterpret_cast<const float4*>(k + (tx + 16 * j) * LD + c);
#pragma unroll
                for (int r = 0; r < RR; ++r) {
                    const float4 x = *reinterpret_cast<const float4*>(sm.q + (ty * RR + r) * LD + c);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[r][j] += x.x * k4[j].x + x.y * k4[j].y + x.z * k4[j].z + x.w * k4[j].w;
                }
            }
#pragma unroll
            for (int r = 0; r < RR; ++r) {
                float top = -INFINITY;
                uint32_t seen[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
                if (!all) {
                    seen[0] = seen_bits(a, tile, depth[r], mask[r], kt * KT);
                    seen[1] = seen_bits(a, tile, depth[r], mask[r], kt * KT + 32);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[r][j] *= a.scale2;
                    if (!((seen[j >> 1] >> (tx + 16 * (j & 1))) & 1u)) s[r][j] = -INFINITY;
                    top = fmaxf(top, s[r][j]);
                }
#pragma unroll
                for (int x = 8; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                top = fmaxf(top, m[r]);
                const float base = top == -INFINITY ? 0.f : top, keep = exp2f(m[r] - base);
                m[r] = top;
                l[r] *= keep;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float w = exp2f(s[r][j] - base);
                    l[r] += w;
                    sm.p[(ty * RR + r) * LP + tx + 16 * j] = w;
                }
#pragma unroll
                for (int c = 0; c < C4; ++c) {
                    o[r][c].x *= keep;
                    o[r][c].y *= keep;
                    o[r][c].z *= keep;
                    o[r][c].w *= keep;
                }
            }
            __syncwarp();  // a row's weights are written and read by one half warp
            auto sums = [&](auto masked_type) {
                constexpr bool masked = decltype(masked_type)::value;
                // (what a row does not see does not reach it, whatever it holds)
                auto add = [](float& x, float w, float y) { x = masked && w == 0.f ? x : fmaf(w, y, x); };
#pragma unroll 2
                for (int j = 0; j < KT; j += 4) {
                    float4 v4[4][C4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int c = 0; c < C4; ++c)
                            v4[i][c] = *reinterpret_cast<const float4*>(v + (j + i) * LD + 4 * tx + 64 * c);
#pragma unroll
                    for (int r = 0; r < RR; ++r) {
                        const float4 w4 = *reinterpret_cast<const float4*>(sm.p + (ty * RR + r) * LP + j);
                        const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int c = 0; c < C4; ++c) {
                                add(o[r][c].x, w[i], v4[i][c].x);
                                add(o[r][c].y, w[i], v4[i][c].y);
                                add(o[r][c].z, w[i], v4[i][c].z);
                                add(o[r][c].w, w[i], v4[i][c].w);
                            }
                    }
                }
            };
            if (all) sums(std::false_type());
            else sums(std::true_type());
            __syncthreads();
        }
#pragma unroll
        for (int r = 0; r < RR; ++r)
#pragma unroll
            for (int x = 8; x; x >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
        if (!p.whole) {  // a slot: [rows][D], then the rows' m and l
            float* out = a.part + size_t(p.slot) * R * (D + 2);
#pragma unroll
            for (int r = 0; r < RR; ++r) {
                const int row = ty * RR + r;
                if (row >= rows) continue;
#pragma unroll
                for (int c = 0; c < C4; ++c)
                    *reinterpret_cast<float4*>(out + row * D + 4 * tx + 64 * c) = o[r][c];
                if (tx == 0) {
                    out[R * D + row] = m[r];
                    out[R * D + R + row] = l[r];
                }
            }
            continue;
        }
#pragma unroll
        for (int r = 0; r < RR; ++r) {
            const int row = ty * RR + r;
            if (row >= rows) continue;
            const float f = l[r] == 0.f ? 0.f : 1.f / l[r];
            float* out = static_cast<float*>(a.o) + (size_t(tile.row + row / a.g) * a.HQ + p.h * a.g + row % a.g) * D;
#pragma unroll
            for (int c = 0; c < C4; ++c)
                *reinterpret_cast<float4*>(out + 4 * tx + 64 * c) =
                    make_float4(o[r][c].x * f, o[r][c].y * f, o[r][c].z * f, o[r][c].w * f);
        }
    }
    if (bad) raise_err(a.err, bad);
}

template <int D, int R>
cudaError_t launch(const Args& a, cudaStream_t st) {
    static OncePerDevice once;
    const auto kernel = attend_kernel<D, R>;
    cudaError_t e = once([&] { return allow_smem(kernel, int(sizeof(Smem<D, R>))); });
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(a.ctas), dim3(NT), sizeof(Smem<D, R>), st, a);
}

}  // namespace simt

// ---------------------------------------------------------------------------
// Joins the pieces of the rows whose (row tile, key head) is cut: W warps a row,
// each with every W-th piece; a lane has D / 32 columns.  Where a row has
// hundreds of pieces (a lone token behind a long cache) the reads in flight are
// what counts.
template <typename OutT, int D, int W>
__global__ void __launch_bounds__(W > 4 ? 32 * W : 128) join_rows_kernel(const Args a) {
    constexpr int ROWS = W > 4 ? 1 : 4 / W, C = D / 32;
    __shared__ float part_o[ROWS * W][D], part_m[ROWS * W], part_l[ROWS * W];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp % W;
    const int64_t id = int64_t(blockIdx.x) * ROWS + warp / W;
    const int row = int(id / a.HQ), hq = int(id % a.HQ), h = hq / a.g;
    bool cut = row < a.N;
    int first = 0, pieces = 0, r = 0;
    if (cut) {
        int b = 0, e = a.B;  // the last sequence that does not begin behind the row
        while (e - b > 1) {
            const int m = (b + e) >> 1;
            if (a.seqs[m].x <= row) b = m; else e = m;
        }
        const int4 s = a.seqs[b];
        cut = row >= s.x && row < s.x + s.y;
        if (cut) {
            const int tile = s.w + (row - s.x) / a.rt;
            r = (row - s.x) % a.rt * a.g + hq % a.g;
            const int64_t units = a.line[a.seqs[a.B].w], at = a.line[tile], per = (a.line[tile + 1] - at) / a.HKV;
            const int ctas = parts(a, units);
            first = cta_of(units, ctas, at + h * per);
            pieces = cta_of(units, ctas, at + (h + 1) * per - 1) - first + 1;
            cut = pieces > 1;
        }
    }
    float m = -INFINITY, l = 0.f, o[C] = {};
    if (cut) {  // (the same for a whole warp)
        const size_t size = size_t(a.slot_rows) * (D + 2);
        const float* stat = a.part + a.slot_rows * D + r;
        for (int base = w; base < pieces; base += 32 * W) {  // a lane reads a piece's statistics
            const int mine = base + W * lane, count = min(32, (pieces - base + W - 1) / W);
            const bool there = mine < pieces;
            const size_t slot = slot_of(first, there ? mine : base) * size;
            const float mi = there ? stat[slot] : -INFINITY, li = there ? stat[slot + a.slot_rows] : 0.f;
            float top = mi;
#pragma unroll
            for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            top = fmaxf(top, m);
            const float from = top == -INFINITY ? 0.f : top, keep = exp2f(m - from), f = exp2f(mi - from);
            m = top;
            l = l * keep + f * li;
#pragma unroll
            for (int c = 0; c < C; ++c) o[c] *= keep;
#pragma unroll 8
            for (int i = 0; i < count; ++i) {
                const float* in = a.part + slot_of(first, base + W * i) * size + r * D + C * lane;
                const float fi = __shfl_sync(0xffffffffu, f, i);
#pragma unroll
                for (int c = 0; c < C; ++c) o[c] += fi * in[c];
            }
        }
#pragma unroll
        for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    }
    if (W > 1) {
#pragma unroll
        for (int c = 0; c < C; ++c) part_o[warp][C * lane + c] = o[c];
        if (lane == 0) {
            part_m[warp] = m;
            part_l[warp] = l;
        }
        __syncthreads();
        if (w != 0) return;
        for (int i = 1; i < W; ++i) m = fmaxf(m, part_m[warp + i]);
        const float from = m == -INFINITY ? 0.f : m;
        l = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) o[c] = 0.f;
        for (int i = 0; i < W; ++i) {
            const float f = exp2f(part_m[warp + i] - from);
            l += f * part_l[warp + i];
#pragma unroll
            for (int c = 0; c < C; ++c) o[c] += f * part_o[warp + i][C * lane + c];
        }
    }
    if (!cut) return;
    const float f = l == 0.f ? 0.f : 1.f / l;
    OutT* out = static_cast<OutT*>(a.o) + (size_t(row) * a.HQ + hq) * D + C * lane;
#pragma unroll
    for (int c = 0; c < C; ++c) store_out(out + c, o[c] * f);
}

template <typename OutT, int D>
cudaError_t launch_join_rows(const Args& a, cudaStream_t st) {
    if (a.ctas == 1) return cudaSuccess;  // nothing is cut
    // (row tile, key head) items, about; each is cut into about ctas / items pieces.  Measured, the whole call with 16,
    // 4 and 1 warps a row, us: 152 pieces (one token behind 262,143, 16/2 heads) 53.6, 58.3 and 88.4; 38 (behind 32,000,
    // 16/8) 31.6, 32.7, 41.9; 19 (two, 32/8) 49.9, 49.9, 53.7; 9 (four behind 16,000) 50.3, 49.8, 52.0; 4 (eight) 88.9,
    // 89.6, 90.5; 2 (sixteen behind 8,000) 91.7, 89.0, 88.5.
    const int64_t rows = int64_t(a.N) * a.HQ, tiles = (a.N + a.rt - 1) / a.rt;
    const int64_t each = a.ctas / ((tiles > a.B ? tiles : a.B) * a.HKV);
    if (each >= 32) return launch_pdl(join_rows_kernel<OutT, D, 16>, dim3(unsigned(rows)), dim3(512), 0, st, a);
    if (each >= 4) return launch_pdl(join_rows_kernel<OutT, D, 4>, dim3(unsigned(rows)), dim3(128), 0, st, a);
    return launch_pdl(join_rows_kernel<OutT, D, 1>, dim3(unsigned((rows + 3) / 4)), dim3(128), 0, st, a);
}
cudaError_t launch_join_bf16(const Args& a, int d, cudaStream_t st) {
    return d == 128 ? launch_join_rows<__nv_bfloat16, 128>(a, st) : launch_join_rows<__nv_bfloat16, 64>(a, st);
}

// ---------------------------------------------------------------------------

int tc_tile_tokens(int g);
int tc_tile_keys(int d);
cudaError_t launch_tc(const Args& a, int d, cudaStream_t st);
cudaError_t launch_few(const Args& a, int d, cudaStream_t st);
bool few_plans(int N, int B);  // whether launch_few makes the plan itself

namespace {

constexpr int kSMs = 152;
constexpr int kLeast = 2;  // units of a CTA at least
constexpr int kFewCtas = 2 * kSMs;  // two CTAs an SM

// Rows of an unfinished piece: those of the largest row tile that a call takes.
int slot_rows(int N, int g) {
    const int64_t rows = int64_t(N) * g;
    return rows <= 16 ? 16 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256;
}

struct Layout {
    size_t seqs, line, first_tile, joins, mask, depth, part, end;
};

// For the smallest row tile that a call of these sizes may take.
Layout layout(int N, int B, int g, int d) {
    Layout w;
    size_t o = 4096;  // the error word
    w.seqs = o;       o = ws_align(o + (size_t(B) + 1) * sizeof(int4));
    w.line = o;       o = ws_align(o + (size_t(N) + B + 1) * 8);
    w.first_tile = o; o = ws_align(o + (kFewCtas + 1) * 8);
    w.joins = o;      o = ws_align(o + kFewCtas * sizeof(int4));
    w.mask = o;       o = ws_align(o + size_t(N) * kMaskWords * 4);
    w.depth = o;      o = ws_align(o + size_t(N) * 4);
    const int rows = slot_rows(N, g);
    const size_t tiles = size_t(2) * kSMs * rows, fewer = size_t(2) * kFewCtas * (rows < 64 ? 16 : 64);
    w.part = o;       o = ws_align(o + (tiles > fewer ? tiles : fewer) * (d + 2) * 4);
    w.end = o;
    return w;
}

}  // namespace

}  // namespace att

size_t attend_ws_bytes(int N, int B, int HQ, int HKV, int d) { return att::layout(N, B, HQ / HKV, d).end; }
// Rows of a sequence and key head on average: up to 16 are one row tile of the
// kernel for few rows, which reads the cache once for each.  Measured, few / tiles,
// us, 4 to 16 rows and from 20 on: 64 streams behind 4,000, 32/8 heads, 170-177 /
// 191-195 and 330-643 / 195-199; 16 streams, 16/4 heads, 32-41 / 38-43 and 60-91 / 43;
// 64 streams of 16/16 heads, 16 rows, 184 / 208.  A lone stream behind 4,000 is
// taken to the tiles early: 17.9 / 21.2 at 16 rows, 20.0 / 25.3 at 32, 22.4 / 25.4 at 64.
// The host knows the average only: 127 single tokens and a chunk of 385 rows (16/4
// heads, behind 4,000) take 220 us with few rows, one row more 236 with tiles, and 214
// in a call each.
canopy_attend_plan_t attend_plan(int N, int B, int HQ, int HKV, int bf16, int d) {
    if (!bf16) return CANOPY_ATTEND_PLAN_FP32;
    const int g = HQ / HKV;
    return g <= 16 && int64_t(N) * g <= int64_t(16) * B ? CANOPY_ATTEND_PLAN_FEW : CANOPY_ATTEND_PLAN_TILES;
}

cudaError_t launch_attend(const void* q, int bf16, const void* kc, const void* vc, const int32_t* table, int pages,
                          int log_page, int max_pages, const int32_t* context, const int32_t* starts,
                          const int32_t* parent, const int32_t* lengths, int N, int B, int HQ, int HKV, int d,
                          int window, int sinks, float scale, void* o, void* workspace, cudaStream_t st) {
    using namespace att;
    Args a;
    a.q = q;
    a.kc = kc;
    a.vc = vc;
    a.o = o;
    a.table = table;
    a.context = context;
    a.starts = starts;
    a.parent = parent;
    a.lengths = lengths;
    a.N = N;
    a.B = B;
    a.T = starts ? N : N / B;
    a.HQ = HQ;
    a.HKV = HKV;
    a.g = HQ / HKV;
    a.pages = pages;
    a.log_page = log_page;
    a.max_pages = max_pages;
    a.window = window > 0 ? window : kNoWindow;
    a.sinks = sinks;
    a.scale2 = scale * 1.4426950408889634f;
    const canopy_attend_plan_t plan = attend_plan(N, B, HQ, HKV, bf16, d);
    const bool tiles = plan == CANOPY_ATTEND_PLAN_TILES, few = plan == CANOPY_ATTEND_PLAN_FEW;
    const int R = a.g <= 16 && int64_t(N) * a.g <= int64_t(16) * B ? 16 : 64;  // rows of a tile, where not on 256
    a.rt = tiles ? tc_tile_tokens(a.g) : R / a.g;
    a.kt = tiles ? tc_tile_keys(d) : 64;
    a.least = bf16 ? kLeast : 1;  // (a unit takes the CUDA cores 3 us)
    // no more CTAs than the units that the page table has room for, were every tile's cache full
    const int64_t most_tiles = N / a.rt + B < N ? N / a.rt + B : N, room = int64_t(max_pages) << log_page;
    const int64_t units = most_tiles * HKV * (room / a.kt + 1) / a.least, ctas = tiles ? kSMs : kFewCtas;
    a.ctas = int(units < ctas ? (units < 1 ? 1 : units) : ctas);
    a.slot_rows = few ? 16 : tiles ? slot_rows(N, a.g) : R;
    const Layout w = layout(N, B, a.g, d);
    char* p = static_cast<char*>(workspace);
    a.err = reinterpret_cast<int32_t*>(p);
    a.seqs = reinterpret_cast<int4*>(p + w.seqs);
    a.line = reinterpret_cast<int64_t*>(p + w.line);
    a.first_tile = reinterpret_cast<int2*>(p + w.first_tile);
    a.joins = reinterpret_cast<int4*>(p + w.joins);
    a.mask = reinterpret_cast<uint32_t*>(p + w.mask);
    a.depth = reinterpret_cast<int32_t*>(p + w.depth);
    a.part = reinterpret_cast<float*>(p + w.part);
    cudaError_t e = cudaSuccess;
    if (!few || parent || !few_plans(N, B)) e = launch_pdl(plan_kernel, dim3(parent ? B + 1 : 1), dim3(256), 0, st, a);
    if (e != cudaSuccess) return e;
    if (tiles) return launch_tc(a, d, st);
    if (few) {
        e = launch_few(a, d, st);
        return e != cudaSuccess ? e : launch_join_bf16(a, d, st);
    }
    if (d == 128) {
        e = R == 16 ? simt::launch<128, 16>(a, st) : simt::launch<128, 64>(a, st);
        return e != cudaSuccess ? e : launch_join_rows<float, 128>(a, st);
    }
    e = R == 16 ? simt::launch<64, 16>(a, st) : simt::launch<64, 64>(a, st);
    return e != cudaSuccess ? e : launch_join_rows<float, 64>(a, st);
}

}  // namespace canopy
