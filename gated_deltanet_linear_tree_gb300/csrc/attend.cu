// Attention of new rows over a paged cache: the plan, the trees' masks, and the
// fp32 path on CUDA cores.
//
// For row i: o_i = sum_j p_ij v_j / sum_j p_ij, p_ij = 2^(s_ij - m_i), s_ij =
// scale log2(e) q_i.k_j over the keys that i sees, m_i the running maximum.
#include "attend.cuh"

namespace canopy {
namespace att {

// Block 0 plans; block 1 + b, with trees, lists the paths of stream b.
__global__ void __launch_bounds__(256) plan_kernel(Args a, int least) {
    pdl_wait();
    if (blockIdx.x == 0) {
        int bad = 0;
        const int ntiles = make_plan<256>(a, &bad);
        if (bad) raise_err(a.err, bad);
        const int64_t units = a.line[ntiles];
        const int ctas = parts(a, units, least);
        if (threadIdx.x == 0) *a.total = ntiles;
        for (int c = threadIdx.x; c < ctas; c += 256)
            a.first_tile[c] = ntiles ? tile_at(a.line, ntiles, cta_begin(units, ctas, c)) : 0;
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
// CUDA cores.  256 threads on R rows x 64 keys: thread (ty, tx) forms the
// scores of R / 16 rows with keys tx + 16 j, and D / 16 columns of those rows'
// outputs; a row's statistics stay with its 16 threads.
namespace simt {

constexpr int KT = 64, NT = 256;

template <int D, int R>
struct Smem {
    static constexpr int LD = D + 4, LP = KT + 4;  // float4 reads of neighbouring rows on other banks
    float q[R * LD], k[KT * LD], v[KT * LD], p[R * LP];
    int last;
};

template <typename InT>
__device__ inline float4 load_row4(const void* cache, const Args& a, const Tile& tile, int h, int D, int key, int c,
                                   int& bad) {
    if (!in_reach(tile, key)) return make_float4(0.f, 0.f, 0.f, 0.f);
    const int page = a.table[size_t(tile.b) * a.max_pages + (key >> a.log_page)];
    if (page < 0 || page >= a.pages) {
        bad = CANOPY_DEVERR_PAGE;
        return make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const size_t row = ((size_t(page) * a.HKV + h) << a.log_page) + (key & ((1 << a.log_page) - 1));
    return load4(static_cast<const InT*>(cache) + row * D + c);
}

template <typename InT, int D, int R>
__global__ void __launch_bounds__(NT) attend_kernel(const Args a, int least) {
    constexpr int RR = R / 16, C4 = D / 64, LD = Smem<D, R>::LD, LP = Smem<D, R>::LP;
    extern __shared__ __align__(16) uint8_t raw[];
    Smem<D, R>& sm = *reinterpret_cast<Smem<D, R>*>(raw);
    pdl_wait();
    const int ntiles = *a.total;
    const int64_t units = a.line[ntiles];
    const int ctas = parts(a, units, least);
    if (int(blockIdx.x) >= ctas || ntiles == 0) return;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    Walk walk{units, cta_begin(units, ctas, blockIdx.x), cta_begin(units, ctas, blockIdx.x + 1), ctas,
              a.first_tile[blockIdx.x]};
    int bad = 0;
    Piece p;
    while (walk.next(a, p)) {
        const Tile& tile = p.tile;
        const int rows = tile.ntok * a.g;
        __syncthreads();
        for (int e = tid; e < R * (D / 4); e += NT) {
            const int r = e / (D / 4), c = 4 * (e % (D / 4));
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows)
                x = load4(static_cast<const InT*>(a.q) +
                          (size_t(tile.row + r / a.g) * a.HQ + p.h * a.g + r % a.g) * D + c);
            *reinterpret_cast<float4*>(sm.q + r * LD + c) = x;
        }
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
            const int key0 = key_tile(tile, u) * KT;
            __syncthreads();
            for (int e = tid; e < KT * (D / 4); e += NT) {
                const int j = e / (D / 4), c = 4 * (e % (D / 4));
                *reinterpret_cast<float4*>(sm.k + j * LD + c) = load_row4<InT>(a.kc, a, tile, p.h, D, key0 + j, c, bad);
                *reinterpret_cast<float4*>(sm.v + j * LD + c) = load_row4<InT>(a.vc, a, tile, p.h, D, key0 + j, c, bad);
            }
            __syncthreads();
            float s[RR][4] = {};
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                float4 k4[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) k4[j] = *reinterpret_cast<const float4*>(sm.k + (tx + 16 * j) * LD + c);
#pragma unroll
                for (int r = 0; r < RR; ++r) {
                    const float4 x = *reinterpret_cast<const float4*>(sm.q + (ty * RR + r) * LD + c);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[r][j] += x.x * k4[j].x + x.y * k4[j].y + x.z * k4[j].z + x.w * k4[j].w;
                }
            }
            const bool all = all_see(a, tile, key0, KT);
#pragma unroll
            for (int r = 0; r < RR; ++r) {
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[r][j] *= a.scale2;
                    if (!all && !sees(a, tile, depth[r], mask[r], key0 + tx + 16 * j)) s[r][j] = -INFINITY;
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
            for (int j = 0; j < KT; ++j) {
                float4 v4[C4];
#pragma unroll
                for (int c = 0; c < C4; ++c)
                    v4[c] = *reinterpret_cast<const float4*>(sm.v + j * LD + 4 * tx + 64 * c);
#pragma unroll
                for (int r = 0; r < RR; ++r) {
                    const float w = sm.p[(ty * RR + r) * LP + j];
                    if (!all && w == 0.f) continue;  // what a row does not see does not reach it, whatever it holds
#pragma unroll
                    for (int c = 0; c < C4; ++c) {
                        o[r][c].x += w * v4[c].x;
                        o[r][c].y += w * v4[c].y;
                        o[r][c].z += w * v4[c].z;
                        o[r][c].w += w * v4[c].w;
                    }
                }
            }
        }
#pragma unroll
        for (int r = 0; r < RR; ++r)
#pragma unroll
            for (int x = 8; x; x >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
        if (p.pieces > 1) {
            const size_t SLOT = size_t(a.slot_rows) * (D + 2);
            float* out = a.part + p.slot * SLOT;
#pragma unroll
            for (int r = 0; r < RR; ++r) {
                const int row = ty * RR + r;
#pragma unroll
                for (int c = 0; c < C4; ++c)
                    *reinterpret_cast<float4*>(out + row * D + 4 * tx + 64 * c) = o[r][c];
                if (tx == 0) {
                    out[R * D + row] = m[r];
                    out[R * D + R + row] = l[r];
                }
            }
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const int before = atomicAdd(a.done + p.first, 1);
                sm.last = before == p.pieces - 1;
                if (sm.last) a.done[p.first] = 0;
            }
            __syncthreads();
            if (!sm.last) continue;
            __threadfence();
#pragma unroll
            for (int r = 0; r < RR; ++r) {
                const int row = ty * RR + r;
                float top = -INFINITY;
                for (int i = 0; i < p.pieces; ++i)
                    top = fmaxf(top, __ldcg(a.part + slot_of(p.first, i) * SLOT + R * D + row));
                const float base = top == -INFINITY ? 0.f : top;
                l[r] = 0.f;
#pragma unroll
                for (int c = 0; c < C4; ++c) o[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int i = 0; i < p.pieces; ++i) {
                    const float* in = a.part + slot_of(p.first, i) * SLOT;
                    const float w = exp2f(__ldcg(in + R * D + row) - base);
                    l[r] += w * __ldcg(in + R * D + R + row);
#pragma unroll
                    for (int c = 0; c < C4; ++c) {
                        const float4 x = __ldcg(reinterpret_cast<const float4*>(in + row * D + 4 * tx + 64 * c));
                        o[r][c].x += w * x.x;
                        o[r][c].y += w * x.y;
                        o[r][c].z += w * x.z;
                        o[r][c].w += w * x.w;
                    }
                }
            }
        }
#pragma unroll
        for (int r = 0; r < RR; ++r) {
            const int row = ty * RR + r;
            if (row >= rows) continue;
            const float f = l[r] == 0.f ? 0.f : 1.f / l[r];
            InT* out = static_cast<InT*>(a.o) + (size_t(tile.row + row / a.g) * a.HQ + p.h * a.g + row % a.g) * D;
#pragma unroll
            for (int c = 0; c < C4; ++c) {
                store_out(out + 4 * tx + 64 * c, o[r][c].x * f);
                store_out(out + 4 * tx + 64 * c + 1, o[r][c].y * f);
                store_out(out + 4 * tx + 64 * c + 2, o[r][c].z * f);
                store_out(out + 4 * tx + 64 * c + 3, o[r][c].w * f);
            }
        }
    }
    if (bad) raise_err(a.err, bad);
}

template <typename InT, int D, int R>
cudaError_t launch(const Args& a, int least, cudaStream_t st) {
    static OncePerDevice once;
    const auto kernel = attend_kernel<InT, D, R>;
    cudaError_t e = once([&] { return allow_smem(kernel, int(sizeof(Smem<D, R>))); });
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(a.ctas), dim3(NT), sizeof(Smem<D, R>), st, a, least);
}

}  // namespace simt

// ---------------------------------------------------------------------------

int tc_tile_tokens(int g);
cudaError_t launch_tc(const Args& a, int d, int least, cudaStream_t st);

namespace {

constexpr int kCtas = 152;  // one on every SM
constexpr int kLeast = 2;      // units of a part

// Rows of an unfinished piece: those of the largest row tile that a call takes.
int slot_rows(int N, int g) {
    const int64_t rows = int64_t(N) * g;
    return rows <= 16 ? 16 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256;
}

struct Layout {
    size_t seqs, tiles, line, first_tile, total, mask, depth, done, part, end;
};

// For the smallest row tile that a call of these sizes may take.
Layout layout(int N, int B, int g, int d) {
    const size_t max_tiles = size_t(N) + B;
    Layout w;
    size_t o = 256;  // the error word, and the count of tiles behind it
    w.total = 128;
    w.done = o;       o = ws_align(o + 2 * kCtas * 4);
    w.seqs = o;       o = ws_align(o + size_t(B) * sizeof(int4));
    w.tiles = o;      o = ws_align(o + max_tiles * sizeof(Tile));
    w.line = o;       o = ws_align(o + (max_tiles + 1) * 8);
    w.first_tile = o; o = ws_align(o + kCtas * 4);
    w.mask = o;       o = ws_align(o + size_t(N) * kMaskWords * 4);
    w.depth = o;      o = ws_align(o + size_t(N) * 4);
    w.part = o;       o = ws_align(o + size_t(2 * kCtas) * slot_rows(N, g) * (d + 2) * 4);
    w.end = o;
    return w;
}

}  // namespace

}  // namespace att

size_t attend_ws_bytes(int N, int B, int HQ, int HKV, int d) { return att::layout(N, B, HQ / HKV, d).end; }
canopy_attend_plan_t attend_plan(int N, int B, int HQ, int HKV, int bf16, int d) {
    if (!bf16) return CANOPY_ATTEND_PLAN_FP32;
    return CANOPY_ATTEND_PLAN_TILES;
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
    const int R = size_t(N) * a.g <= size_t(16) * B && a.g <= 16 ? 16 : 64;
    a.rt = plan == CANOPY_ATTEND_PLAN_TILES ? tc_tile_tokens(a.g) : R / a.g;
    a.log_kt = plan == CANOPY_ATTEND_PLAN_TILES ? 7 : 6;
    a.ctas = kCtas;
    a.max_tiles = N + B;
    a.slot_rows = slot_rows(N, a.g);
    const Layout w = layout(N, B, a.g, d);
    char* p = static_cast<char*>(workspace);
    a.err = reinterpret_cast<int32_t*>(p);
    a.total = reinterpret_cast<int*>(p + w.total);
    a.done = reinterpret_cast<int32_t*>(p + w.done);
    a.seqs = reinterpret_cast<int4*>(p + w.seqs);
    a.tiles = reinterpret_cast<Tile*>(p + w.tiles);
    a.line = reinterpret_cast<int64_t*>(p + w.line);
    a.first_tile = reinterpret_cast<int*>(p + w.first_tile);
    a.mask = reinterpret_cast<uint32_t*>(p + w.mask);
    a.depth = reinterpret_cast<int32_t*>(p + w.depth);
    a.part = reinterpret_cast<float*>(p + w.part);
    cudaError_t e = launch_pdl(plan_kernel, dim3(parent ? B + 1 : 1), dim3(256), 0, st, a, kLeast);
    if (e != cudaSuccess) return e;
    if (plan == CANOPY_ATTEND_PLAN_TILES) return launch_tc(a, d, kLeast, st);
    if (d == 128)
        return R == 16 ? simt::launch<float, 128, 16>(a, kLeast, st) : simt::launch<float, 128, 64>(a, kLeast, st);
    return R == 16 ? simt::launch<float, 64, 16>(a, kLeast, st) : simt::launch<float, 64, 64>(a, kLeast, st);
}

}  // namespace canopy
