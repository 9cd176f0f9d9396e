// Attention of few rows over a paged cache (bf16): the next token of every
// stream, or a few tokens of each.
//
// Bound by the reads of K and V: 16 rows (tokens by the g query heads of a key
// head) against a key take 4 d operations for each of its 4 d bytes and row, an
// eighth of what the tensor cores would do meanwhile.  So nothing is gained
// from 128-row products; the rows stay in registers as 16-row operands of warp
// products (mma m16n8k16), whose scores come out as the operand that the second
// product takes.  A CTA of two such warps, 32 keys of each unit of 64 to either,
// and one that loads: three stages of K and V tiles by TMA, one box per page and
// 64 columns.  Two CTAs an SM, 192 KB of reads in flight.
//
// 64 streams behind 4,000 to 16,000 tokens, 32/8 heads: 394 to 399 us, 6.7 TB/s, 0.98
// of the measured copy bandwidth (128-row products in attend_tc.cu: 492).  One behind
// 262,143 tokens, 16/2 heads: 44 us, 0.9 of it, and 10 for the launch that joins the
// pieces.  One behind 700: two launches' latencies, 10.8 us.
//
// The running maximum is kept until it grows by 2^8 (attend_tc.cu), and the two
// warps keep one each until the piece ends, when the second's sums join the
// first's.
#include "attend.cuh"

namespace canopy {
namespace att {
namespace few {

constexpr int KT = 64, NT = 96;
// Up to these sizes every CTA makes the plan for itself: what shared memory has room for.  Measured against a launch
// that plans, us: one stream behind 100 tokens 7.9 / 9.7, 32 10.0 / 12.8, 128 21.6 / 24.9; behind 2,000 9.5 / 11.7,
// 34 / 38 and 96 / 99 (16/4 heads).
constexpr int kPlanSeqs = 128, kPlanTiles = 256;

template <int D>
struct Smem {
    static constexpr int STAGES = D == 128 ? 3 : 6;
    static constexpr int TILE = KT * D * 2;  // K or V: [d / 64][64 keys][128 bytes]
    uint8_t kv[STAGES][2][TILE];
    float other[16][D + 4];  // the second warp's sums (rows on other banks)
    float other_m[16], other_l[16];
    uint32_t other_left;  // rows of which its products left out a value that they see
    int4 seqs[kPlanSeqs + 1];
    int64_t line[kPlanTiles + 1];
    uint64_t full[STAGES], empty[STAGES], given, taken;
};
static_assert(2 * (sizeof(Smem<128>) + 2048) <= 233472 && 2 * (sizeof(Smem<64>) + 2048) <= 233472, "shared memory");

__device__ inline void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ inline void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// c += a b, a 16 x 16 (rows x k), b 16 x 8, bf16 with fp32 sums.
__device__ inline void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Keeps of a pair of values (two keys of one column) those with a bit.
__device__ inline uint32_t keep_pair(uint32_t x, uint32_t bits) {
    return x & ((bits & 1 ? 0x0000FFFFu : 0u) | (bits & 2 ? 0xFFFF0000u : 0u));
}

template <int D>
__global__ void __launch_bounds__(NT, 2)
    attend_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV, const Args a,
                  int plans) {
    constexpr int HALVES = D / 64, STAGES = Smem<D>::STAGES;
    extern __shared__ uint8_t raw[];
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw + ((1024 - (smem_u32(raw) & 1023)) & 1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 64) {
        prefetch_map(&mapK);
        prefetch_map(&mapV);
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(sm.full + i, 1);
            mbar_init(sm.empty + i, 2);
        }
        mbar_init(&sm.given, 32);
        mbar_init(&sm.taken, 32);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();  // after the wait: the next launch may rely on everything before this one
    const int4* seqs = a.seqs;
    const int64_t* line = a.line;
    if (plans) {
        int bad = 0;
        const int ntiles = make_plan<NT>(a, sm.seqs, sm.line, &bad);
        seqs = sm.seqs;
        line = sm.line;
        if (blockIdx.x == 0) {  // for the launch that joins the pieces
            if (bad) raise_err(a.err, bad);
            for (int i = threadIdx.x; i <= a.B; i += NT) a.seqs[i] = seqs[i];
            for (int i = threadIdx.x; i <= ntiles; i += NT) a.line[i] = line[i];
        }
    }
    __syncthreads();
    Walk walk(a, seqs, line, blockIdx.x, plans ? nullptr : a.first_tile);
    bool ok = true;
    Piece p;
    Ring<STAGES> ring;

    if (warp == 2) {
        // ---- loads -------------------------------------------------------------------
        const int box = min(1 << a.log_page, KT), boxes = KT / box;
        const int i = lane / (2 * HALVES), kv = lane / HALVES % 2, part = lane % HALVES;  // a lane's box
        int bad = 0, loads = 0;
        while (ok && walk.next(a, p)) {
            const Tile& tile = p.tile;
            for (int u = p.u0; u < p.u1; ++u) {
                const int key = key_tile(tile, u) * KT + i * box;
                int z = a.pages * a.HKV;  // outside: zeros
                if (i < boxes && (key < tile.sink_end || (key + box > tile.near && key < tile.hi))) {
                    const int page = a.table[size_t(tile.b) * a.max_pages + (key >> a.log_page)];
                    if (page < 0 || page >= a.pages) bad = CANOPY_DEVERR_PAGE;
                    else z = page * a.HKV + p.h;
                }
                ok = warp_wait(sm.empty + ring.at, ring.phase ^ 1);
                if (!ok) break;
                ++loads;
                if (lane == 0) mbar_expect_tx(sm.full + ring.at, 2 * Smem<D>::TILE);
                __syncwarp();
                if (i < boxes)
                    tma_load_3d(sm.kv[ring.at][kv] + part * (KT * 128) + i * box * 128, kv ? &mapV : &mapK,
                                sm.full + ring.at, 64 * part, key & ((1 << a.log_page) - 1), z);
                ring.step();
            }
        }
        if (bad) raise_err(a.err, bad);
        // no copy is left in flight, should another warp have given up
        for (int n = min(loads, STAGES); n > 0; --n) {
            ring.back();
            warp_wait(sm.full + ring.at, ring.phase);
        }
    } else {
        // ---- scores, softmax, sums -----------------------------------------------------
        Phase given, taken;
        bool first_piece = true;
        const int r0 = lane >> 2, c0 = 2 * (lane & 3);  // rows r0 and r0 + 8, columns c0, c0 + 1 of every 8
        while (ok && walk.next(a, p)) {
            const Tile& tile = p.tile;
            const int rows = tile.ntok * a.g;
            uint32_t q[D / 16][4];
            int depth[2];
            const uint32_t* mask[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = r0 + 8 * x, i = min(r / a.g, tile.ntok - 1);
                const bool valid = r < rows;
                depth[x] = a.parent ? a.depth[tile.row + i] : tile.t0 + i;
                mask[x] = a.parent ? a.mask + size_t(tile.row + i) * kMaskWords : nullptr;
                const uint32_t* in = reinterpret_cast<const uint32_t*>(
                    static_cast<const __nv_bfloat16*>(a.q) +
                    (size_t(tile.row + i) * a.HQ + p.h * a.g + (valid ? r % a.g : 0)) * D + c0);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    q[k][x] = valid ? __ldg(in + 8 * k) : 0u;
                    q[k][x + 2] = valid ? __ldg(in + 8 * k + 4) : 0u;
                }
            }
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[D / 8][4];
            uint32_t left_out = 0;  // which of the 16 rows see a value that their products leave out
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
            for (int u = p.u0; u < p.u1; ++u) {
                const int kt = key_tile(tile, u), key = kt * KT + 32 * warp;  // this warp's 32 keys
                ok = warp_wait(sm.full + ring.at, ring.phase);
                if (!ok) break;
                const uint32_t K = smem_u32(sm.kv[ring.at][0]), V = smem_u32(sm.kv[ring.at][1]);
                float s[4][4] = {};
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        // keys 16 n .. + 15 (by 8), columns 16 k .. + 15 (by 8)
                        const int row = 32 * warp + 16 * n + (lane & 7) + ((lane >> 4) << 3);
                        const int chunk = (2 * k + ((lane >> 3) & 1)) & 7;
                        uint32_t b[4];
                        ldmatrix4(K + (k >> 2) * (KT * 128) + row * 128 + ((chunk ^ (row & 7)) << 4), b);
                        mma16816(s[2 * n], q[k], b[0], b[1]);
                        mma16816(s[2 * n + 1], q[k], b[2], b[3]);
                    }
                const bool all = all_see(tile, kt);
                uint32_t keep = 0xFFFFFFFFu, check = 0;  // keys that some row sees; those that some but not all see
                uint32_t seen[2] = {keep, keep};
                if (!all) {
                    uint32_t every = 0xFFFFFFFFu;
                    keep = 0;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const bool valid = r0 + 8 * x < rows;
                        seen[x] = valid ? seen_bits(a, tile, depth[x], mask[x], key) : 0u;
                        keep |= seen[x];
                        if (valid) every &= seen[x];
#pragma unroll
                        for (int n = 0; n < 4; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (!((seen[x] >> (8 * n + c0 + e)) & 1u)) s[n][2 * x + e] = -INFINITY;
                    }
                    keep = __reduce_or_sync(0xffffffffu, keep);
                    check = keep & ~__reduce_and_sync(0xffffffffu, every);
                }
                float base[2];
                bool grow = false;
                float f[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float t = -INFINITY;
#pragma unroll
                    for (int n = 0; n < 4; ++n) t = fmaxf(t, fmaxf(s[n][2 * x], s[n][2 * x + 1]));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                    t = a.scale2 * fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                    f[x] = 1.f;
                    if (t > m[x] + kGrow) {
                        f[x] = exp2_approx(m[x] - t);
                        m[x] = t;
                        grow = true;
                    }
                    base[x] = m[x] == -INFINITY ? 0.f : m[x];
                }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        l[x] *= f[x];
#pragma unroll
                        for (int n = 0; n < D / 8; ++n) {
                            o[n][2 * x] *= f[x];
                            o[n][2 * x + 1] *= f[x];
                        }
                    }
                }
                uint32_t w[2][4];  // the weights, as rows x 16 keys operands
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float y = exp2_approx(fmaf(s[n][2 * x], a.scale2, -base[x]));
                        const float z = exp2_approx(fmaf(s[n][2 * x + 1], a.scale2, -base[x]));
                        l[x] += y + z;
                        w[n >> 1][2 * (n & 1) + x] = pack_bf16(y, z);
                    }
                if (check) {  // values that are not finite, where not every row sees every key
                    uint32_t bad = 0;
                    for (int e = lane; e < 32 * D / 2; e += 32) {
                        const int j = e / (D / 2), c = e % (D / 2);
                        // (the order of a row's chunks does not matter)
                        uint32_t& x = reinterpret_cast<uint32_t*>(
                            sm.kv[ring.at][1])[(c / 32) * (KT * 32) + (32 * warp + j) * 32 + (c & 31)];
                        if (!finite_pair(x)) {
                            bad |= 1u << j;
                            x = finite_part(x);
                        }
                    }
                    bad = __reduce_or_sync(0xffffffffu, bad) & keep;
                    if (bad & seen[0]) left_out |= 1u << r0;
                    if (bad & seen[1]) left_out |= 1u << (r0 + 8);
                    fence_proxy_async_smem();  // (before the stage's next load)
                    __syncwarp();
                }
#pragma unroll
                for (int n = 0; n < D / 16; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        // keys 16 k .. + 15 (by 8), columns 16 n .. + 15 (by 8)
                        const int row = 32 * warp + 16 * k + (lane & 15);
                        const int chunk = (2 * n + (lane >> 4)) & 7;
                        uint32_t b[4];
                        ldmatrix4_trans(V + (n >> 2) * (KT * 128) + row * 128 + ((chunk ^ (row & 7)) << 4), b);
                        if (!all) {
                            const uint32_t lo = keep >> (16 * k + c0), hi = keep >> (16 * k + 8 + c0);
                            b[0] = keep_pair(b[0], lo);
                            b[1] = keep_pair(b[1], hi);
                            b[2] = keep_pair(b[2], lo);
                            b[3] = keep_pair(b[3], hi);
                        }
                        mma16816(o[2 * n], w[k], b[0], b[1]);
                        mma16816(o[2 * n + 1], w[k], b[2], b[3]);
                    }
                __syncwarp();
                if (lane == 0) mbar_arrive(sm.empty + ring.at);
                ring.step();
            }
            if (!ok) break;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
                l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
            }
            if (warp == 1) {
                if (!first_piece) ok = taken.wait(&sm.taken);
                first_piece = false;
                if (!ok) break;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
                        *reinterpret_cast<float2*>(&sm.other[r0 + 8 * x][8 * n + c0]) =
                            make_float2(o[n][2 * x], o[n][2 * x + 1]);
                    if (c0 == 0) {
                        sm.other_m[r0 + 8 * x] = m[x];
                        sm.other_l[r0 + 8 * x] = l[x];
                    }
                }
                left_out = __reduce_or_sync(0xffffffffu, left_out);
                if (lane == 0) sm.other_left = left_out;
                mbar_arrive(&sm.given);
                continue;
            }
            ok = given.wait(&sm.given);
            if (!ok) break;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = r0 + 8 * x;
                const float om = sm.other_m[r], top = fmaxf(m[x], om), base = top == -INFINITY ? 0.f : top;
                float mine = exp2_approx(m[x] - base), other = exp2_approx(om - base);
                l[x] = mine * l[x] + other * sm.other_l[r];
                if (r >= rows) continue;
                if (p.whole) {
                    const float inv = l[x] == 0.f ? 0.f : 1.f / l[x];
                    mine *= inv;
                    other *= inv;
                    uint32_t* out = reinterpret_cast<uint32_t*>(
                        static_cast<__nv_bfloat16*>(a.o) +
                        (size_t(tile.row + r / a.g) * a.HQ + p.h * a.g + r % a.g) * D + c0);
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        const float2 y = *reinterpret_cast<const float2*>(&sm.other[r][8 * n + c0]);
                        out[4 * n] = pack_bf16(mine * o[n][2 * x] + other * y.x, mine * o[n][2 * x + 1] + other * y.y);
                    }
                } else {
                    float* slot = a.part + size_t(p.slot) * 16 * (D + 2);
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        const float2 y = *reinterpret_cast<const float2*>(&sm.other[r][8 * n + c0]);
                        *reinterpret_cast<float2*>(slot + r * D + 8 * n + c0) =
                            make_float2(mine * o[n][2 * x] + other * y.x, mine * o[n][2 * x + 1] + other * y.y);
                    }
                    if (c0 == 0) {
                        slot[16 * D + r] = top;
                        slot[16 * D + 16 + r] = l[x];
                    }
                }
            }
            left_out |= sm.other_left;
            if (left_out)
#pragma unroll 1
                for (int x = 0; x < 2; ++x) {
                    const int r = r0 + 8 * x;
                    if (!((left_out >> r) & 1u)) continue;
                    uint32_t* out = reinterpret_cast<uint32_t*>(
                        static_cast<__nv_bfloat16*>(a.o) +
                        (size_t(tile.row + r / a.g) * a.HQ + p.h * a.g + r % a.g) * D);
                    float* sum = a.part + size_t(p.slot) * 16 * (D + 2) + r * D;
                    const auto add = [&](int c, float y, float z) {
                        if (p.whole) {
                            out[c] = pack_bf16(first_of(out[c]) + y, second_of(out[c]) + z);
                        } else {
                            sum[2 * c] += y;
                            sum[2 * c + 1] += z;
                        }
                    };
                    add_not_finite<uint32_t>(a, p, x ? depth[1] : depth[0], x ? mask[1] : mask[0], D, c0 / 2, 4, add);
                }
            mbar_arrive(&sm.taken);
        }
    }
    if (!ok && lane == 0) raise_err(a.err, CANOPY_DEVERR_TIMEOUT);
}

}  // namespace few

bool few_plans(int N, int B) { return B <= few::kPlanSeqs && int64_t(N) + B <= few::kPlanTiles; }

template <int D>
static cudaError_t launch_few_d(const Args& a, cudaStream_t st) {
    CUtensorMap mk, mv;
    const uint64_t row = D * 2, page = uint64_t(1) << a.log_page;
    const uint32_t keys = uint32_t(page < few::KT ? page : few::KT);
    if (!make_bf16_box_map(&mk, a.kc, {D, page, uint64_t(a.pages) * a.HKV}, {row, page * row}, {64, keys, 1}) ||
        !make_bf16_box_map(&mv, a.vc, {D, page, uint64_t(a.pages) * a.HKV}, {row, page * row}, {64, keys, 1}))
        return cudaErrorInvalidValue;
    const int smem = int(sizeof(few::Smem<D>)) + 1024;
    static OncePerDevice once;
    const cudaError_t e = once([=] { return allow_smem(few::attend_kernel<D>, smem); });
    if (e != cudaSuccess) return e;
    return launch_pdl(few::attend_kernel<D>, dim3(a.ctas), dim3(few::NT), smem, st, mk, mv, a,
                      int(!a.parent && few_plans(a.N, a.B)));
}

cudaError_t launch_few(const Args& a, int d, cudaStream_t st) {
    return d == 128 ? launch_few_d<128>(a, st) : launch_few_d<64>(a, st);
}

}  // namespace att
}  // namespace canopy
