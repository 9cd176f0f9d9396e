// Queries and keys of an attention layer: each head's norm, the rotation by the
// token's position, and keys and values into the cache's pages, in one pass.
//
// Per token and head, with y = w x / sqrt(mean x^2 + eps) (rms), x / sqrt(sum
// x^2 + eps) (unit rows) or x: pair j of the first R columns turns by
// position * freq_j (the position on the frequency's axis),
//     (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin).
// All in fp32, rounded once to the type.  The angle is kept in turns: freq_j /
// 2 pi as a 64-bit binary fraction times the whole position wraps at whole turns
// by itself, so that far positions lose nothing.  (fp64 has a 64th of the fp32 rate:
// with its products 16,383 tokens took 220 us, with whole numbers 166.)
// Sine and cosine are their series about the nearest quarter turn, to the terms
// that are below 2^-25 at an eighth of a turn.
//
// A lane holds four pairs of a head: for pairs (j, j + R/2) two chunks of four
// elements R/2 apart, else eight elements in a row, so that a pair never leaves
// its lane; d / 8 lanes share a head and a warp takes 256 / d heads at a time.  The
// angles serve all heads that a warp takes of one token.
//
// 16,383 tokens, 32/8 heads, three axes, into pages of 16: 82 us, 4.9 TB/s (0.73 of
// the measured copy bandwidth; the reads in flight bound it, at 20 warps an SM and
// 64 bytes a lane: more warps spill, fewer have less in flight); in fp32 137 us, 0.87.
// 1,024 unit rows of 16/16 heads 5.5 us in a graph, 6.8 to 8.3 by calls; one token 2.8
// us in a graph, 5.4 to 6.8 by its call.
#include "common.cuh"

namespace canopy {
namespace qkp {

struct Args {
    const void *q, *k, *v;
    void *qo, *ko, *kc, *vc;
    int64_t ldq, ldk, ldv;        // elements from a token to the next
    int64_t axis_step, row_step;  // of the positions: from an axis, from a token to the next
    const float *qw, *kw, *freqs;
    const int32_t *positions, *axis, *table, *context, *starts, *lengths;
    int32_t* err;
    float eps;
    int norm, R, adjacent, axes;
    int N, T, B, HQ, HKV;
    int pages, log_page, max_pages;
    int chunks, sets;  // warps per token; sets of heads each takes
};

// Four elements in fp32 (two pairs), and back.
struct Four {
    uint64_t lo, hi;
};
__device__ inline Four get4(const float* p) {
    const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(p);
    return {t.x, t.y};
}
__device__ inline Four get4(const __nv_bfloat16* p) {
    const uint2 t = *reinterpret_cast<const uint2*>(p);
    return {pack2(__uint_as_float(t.x << 16), __uint_as_float(t.x & 0xFFFF0000u)),
            pack2(__uint_as_float(t.y << 16), __uint_as_float(t.y & 0xFFFF0000u))};
}
__device__ inline void put4(float* p, const Four& x) {
    *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(x.lo, x.hi);
}
__device__ inline void put4(__nv_bfloat16* p, const Four& x) {
    float a, b, c, d;
    unpack2(x.lo, a, b);
    unpack2(x.hi, c, d);
    const __nv_bfloat162 y = __floats2bfloat162_rn(a, b), z = __floats2bfloat162_rn(c, d);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&y), *reinterpret_cast<const uint32_t*>(&z));
}
__device__ inline Four operator*(const Four& a, const Four& b) { return {mul2(a.lo, b.lo), mul2(a.hi, b.hi)}; }
__device__ inline Four fma4(const Four& a, const Four& b, const Four& c) {
    return {fma2(a.lo, b.lo, c.lo), fma2(a.hi, b.hi, c.hi)};
}
__device__ inline float sum4(const Four& x) {
    float a, b;
    unpack2(add2(x.lo, x.hi), a, b);
    return a + b;
}

// The sequence that token n belongs to (-1: none) and its index there; for a
// whole warp.
__device__ inline int sequence_of(const Args& a, int n, int& i, int* bad) {
    int b, lo, len;
    if (!a.starts) {
        b = n / a.T;
        lo = b * a.T;
    } else {
        // the first start beyond n; those before it, brought into range, have the largest as the sequence's own
        int first = a.B + 1;
        lo = 0;
        for (int s0 = 0; s0 <= a.B; s0 += 32) {
            const int s = s0 + int(threadIdx.x & 31);
            const int at = s <= a.B ? start_in_range(a.starts, s, a.N) : a.N;
            const uint32_t beyond = __ballot_sync(0xffffffffu, s <= a.B && at > n);
            const uint32_t mine = beyond ? (1u << (__ffs(beyond) - 1)) - 1 : 0xffffffffu;
            const int here = ((mine >> (threadIdx.x & 31)) & 1u) && s <= a.B ? at : 0;
            lo = max(lo, __reduce_max_sync(0xffffffffu, here));
            if (beyond) {
                first = s0 + __ffs(beyond) - 1;
                break;
            }
        }
        b = first - 1;
        if (b < 0 || b >= a.B) return -1;
        if (a.starts[b] != lo) *bad |= CANOPY_DEVERR_LENGTH;
    }
    i = n - lo;
    if (a.lengths) {
        len = a.lengths[b];
        if (len < 0 || len > a.T) *bad |= CANOPY_DEVERR_LENGTH;
        if (i >= len) return -1;
    }
    return b;
}

// freq / 2 pi as a 64-bit fraction of a turn: the significand, at the top of 64
// bits, times 2^66 / 2 pi, its place given by the exponent.  The product keeps 64
// bits: off by up to 2^-64 of a turn below freq = 2, doubling with every power of
// two above; times a position of 2^31 that is an angle of 2.3e-8 at freq = 64.
__device__ inline uint64_t turns_of(float freq) {
    const uint32_t bits = __float_as_uint(freq);
    const int exponent = int((bits >> 23) & 255) - 150;  // freq = significand * 2^exponent
    const uint64_t significand = (bits & 0x7FFFFFu) | 0x800000u;
    const uint64_t hi = __umul64hi(significand << 40, 0xA2F9836E4E44152Aull);  // significand * 2^42 / 2 pi
    const int left = exponent + 22;
    const uint64_t turns = left >= 64 || left <= -64 ? 0 : left >= 0 ? hi << left : hi >> -left;
    return bits >> 31 ? 0 - turns : turns;
}
// cos and sin of `position` times a frequency.
__device__ inline void turn(int position, uint64_t turns, float& c, float& s) {
    const uint32_t top = uint32_t((turns * uint64_t(int64_t(position)) + 0x80000000ull) >> 32);
    const uint32_t quarter = (top + 0x20000000u) >> 30;
    const float x = float(int32_t(top - (quarter << 30))) * 1.4629180792671596e-9f;  // 2 pi / 2^32
    const float y = x * x;
    const float si = x * fmaf(y, fmaf(y, fmaf(y, fmaf(y, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), 1.f);
    const float co = fmaf(y, fmaf(y, fmaf(y, fmaf(y, 1.f / 40320, -1.f / 720), 1.f / 24), -0.5f), 1.f);
    c = quarter & 1 ? si : co;
    s = quarter & 1 ? co : si;
    if ((quarter + 1) & 2) c = -c;
    if (quarter & 2) s = -s;
}

// A lane's columns of a head, and what it does to them.
template <int D>
struct Lane {
    static constexpr int LANES = D / 8, HEADS = 32 / LANES;  // lanes a head, heads of a set
    int sub, l, oa, ob;                                      // which head of a set, which lane of it; two columns
    bool turned, split;
    uint64_t turns[4];
    int axis[4];
    Four co, si, minus;  // cosines, sines and their negatives of the lane's pairs

    __device__ explicit Lane(const Args& a) {
        const int lane = threadIdx.x & 31;
        l = lane % LANES;
        sub = lane / LANES;
        turned = 8 * l < a.R;
        split = !a.adjacent && turned;
        oa = split ? 4 * l : 8 * l;
        ob = split ? oa + a.R / 2 : oa + 4;
        if (turned)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                turns[j] = turns_of(a.freqs[4 * l + j]);
                axis[j] = a.axis ? min(max(a.axis[4 * l + j], 0), a.axes - 1) : 0;
            }
    }
    // The angles of token n at place `at` of its stream.
    __device__ void token(const Args& a, int n, int at) {
        if (!turned) return;
        float c[4], s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            turn(a.positions ? a.positions[axis[j] * a.axis_step + n * a.row_step] : at, turns[j], c[j], s[j]);
        co = {pack2(c[0], c[1]), pack2(c[2], c[3])};
        si = {pack2(s[0], s[1]), pack2(s[2], s[3])};
        minus = {pack2(-s[0], -s[1]), pack2(-s[2], -s[3])};
    }
    // Norm and rotation of a head's columns; wx, wy the weights.  (A lane without a head takes part in the sum of
    // none.)
    __device__ void finish(const Args& a, Four& x, Four& y, const Four& wx, const Four& wy) const {
        if (a.norm != CANOPY_NORM_NONE) {
            float ss = sum4(fma4(x, x, y * y));
#pragma unroll
            for (int m = LANES / 2; m; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
            const float r = rsqrtf(fmaf(ss, a.norm == CANOPY_NORM_RMS ? 1.f / D : 1.f, a.eps));
            const Four rr = {pack2(r, r), pack2(r, r)};
            x = x * (rr * wx);
            y = y * (rr * wy);
        }
        if (split) {
            const Four t = x;
            x = fma4(y, minus, x * co);
            y = fma4(t, si, y * co);
        } else if (turned) {  // neighbours: (x0, x1), (x2, x3), (y0, y1), (y2, y3)
            float p0, p1, p2, p3, p4, p5, p6, p7;
            unpack2(x.lo, p0, p1);
            unpack2(x.hi, p2, p3);
            unpack2(y.lo, p4, p5);
            unpack2(y.hi, p6, p7);
            const Four e = {pack2(p0, p2), pack2(p4, p6)}, o = {pack2(p1, p3), pack2(p5, p7)};
            const Four te = fma4(o, minus, e * co), to = fma4(e, si, o * co);
            unpack2(te.lo, p0, p2);
            unpack2(te.hi, p4, p6);
            unpack2(to.lo, p1, p3);
            unpack2(to.hi, p5, p7);
            x = {pack2(p0, p1), pack2(p2, p3)};
            y = {pack2(p4, p5), pack2(p6, p7)};
        }
    }
    __device__ void weights(const float* w, Four& wx, Four& wy) const {
        const uint64_t one = pack2(1.f, 1.f);
        wx = w ? get4(w + oa) : Four{one, one};
        wy = w ? get4(w + ob) : Four{one, one};
    }
};

// Where token n goes: whether it is there at all, its place in its stream (n without a cache), and its row in the
// pages without the head (-1: none).  For a whole warp.
__device__ inline bool place_of(const Args& a, int n, int& at, int64_t& slot) {
    at = n;
    slot = -1;
    if (!a.context) return true;
    int bad = 0, i = 0;
    const int b = sequence_of(a, n, i, &bad);
    if (b >= 0) {
        const int ctx = a.context[b];
        const int64_t pos = int64_t(ctx < 0 ? 0 : ctx) + i;
        at = int(pos < 0x7FFFFFFF ? pos : 0x7FFFFFFF);
        if (ctx < 0) {  // (its first places hold tokens: only the queries go on, from place 0)
            bad |= CANOPY_DEVERR_LENGTH;
        } else {
            const int64_t entry = pos >> a.log_page;
            const int page = entry < a.max_pages ? a.table[int64_t(b) * a.max_pages + entry] : -1;
            if (page < 0 || page >= a.pages)
                bad |= CANOPY_DEVERR_PAGE;
            else
                slot = ((int64_t(page) * a.HKV) << a.log_page) + (pos & ((1 << a.log_page) - 1));
        }
    }
    if (bad && (threadIdx.x & 31) == 0 && a.err) raise_err(a.err, bad);
    return b >= 0;
}

// Few tokens: a warp to every set of heads (queries, keys and values have sets of their own), whose columns are on
// their way while the token's place is looked up.
template <typename T, int D>
__global__ void __launch_bounds__(128) prep_few_kernel(const Args a) {
    pdl_wait();
    pdl_trigger();
    using L = Lane<D>;
    const uint32_t w = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (w >= uint32_t(a.N) * a.sets) return;
    const int n = int(w / a.sets), s = int(w % a.sets);
    const int qsets = (a.HQ + L::HEADS - 1) / L::HEADS, ksets = (a.HKV + L::HEADS - 1) / L::HEADS;
    const bool query = s < qsets, value = s >= qsets + ksets;
    L lane(a);
    const int h = (query ? s : value ? s - qsets - ksets : s - qsets) * L::HEADS + lane.sub;
    const bool there = h < (query ? a.HQ : a.HKV);
    const T* in = query ? static_cast<const T*>(a.q) + n * a.ldq
                        : value ? static_cast<const T*>(a.v) + n * a.ldv : static_cast<const T*>(a.k) + n * a.ldk;
    Four x = {0, 0}, y = {0, 0}, wx, wy;
    if (there) {
        x = get4(in + h * D + lane.oa);
        y = get4(in + h * D + lane.ob);
    }
    lane.weights(query ? a.qw : a.kw, wx, wy);
    int at;
    int64_t slot;
    if (!place_of(a, n, at, slot)) return;
    if (!value) {
        lane.token(a, n, at);
        lane.finish(a, x, y, wx, wy);
    }
    if (!there || (!query && a.kc && slot < 0)) return;
    T* out = query ? static_cast<T*>(a.qo) + (int64_t(n) * a.HQ + h) * D
                   : !a.kc ? static_cast<T*>(a.ko) + (int64_t(n) * a.HKV + h) * D
                           : static_cast<T*>(value ? a.vc : a.kc) + (slot + (int64_t(h) << a.log_page)) * D;
    put4(out + lane.oa, x);
    put4(out + lane.ob, y);
}

// Many tokens: a warp goes from token to token, four sets of heads at a time at constant distances (the addresses
// of one set at a time took half of all instructions).  `chunks` warps share a token, each kind's sets between them.
template <typename T, int D>
__global__ void __launch_bounds__(128, 5) prep_many_kernel(const Args a) {
    pdl_wait();
    pdl_trigger();
    using L = Lane<D>;
    constexpr int IT = 4, STEP = L::HEADS * D;
    L lane(a);
    // `heads` rows from in to out, those out_step apart per set
    auto run = [&](const T* in, T* out, int64_t out_step, int heads, int chunk, const float* weight, bool plain) {
        const int sets = (heads + L::HEADS - 1) / L::HEADS, each = (sets + a.chunks - 1) / a.chunks;
        int s = chunk * each;
        const int end = min(sets, s + each);
        in += s * STEP + lane.sub * D;
        out += s * out_step;
        Four wx, wy;
        lane.weights(weight, wx, wy);
        for (; s < end; s += IT, in += IT * STEP, out += IT * out_step) {
            // sets in which this lane has a head, and sets of this batch
            const int left = (heads - s * L::HEADS - lane.sub + L::HEADS - 1) / L::HEADS;
            const int many = min(IT, end - s);
            Four x[IT], y[IT];
#pragma unroll
            for (int u = 0; u < IT; ++u) {
                x[u] = y[u] = {0, 0};
                if (u < many && u < left) {
                    x[u] = get4(in + u * STEP + lane.oa);
                    y[u] = get4(in + u * STEP + lane.ob);
                }
            }
            T* to = out;
#pragma unroll
            for (int u = 0; u < IT; ++u, to += out_step) {
                if (u >= many) break;
                if (!plain) lane.finish(a, x[u], y[u], wx, wy);
                if (u < left) {
                    put4(to + lane.oa, x[u]);
                    put4(to + lane.ob, y[u]);
                }
            }
        }
    };
    for (uint32_t w = blockIdx.x * 4 + (threadIdx.x >> 5); w < uint32_t(a.N) * a.chunks; w += 4 * gridDim.x) {
        const int n = int(w / a.chunks), chunk = int(w % a.chunks);
        int at;
        int64_t slot;
        if (!place_of(a, n, at, slot)) continue;
        lane.token(a, n, at);
        run(static_cast<const T*>(a.q) + n * a.ldq, static_cast<T*>(a.qo) + (int64_t(n) * a.HQ + lane.sub) * D, STEP,
            a.HQ, chunk, a.qw, false);
        if (!a.kc) {
            run(static_cast<const T*>(a.k) + n * a.ldk, static_cast<T*>(a.ko) + (int64_t(n) * a.HKV + lane.sub) * D,
                STEP, a.HKV, chunk, a.kw, false);
        } else if (slot >= 0) {
            const int64_t row = (slot + (int64_t(lane.sub) << a.log_page)) * D, step = int64_t(STEP) << a.log_page;
            run(static_cast<const T*>(a.k) + n * a.ldk, static_cast<T*>(a.kc) + row, step, a.HKV, chunk, a.kw, false);
            run(static_cast<const T*>(a.v) + n * a.ldv, static_cast<T*>(a.vc) + row, step, a.HKV, chunk, nullptr, true);
        }
    }
}

template <typename T, int D>
cudaError_t launch(Args a, cudaStream_t st) {
    constexpr int HEADS = 256 / D, MOST = 152 * 5;  // resident blocks
    a.sets = (a.HQ + HEADS - 1) / HEADS + (a.kc ? 2 : 1) * ((a.HKV + HEADS - 1) / HEADS);
    const int64_t warps = int64_t(a.N) * a.sets;
    // Up to eight warps a scheduler (four an SM), a warp a set.  Measured, few / many, us in a graph: 16/4 heads
    // into the cache 4.9 / 7.7 at 4,864 warps, 7.0 / 8.9 at 8,000, 9.5 / 9.2 at 12,000, 28 / 18 at 40,000; unit rows of
    // 16/16 heads 2.2 / 3.2, 3.1 / 5.2, 4.4 / 5.4 and 12.9 / 10.0; fp32, 16/4 heads of 64, 4.7 / 7.6, 6.7 / 7.8, 9.5 /
    // 11.3 and 27 / 20.  (The sides cross at 12,000 to 20,000 warps: the border is on the low side.)
    if (warps <= 8 * 152 * 4)
        return launch_pdl(prep_few_kernel<T, D>, dim3(unsigned((warps + 3) / 4)), dim3(128), 0, st, a);
    // as many warps to a token as leave none of the resident ones idle
    a.chunks = (4 * MOST + a.N - 1) / a.N;
    const int64_t blocks = (int64_t(a.N) * a.chunks + 3) / 4;
    return launch_pdl(prep_many_kernel<T, D>, dim3(unsigned(blocks < MOST ? blocks : MOST)), dim3(128), 0, st, a);
}

}  // namespace qkp

cudaError_t launch_qk_prep(const void* q, const void* k, const void* v, int bf16, int64_t ldq, int64_t ldk,
                           int64_t ldv, int norm, const float* qw, const float* kw, float eps, const float* freqs,
                           int R, const int32_t* positions, int axes, int64_t axis_step, int64_t row_step,
                           const int32_t* axis, int adjacent, int N, int B, int HQ, int HKV, int d, void* qo, void* ko,
                           void* kc, void* vc, const int32_t* table, int pages, int log_page, int max_pages,
                           const int32_t* context, const int32_t* starts, const int32_t* lengths, int32_t* err,
                           cudaStream_t st) {
    qkp::Args a = {q, k, v, qo, ko, kc, vc, ldq, ldk, ldv, axis_step, row_step, qw, kw, freqs, positions, axis, table,
                   context, starts, lengths, err, eps, norm, R, adjacent, axes, N, B ? N / B : N, B, HQ, HKV, pages,
                   log_page, max_pages, 0, 0};
    using bf = __nv_bfloat16;
    if (bf16) return d == 128 ? qkp::launch<bf, 128>(a, st) : qkp::launch<bf, 64>(a, st);
    return d == 128 ? qkp::launch<float, 128>(a, st) : qkp::launch<float, 64>(a, st);
}

}  // namespace canopy
