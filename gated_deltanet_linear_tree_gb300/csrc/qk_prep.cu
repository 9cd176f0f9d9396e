// Queries and keys of an attention layer: each head's norm, the rotation by the
// token's position, and keys and values into the cache's pages, in one pass.
//
// Per token and head, with y = w x / sqrt(mean x^2 + eps) (rms), x / sqrt(sum
// x^2 + eps) (unit rows) or x: pair j of the first R columns turns by
// position * freq_j (the position on the frequency's axis),
//     (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin).
// All in fp32, rounded once to the type.  The angle is kept in turns: freq_j /
// 2 pi as a 64-bit binary fraction times the whole position wraps at whole turns
// by itself, so that far positions lose nothing.  (The GPU has a 64th of the fp32
// rate in fp64: two fp64 products a pair took 110 of 220 us for 16,383 tokens.)
// Sine and cosine are their series about the nearest quarter turn, to the terms
// that are below 2^-25 at an eighth of a turn.
//
// A lane holds four pairs of a head: for pairs (j, j + R/2) two chunks of four
// elements R/2 apart, else eight elements in a row, so that a pair never leaves
// its lane; d / 8 lanes share a head and a warp takes 256 / d heads at a time.  The
// angles serve all heads that a warp takes of one token.
#include "common.cuh"

namespace canopy {
namespace qkp {

struct Args {
    const void *q, *k, *v;
    void *qo, *ko, *kc, *vc;
    int64_t ldq, ldk, ldv;  // elements from a token to the next
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
__device__ inline void put4(float* p, const Four& x) { *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(x.lo, x.hi); }
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
// bits, times 2^66 / 2 pi, its place given by the exponent.
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

// A warp: `sets` of a token's sets of 32 / LANES heads (queries, keys and values have
// sets of their own, so that a warp does one thing at a time), IT sets at a time.
template <typename T, int D, int IT>
__global__ void __launch_bounds__(128, IT == 1 ? 8 : 7) prep_kernel(const Args a) {
    constexpr int LANES = D / 8, HEADS = 32 / LANES;  // lanes a head, heads of a set
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, l = lane % LANES, sub = lane / LANES;
    const bool turned = 8 * l < a.R, split = !a.adjacent && turned;
    const int oa = split ? 4 * l : 8 * l, ob = split ? oa + a.R / 2 : oa + 4;
    const int qsets = (a.HQ + HEADS - 1) / HEADS, ksets = (a.HKV + HEADS - 1) / HEADS;
    uint64_t turns[4] = {};
    int axis[4] = {};
    if (turned) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            turns[j] = turns_of(a.freqs[4 * l + j]);
            axis[j] = a.axis ? min(max(a.axis[4 * l + j], 0), a.axes - 1) : 0;
        }
    }
    for (uint32_t w = blockIdx.x * 4 + (threadIdx.x >> 5); w < uint32_t(a.N) * a.chunks; w += 4 * gridDim.x) {
        const int n = int(w / a.chunks), chunk = int(w % a.chunks);
        const int first = chunk * a.sets, end = min(qsets + (a.kc ? 2 : 1) * ksets, first + a.sets);
        const T *q = static_cast<const T*>(a.q) + n * a.ldq, *k = static_cast<const T*>(a.k) + n * a.ldk,
                *v = static_cast<const T*>(a.v) + n * a.ldv;
        Four xa[IT], xb[IT];
        auto load = [&](int s0) {
#pragma unroll
            for (int u = 0; u < IT; ++u) {
                const int s = s0 + u;
                if (s >= end) continue;
                const bool query = s < qsets;
                const int h = (query ? s : s < qsets + ksets ? s - qsets : s - qsets - ksets) * HEADS + sub;
                const T* x = (query ? q : s < qsets + ksets ? k : v) + h * D;
                if (h >= (query ? a.HQ : a.HKV)) continue;
                xa[u] = get4(x + oa);
                xb[u] = get4(x + ob);
            }
        };
        load(first);  // ahead of the places' lookups

        int bad = 0, i = 0, b = -1;
        bool here = true;
        if (a.context) {
            b = sequence_of(a, n, i, &bad);
            here = b >= 0;
        }
        int64_t slot = -1;  // the token's row in the pages, without the head
        int at = n;
        if (b >= 0) {
            int ctx = a.context[b];
            if (ctx < 0) {
                bad |= CANOPY_DEVERR_LENGTH;
                ctx = 0;
            }
            const int64_t pos = int64_t(ctx) + i;
            at = int(pos < 0x7FFFFFFF ? pos : 0x7FFFFFFF);
            const int64_t entry = pos >> a.log_page;
            const int page = entry < a.max_pages ? a.table[int64_t(b) * a.max_pages + entry] : -1;
            if (page < 0 || page >= a.pages)
                bad |= CANOPY_DEVERR_PAGE;
            else
                slot = ((int64_t(page) * a.HKV) << a.log_page) + (pos & ((1 << a.log_page) - 1));
        }
        if (bad && lane == 0 && a.err) raise_err(a.err, bad);
        if (!here) continue;

        Four co = {0, 0}, si = {0, 0}, minus = {0, 0};  // cosines, sines and their negatives of this lane's pairs
        if (turned && first < qsets + ksets) {
            float c[4], s[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                turn(a.positions ? a.positions[int64_t(axis[j]) * a.N + n] : at, turns[j], c[j], s[j]);
            co = {pack2(c[0], c[1]), pack2(c[2], c[3])};
            si = {pack2(s[0], s[1]), pack2(s[2], s[3])};
            minus = {pack2(-s[0], -s[1]), pack2(-s[2], -s[3])};
        }
        const float share = a.norm == CANOPY_NORM_RMS ? 1.f / D : 1.f;
        T* qo = static_cast<T*>(a.qo) + int64_t(n) * a.HQ * D;
        T* ko = a.kc ? nullptr : static_cast<T*>(a.ko) + int64_t(n) * a.HKV * D;
        // norm and rotation; `weight` this head's, or null
        auto finish = [&](Four& x, Four& y, bool there, const float* weight) {
            if (a.norm != CANOPY_NORM_NONE) {
                float ss = there ? sum4(fma4(x, x, y * y)) : 0.f;
#pragma unroll
                for (int m = LANES / 2; m; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
                const float r = rsqrtf(fmaf(ss, share, a.eps));
                const Four rr = {pack2(r, r), pack2(r, r)};
                if (weight) {
                    x = x * (rr * get4(weight + oa));
                    y = y * (rr * get4(weight + ob));
                } else {
                    x = x * rr;
                    y = y * rr;
                }
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
        };
        for (int s0 = first; s0 < end; s0 += IT) {
            if (s0 != first) load(s0);
#pragma unroll
            for (int u = 0; u < IT; ++u) {
                const int s = s0 + u;
                if (s >= end) continue;
                if (s < qsets) {
                    const int h = s * HEADS + sub;
                    finish(xa[u], xb[u], h < a.HQ, a.qw);
                    if (h >= a.HQ) continue;
                    put4(qo + h * D + oa, xa[u]);
                    put4(qo + h * D + ob, xb[u]);
                    continue;
                }
                const bool value = s >= qsets + ksets;
                const int h = (value ? s - qsets - ksets : s - qsets) * HEADS + sub;
                if (!value) finish(xa[u], xb[u], h < a.HKV, a.kw);
                if (h >= a.HKV || (a.kc && slot < 0)) continue;
                T* out = !a.kc ? ko + h * D
                               : static_cast<T*>(value ? a.vc : a.kc) + (slot + (int64_t(h) << a.log_page)) * D;
                put4(out + oa, xa[u]);
                put4(out + ob, xb[u]);
            }
        }
    }
}

template <typename T, int D>
cudaError_t launch(Args a, cudaStream_t st) {
    constexpr int HEADS = 256 / D;
    const int sets = (a.HQ + HEADS - 1) / HEADS + (a.kc ? 2 : 1) * ((a.HKV + HEADS - 1) / HEADS);
    // few tokens: a warp to every set of heads; many: up to all sets of a token to a warp, which goes from token
    // to token (what it does once for all tokens and once for a token's sets is as much as ten sets take)
    constexpr int MOST = 152 * 7;  // resident blocks
    const bool many = int64_t(a.N) * sets > 8 * 152 * 4;
    int chunks = sets;
    if (many) {
        chunks = int((2 * 4 * MOST + a.N - 1) / a.N);
        if (chunks > (sets + 3) / 4) chunks = (sets + 3) / 4;
    }
    a.sets = (sets + chunks - 1) / chunks;
    a.chunks = (sets + a.sets - 1) / a.sets;
    const int64_t blocks = (int64_t(a.N) * a.chunks + 3) / 4;
    if (many)
        return launch_pdl(prep_kernel<T, D, 4>, dim3(unsigned(blocks < MOST ? blocks : MOST)), dim3(128), 0, st, a);
    return launch_pdl(prep_kernel<T, D, 1>, dim3(unsigned(blocks)), dim3(128), 0, st, a);
}

}  // namespace qkp

cudaError_t launch_qk_prep(const void* q, const void* k, const void* v, int bf16, int64_t ldq, int64_t ldk,
                           int64_t ldv, int norm, const float* qw, const float* kw, float eps, const float* freqs,
                           int R, const int32_t* positions, int axes, const int32_t* axis, int adjacent, int N, int B,
                           int HQ, int HKV, int d, void* qo, void* ko, void* kc, void* vc, const int32_t* table,
                           int pages, int log_page, int max_pages, const int32_t* context, const int32_t* starts,
                           const int32_t* lengths, int32_t* err, cudaStream_t st) {
    qkp::Args a = {q, k, v, qo, ko, kc, vc, ldq, ldk, ldv, qw, kw, freqs, positions, axis, table, context, starts,
                   lengths, err, eps, norm, R, adjacent, axes, N, B ? N / B : N, B, HQ, HKV, pages, log_page,
                   max_pages, 0, 0};
    using bf = __nv_bfloat16;
    if (bf16) return d == 128 ? qkp::launch<bf, 128>(a, st) : qkp::launch<bf, 64>(a, st);
    return d == 128 ? qkp::launch<float, 128>(a, st) : qkp::launch<float, 64>(a, st);
}

}  // namespace canopy
