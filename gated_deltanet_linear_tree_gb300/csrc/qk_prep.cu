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

// Four elements in fp32, and back.
__device__ inline void get4(const float* p, float (&x)[4]) {
    const float4 t = *reinterpret_cast<const float4*>(p);
    x[0] = t.x; x[1] = t.y; x[2] = t.z; x[3] = t.w;
}
__device__ inline void get4(const __nv_bfloat16* p, float (&x)[4]) {
    const uint2 t = *reinterpret_cast<const uint2*>(p);
    x[0] = __uint_as_float(t.x << 16); x[1] = __uint_as_float(t.x & 0xFFFF0000u);
    x[2] = __uint_as_float(t.y << 16); x[3] = __uint_as_float(t.y & 0xFFFF0000u);
}
__device__ inline void put4(float* p, const float (&x)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ inline void put4(__nv_bfloat16* p, const float (&x)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    uint2 t;
    t.x = *reinterpret_cast<const uint32_t*>(&a);
    t.y = *reinterpret_cast<const uint32_t*>(&b);
    *reinterpret_cast<uint2*>(p) = t;
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

// A warp: `sets` times 32 / LANES heads of a token, IT sets at a time.
template <typename T, int D, int IT>
__global__ void __launch_bounds__(128) prep_kernel(const Args a) {
    constexpr int LANES = D / 8, HEADS = 32 / LANES;  // lanes a head, heads a warp takes at a time
    pdl_wait();
    pdl_trigger();
    const int64_t w = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int n = int(w / a.chunks), chunk = int(w % a.chunks);
    if (n >= a.N) return;
    const int lane = threadIdx.x & 31, l = lane % LANES;
    const bool turned = 8 * l < a.R, split = !a.adjacent && turned;
    const int oa = split ? 4 * l : 8 * l, ob = split ? oa + a.R / 2 : oa + 4;
    const int total = a.HQ + (a.kc ? 2 : 1) * a.HKV;
    const int first = chunk * a.sets * HEADS + lane / LANES, end = min(total, (chunk + 1) * a.sets * HEADS);
    const T *q = static_cast<const T*>(a.q) + n * a.ldq, *k = static_cast<const T*>(a.k) + n * a.ldk,
            *v = static_cast<const T*>(a.v) + n * a.ldv;
    float xa[IT][4], xb[IT][4];
    auto load = [&](int h0) {
#pragma unroll
        for (int u = 0; u < IT; ++u) {
            const int h = h0 + u * HEADS;
            if (h >= end) continue;
            const T* x = h < a.HQ ? q + h * D : h < a.HQ + a.HKV ? k + (h - a.HQ) * D : v + (h - a.HQ - a.HKV) * D;
            get4(x + oa, xa[u]);
            get4(x + ob, xb[u]);
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
    if (!here) return;

    float c[4], s[4];
    if (turned) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int f = 4 * l + j;
            const int axis = a.axis ? min(max(a.axis[f], 0), a.axes - 1) : 0;
            turn(a.positions ? a.positions[int64_t(axis) * a.N + n] : at, turns_of(a.freqs[f]), c[j], s[j]);
        }
    }
    float wq[8], wk[8];  // the weights of this lane's columns
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int col = j < 4 ? oa + j : ob + j - 4;
        wq[j] = a.qw ? a.qw[col] : 1.f;
        wk[j] = a.kw ? a.kw[col] : 1.f;
    }
    const float share = a.norm == CANOPY_NORM_RMS ? 1.f / D : 1.f;
    T* qo = static_cast<T*>(a.qo) + int64_t(n) * a.HQ * D;
    T* ko = a.kc ? nullptr : static_cast<T*>(a.ko) + int64_t(n) * a.HKV * D;
    for (int h0 = first; h0 - lane / LANES < end; h0 += IT * HEADS) {  // (a warp's lanes stay together)
        if (h0 != first) load(h0);
#pragma unroll
        for (int u = 0; u < IT; ++u) {
            const int h = h0 + u * HEADS;
            const bool there = h < end, query = h < a.HQ, value = h >= a.HQ + a.HKV;
            float r = 1.f;
            if (a.norm != CANOPY_NORM_NONE) {
                float ss = 0.f;
                if (there)
#pragma unroll
                    for (int j = 0; j < 4; ++j) ss += xa[u][j] * xa[u][j] + xb[u][j] * xb[u][j];
#pragma unroll
                for (int m = LANES / 2; m; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
                r = rsqrtf(fmaf(ss, share, a.eps));
            }
            if (!there) continue;
            if (!value) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    xa[u][j] *= r * (query ? wq[j] : wk[j]);
                    xb[u][j] *= r * (query ? wq[4 + j] : wk[4 + j]);
                }
                if (split) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float y = xa[u][j], z = xb[u][j];
                        xa[u][j] = y * c[j] - z * s[j];
                        xb[u][j] = z * c[j] + y * s[j];
                    }
                } else if (turned) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float* p = j < 2 ? xa[u] + 2 * j : xb[u] + 2 * j - 4;
                        const float y = p[0], z = p[1];
                        p[0] = y * c[j] - z * s[j];
                        p[1] = z * c[j] + y * s[j];
                    }
                }
            }
            T* out;
            if (query) {
                out = qo + h * D;
            } else if (!a.kc) {
                out = ko + (h - a.HQ) * D;
            } else {
                if (slot < 0) continue;
                const int hk = value ? h - a.HQ - a.HKV : h - a.HQ;
                out = static_cast<T*>(value ? a.vc : a.kc) + (slot + (int64_t(hk) << a.log_page)) * D;
            }
            put4(out + oa, xa[u]);
            put4(out + ob, xb[u]);
        }
    }
}

template <typename T, int D>
cudaError_t launch(Args a, cudaStream_t st) {
    constexpr int HEADS = 256 / D;
    const int sets = (a.HQ + (a.kc ? 2 : 1) * a.HKV + HEADS - 1) / HEADS;
    // few tokens: a warp to every set of heads; many: as many sets a warp, in fours, as leave four warps to
    // each place on the SMs, the angles serving them all
    const bool many = int64_t(a.N) * sets > 8 * 152 * 4;
    a.sets = 1;
    if (many) {
        const int64_t fours = int64_t(a.N) * sets / (4 * 152 * 64);
        a.sets = int(4 * (fours < 4 ? 1 : fours / 4));
        if (a.sets > sets) a.sets = (sets + 3) / 4 * 4;
    }
    a.chunks = (sets + a.sets - 1) / a.sets;
    const dim3 grid(unsigned((int64_t(a.N) * a.chunks + 3) / 4));
    if (many) return launch_pdl(prep_kernel<T, D, 4>, grid, dim3(128), 0, st, a);
    return launch_pdl(prep_kernel<T, D, 1>, grid, dim3(128), 0, st, a);
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
