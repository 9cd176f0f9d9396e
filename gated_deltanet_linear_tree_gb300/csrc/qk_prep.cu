// Queries and keys of an attention layer: each head's norm, the rotation by the
// token's position, and keys and values into the cache's pages, in one pass.
//
// Per token and head, with y = w x / sqrt(mean x^2 + eps) (rms), x / sqrt(sum
// x^2 + eps) (unit rows) or x: pair j of the first R columns turns by
// position * freq_j (the position on the frequency's axis),
//     (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin).
// All in fp32, rounded once to the type.  The angle is kept in turns: freq_j /
// 2 pi as a 64-bit binary fraction times the whole position wraps at whole turns
// by itself, so that far positions lose nothing, and the top 32 bits go to
// sincospi.
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
    int chunks;  // warps per token
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

// cos and sin of `position` times the frequency `f` (turns as a 64-bit fraction).
__device__ inline void turn(int position, float freq, float& c, float& s) {
    const double turns = double(freq) * 0.15915494309189535;  // 1 / 2 pi
    const double part = turns - floor(turns);
    const uint64_t fraction = uint64_t(part * 18446744073709551616.0);  // (2^64 for part rounding to 1 wraps to 0)
    const int32_t top = int32_t((fraction * uint64_t(int64_t(position)) + 0x80000000ull) >> 32);
    sincospif(float(top) * 4.656612873077393e-10f, &s, &c);  // 2^-31: top 2^-32 turns are top 2^-31 pi
}

template <typename T, int D, int IT>
__global__ void __launch_bounds__(128) prep_kernel(const Args a) {
    constexpr int LANES = D / 8, HEADS = 32 / LANES;  // lanes a head, heads a warp takes at a time
    pdl_wait();
    pdl_trigger();
    const int64_t w = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int n = int(w / a.chunks), chunk = int(w % a.chunks);
    if (n >= a.N) return;
    const int lane = threadIdx.x & 31, l = lane % LANES;
    int bad = 0, i = 0, b = -1;
    if (a.context) {
        b = sequence_of(a, n, i, &bad);
        if (b < 0) {
            if (bad && lane == 0 && a.err) raise_err(a.err, bad);
            return;
        }
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

    const bool split = !a.adjacent && l < a.R / 8;
    const int oa = split ? 4 * l : 8 * l, ob = split ? oa + a.R / 2 : oa + 4;
    float c[4], s[4];
    if (8 * l < a.R) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int f = 4 * l + j;
            const int axis = a.axis ? min(max(a.axis[f], 0), a.axes - 1) : 0;
            turn(a.positions ? a.positions[int64_t(axis) * a.N + n] : at, a.freqs[f], c[j], s[j]);
        }
    }
    const int total = a.HQ + (a.kc ? 2 : 1) * a.HKV;
    const int h0 = (chunk * IT) * HEADS + lane / LANES;
    float xa[IT][4], xb[IT][4];
#pragma unroll
    for (int u = 0; u < IT; ++u) {
        const int h = h0 + u * HEADS;
        if (h >= total) continue;
        const T* x;
        if (h < a.HQ)
            x = static_cast<const T*>(a.q) + n * a.ldq + h * D;
        else if (h < a.HQ + a.HKV)
            x = static_cast<const T*>(a.k) + n * a.ldk + (h - a.HQ) * D;
        else
            x = static_cast<const T*>(a.v) + n * a.ldv + (h - a.HQ - a.HKV) * D;
        get4(x + oa, xa[u]);
        get4(x + ob, xb[u]);
    }
#pragma unroll
    for (int u = 0; u < IT; ++u) {
        const int h = h0 + u * HEADS;
        const bool value = h >= a.HQ + a.HKV, key = h >= a.HQ && !value;
        float ss = 0.f;
        if (h < total)
#pragma unroll
            for (int j = 0; j < 4; ++j) ss += xa[u][j] * xa[u][j] + xb[u][j] * xb[u][j];
#pragma unroll
        for (int m = LANES / 2; m; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        if (h >= total) continue;
        if (!value) {
            if (a.norm != CANOPY_NORM_NONE) {
                const float r = 1.f / sqrtf((a.norm == CANOPY_NORM_RMS ? ss * (1.f / D) : ss) + a.eps);
                const float* wt = key ? a.kw : a.qw;
                float wa[4] = {1.f, 1.f, 1.f, 1.f}, wb[4] = {1.f, 1.f, 1.f, 1.f};
                if (wt) {
                    get4(wt + oa, wa);
                    get4(wt + ob, wb);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    xa[u][j] *= r * wa[j];
                    xb[u][j] *= r * wb[j];
                }
            }
            if (8 * l < a.R) {
                if (split) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float y = xa[u][j], z = xb[u][j];
                        xa[u][j] = y * c[j] - z * s[j];
                        xb[u][j] = z * c[j] + y * s[j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float* p = j < 2 ? xa[u] + 2 * j : xb[u] + 2 * j - 4;
                        const float y = p[0], z = p[1];
                        p[0] = y * c[j] - z * s[j];
                        p[1] = z * c[j] + y * s[j];
                    }
                }
            }
        }
        T* out;
        if (h < a.HQ) {
            out = static_cast<T*>(a.qo) + (int64_t(n) * a.HQ + h) * D;
        } else if (!a.kc) {
            out = static_cast<T*>(a.ko) + (int64_t(n) * a.HKV + h - a.HQ) * D;
        } else {
            if (slot < 0) continue;
            const int hk = value ? h - a.HQ - a.HKV : h - a.HQ;
            out = static_cast<T*>(value ? a.vc : a.kc) + (slot + (int64_t(hk) << a.log_page)) * D;
        }
        put4(out + oa, xa[u]);
        put4(out + ob, xb[u]);
    }
}

template <typename T, int D>
cudaError_t launch(Args a, cudaStream_t st) {
    constexpr int HEADS = 256 / D;
    const int sets = (a.HQ + (a.kc ? 2 : 1) * a.HKV + HEADS - 1) / HEADS;
    // few tokens: a warp to every set of heads; many: four sets a warp, the angles serving them all
    const bool many = int64_t(a.N) * sets > 8 * 152 * 4;
    const int it = many ? 4 : 1;
    a.chunks = (sets + it - 1) / it;
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
                   max_pages, 0};
    using bf = __nv_bfloat16;
    if (bf16) return d == 128 ? qkp::launch<bf, 128>(a, st) : qkp::launch<bf, 64>(a, st);
    return d == 128 ? qkp::launch<float, 128>(a, st) : qkp::launch<float, 64>(a, st);
}

}  // namespace canopy
