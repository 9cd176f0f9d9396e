// The layer over packed prompts, token by token in fp32: every input type
// and head size.
//
// canopy page (projects.dotslasha.me/p/canopy.md), "The gated delta rule":
// per sequence and value head, for its tokens in order,
//     u = beta (v - g S k),  S <- g S + u k^T,  o = scale S q.
// Value rows are independent: a CTA of 128 threads keeps 16 rows of one
// state in registers (eight lanes per row, dk / 8 entries each) and walks
// the sequence.  What a token waits for is S k on the token before: four
// short sums, a three-step reduction and the update; o hangs off it.  Blocks
// of 16 tokens are read into registers while the block before them is
// computed from shared memory.
//
// Bound by instruction issue and, with several CTAs on an SM, by the reads of
// k and q from shared memory, which every group of eight lanes repeats:
// 0.16 us a token for one sequence of 16 heads (256 tokens: 42.5 us), 96 us
// for four fp32 ones of 600 tokens together, the longest of 414.  Sixteen
// lanes per row were 20 % slower throughout.
#include "common.cuh"

namespace canopy {

namespace scan {

constexpr int ROWS = 16;  // state rows per CTA
constexpr int TB = 16;    // tokens per block
constexpr int NT = 128;

// Tokens [lo, hi) of sequence b; bounds outside [0, N] or out of order are
// read as the nearest admissible ones and reported.
__device__ inline void sequence(const int32_t* starts, int b, int N, int& lo, int& hi, int* bad) {
    const int s0 = starts[b], s1 = starts[b + 1];
    lo = min(max(s0, 0), N);
    hi = min(max(s1, lo), N);
    if (s0 != lo || s1 != hi) *bad |= CANOPY_DEVERR_LENGTH;
}

// Four elements as they are in memory, and as fp32.
template <typename InT>
struct Four {
    using type = float4;
};
template <>
struct Four<__nv_bfloat16> {
    using type = uint2;
};
__device__ inline float4 to_f4(float4 x) { return x; }
__device__ inline float4 to_f4(uint2 x) {
    return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xFFFF0000u), __uint_as_float(x.y << 16),
                       __uint_as_float(x.y & 0xFFFF0000u));
}

// (the bound of four blocks is for the register count, 128: with fewer the
// loop's reads are not moved ahead, 56 us instead of 43 for 256 bf16 tokens)
template <typename InT, typename OutT, int D>
__global__ void __launch_bounds__(NT, 4) scan_kernel(const InT* __restrict__ q, const InT* __restrict__ k,
                                                  const InT* __restrict__ v, const float* __restrict__ g,
                                                  const float* __restrict__ beta, const float* S0, float* S_new,
                                                  const int32_t* __restrict__ starts, OutT* __restrict__ o, int N,
                                                  int HV, int ratio, float scale, int32_t* __restrict__ err) {
    using Raw4 = typename Four<InT>::type;
    constexpr int C4 = D / 32;             // float4 chunks per lane
    constexpr int PER = TB * D / 4 / NT;   // float4 chunks of a block's q (and k) per thread
    static_assert(PER >= 1 && TB * ROWS / NT == 2, "staging");
    __shared__ float4 sQ[2][TB][D / 4], sK[2][TB][D / 4];
    __shared__ float sV[2][TB][ROWS];
    __shared__ float2 sGB[2][TB];  // g, beta
    const int h = blockIdx.y, b = blockIdx.z, t = threadIdx.x;
    const int gl = t & 7, row = t >> 3, r0 = blockIdx.x * ROWS;
    const int H = HV / ratio, hk = h / ratio;
    pdl_wait();
    pdl_trigger();  // after the wait: the next kernel may rely on everything before this one
    int lo, hi, bad = 0;
    sequence(starts, b, N, lo, hi, &bad);

    const size_t at = ((size_t(b) * HV + h) * D + r0 + row) * D;
    float4 s[C4];
#pragma unroll
    for (int c = 0; c < C4; ++c)
        s[c] = S0 ? *reinterpret_cast<const float4*>(S0 + at + (c * 8 + gl) * 4) : make_float4(0.f, 0.f, 0.f, 0.f);

    // The block from token n0 into registers, as it is: whatever looks at a
    // value (the conversion to fp32, the check of a gate) waits for its load,
    // so that comes a block later.  Tokens past the end are not read.
    Raw4 nq[PER], nk[PER];
    InT nv[2];
    float ng, nb;
    auto fetch = [&](int n0) {
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int i = t + e * NT, n = n0 + i / (D / 4), c = i % (D / 4);
            nq[e] = nk[e] = Raw4{};
            if (n < hi) {
                const size_t p = (size_t(n) * H + hk) * D + c * 4;
                nq[e] = __ldg(reinterpret_cast<const Raw4*>(q + p));
                nk[e] = __ldg(reinterpret_cast<const Raw4*>(k + p));
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = t + e * NT, n = n0 + i / ROWS;
            nv[e] = n < hi ? v[(size_t(n) * HV + h) * D + r0 + i % ROWS] : InT(0.f);
        }
        ng = 1.f;
        nb = 0.f;
        if (t < TB && n0 + t < hi) {
            ng = g[size_t(n0 + t) * HV + h];
            nb = beta[size_t(n0 + t) * HV + h];
        }
    };
    if (lo < hi) fetch(lo);
    int buf = 0;
    for (int n0 = lo; n0 < hi; n0 += TB, buf ^= 1) {
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int i = t + e * NT;
            sQ[buf][i / (D / 4)][i % (D / 4)] = to_f4(nq[e]);
            sK[buf][i / (D / 4)][i % (D / 4)] = to_f4(nk[e]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) sV[buf][(t + e * NT) / ROWS][(t + e * NT) % ROWS] = to_f(nv[e]);
        if (t < TB) {
            if (!gate_ok(ng, nb)) {
                bad |= CANOPY_DEVERR_GATE;
                ng = 1.f;
                nb = 0.f;
            }
            sGB[buf][t] = make_float2(ng, nb);
        }
        // (the other buffer's readers are past it: they have met here since)
        __syncthreads();
        if (n0 + TB < hi) fetch(n0 + TB);
        const int m = min(TB, hi - n0);
        OutT* op = o + (size_t(n0) * HV + h) * D + r0 + row;
        // by fours; a token past the end has k = 0, g = 1, beta = 0 and leaves S alone
#pragma unroll 1
        for (int n4 = 0; n4 < m; n4 += 4) {
#pragma unroll
            for (int nn = 0; nn < 4; ++nn) {
                const int n = n4 + nn;
                const float2 gb = sGB[buf][n];
                const float vv = sV[buf][n][row];
                float4 kk[C4];
                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < C4; ++c) {
                    kk[c] = sK[buf][n][c * 8 + gl];
                    part[0] += s[c].x * kk[c].x;
                    part[1] += s[c].y * kk[c].y;
                    part[2] += s[c].z * kk[c].z;
                    part[3] += s[c].w * kk[c].w;
                }
                float sk = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
                for (int x = 4; x; x >>= 1) sk += __shfl_xor_sync(0xffffffffu, sk, x);
                const float a = gb.x, u = gb.y * (vv - a * sk);
                part[0] = part[1] = part[2] = part[3] = 0.f;
#pragma unroll
                for (int c = 0; c < C4; ++c) {
                    s[c].x = a * s[c].x + u * kk[c].x;
                    s[c].y = a * s[c].y + u * kk[c].y;
                    s[c].z = a * s[c].z + u * kk[c].z;
                    s[c].w = a * s[c].w + u * kk[c].w;
                    const float4 qq = sQ[buf][n][c * 8 + gl];
                    part[0] += s[c].x * qq.x;
                    part[1] += s[c].y * qq.y;
                    part[2] += s[c].z * qq.z;
                    part[3] += s[c].w * qq.w;
                }
                float so = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
                for (int x = 4; x; x >>= 1) so += __shfl_xor_sync(0xffffffffu, so, x);
                if (gl == 0 && n < m) store_out(op + size_t(n) * HV * D, scale * so);
            }
        }
    }
#pragma unroll
    for (int c = 0; c < C4; ++c) *reinterpret_cast<float4*>(S_new + at + (c * 8 + gl) * 4) = s[c];
    if (bad && blockIdx.x == 0) raise_err(err, bad);
}

template <typename InT, typename OutT, int D>
cudaError_t launch(const void* q, const void* k, const void* v, const float* g, const float* beta, const float* S0,
                   float* S_new, const int32_t* starts, void* o, int N, int B, int H, int HV, float scale,
                   int32_t* err, cudaStream_t st) {
    return launch_pdl(scan_kernel<InT, OutT, D>, dim3(D / ROWS, HV, B), dim3(NT), 0, st, static_cast<const InT*>(q),
                      static_cast<const InT*>(k), static_cast<const InT*>(v), g, beta, S0, S_new, starts,
                      static_cast<OutT*>(o), N, HV, HV / H, scale, err);
}

}  // namespace scan

cudaError_t launch_prefill_scan(const void* q, const void* k, const void* v, int in_bf16, const float* g,
                                const float* beta, const float* S0, float* S_new, const int32_t* starts, int N, int B,
                                int H, int HV, int d, void* o, int o_bf16, float scale, int32_t* err,
                                cudaStream_t st) {
    using bf = __nv_bfloat16;
#define CANOPY_SCAN(IT, OT, D) \
    return scan::launch<IT, OT, D>(q, k, v, g, beta, S0, S_new, starts, o, N, B, H, HV, scale, err, st)
    if (d == 128) {
        if (in_bf16) {
            if (o_bf16) CANOPY_SCAN(bf, bf, 128);
            CANOPY_SCAN(bf, float, 128);
        }
        if (o_bf16) CANOPY_SCAN(float, bf, 128);
        CANOPY_SCAN(float, float, 128);
    }
    if (in_bf16) {
        if (o_bf16) CANOPY_SCAN(bf, bf, 32);
        CANOPY_SCAN(bf, float, 32);
    }
    if (o_bf16) CANOPY_SCAN(float, bf, 32);
    CANOPY_SCAN(float, float, 32);
#undef CANOPY_SCAN
}

}  // namespace canopy
