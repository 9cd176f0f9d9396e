// The layer over packed prompts, token by token in fp32: every input type
// and head size.
//
// canopy page (projects.dotslasha.me/p/canopy.md), "The gated delta rule":
// per sequence and value head, for its tokens in order,
//     u = beta (v - g S k),  S <- g S + u k^T,  o = scale S q.
// Value rows are independent: a CTA of 128 threads keeps 16 or 32 rows of one
// state in registers (eight lanes per row, dk / 8 entries of one or two rows
// each) and walks the sequence.  What a token waits for is S k on the token
// before: four short sums, a three-step reduction and the update; o hangs off
// it.  Blocks of 16 tokens are read into registers while the block before
// them is computed from shared memory.
//
// Bound by the reads of k and q from shared memory, which every eight lanes
// repeat (130 of the 300 cycles of a token of 16 rows on an SM), and by the
// chain.  With two rows a lane those reads serve both: slower alone (0.21 us a
// token for 0.17), but two such blocks on an SM take 0.31 and three 0.41, where
// two of 16 rows take 0.25 and four 0.40.  So 16 rows where every block has an
// SM for itself.  100 bf16 tokens, d = 128, us at 16 or 32 rows a block:
// 16 states 18 / 21, 32 states 25 / 21, 64 states 40 / 31, 128 states 70 / 59,
// 512 states 260 / 187.  Four rows a lane: 30, 31 (32, 64 states), 191 (512).
// Sixteen or 32 lanes per row, and blocks of 2 or 4 tokens in closed form,
// were slower or no faster.  Long prompts take as long per token: 16,384 of fp32
// 2.6 ms with 16 value heads and 3.2 with 32, bf16 ones of d = 32 1.7.
#include "common.cuh"

namespace canopy {

namespace scan {

constexpr size_t kSMs = 152;
constexpr int TB = 16;  // tokens per block
constexpr int NT = 128;

// starts in order, for calls of more than kMaxUnordered sequences: one block,
// a segment of them per thread.
constexpr int kOrderThreads = 1024;
__global__ void __launch_bounds__(kOrderThreads) order_starts_kernel(const int32_t* __restrict__ starts, int N, int B,
                                                                     int32_t* __restrict__ ordered,
                                                                     int32_t* __restrict__ err) {
    __shared__ int sMax[kOrderThreads];
    const int t = threadIdx.x, per = B / kOrderThreads + 1;  // of B + 1 starts
    const int i0 = t * per, i1 = min(i0 + per, B + 1);
    pdl_wait();
    pdl_trigger();  // after the wait: the next kernel may rely on everything before this one
    int s = 0, bad = 0;
    for (int i = i0; i < i1; ++i) s = max(s, start_in_range(starts, i, N));
    sMax[t] = s;
    __syncthreads();
    for (int step = 1; step < kOrderThreads; step *= 2) {  // sMax[t]: the largest of segments 0 .. t
        const int y = t >= step ? sMax[t - step] : 0;
        __syncthreads();
        sMax[t] = max(sMax[t], y);
        __syncthreads();
    }
    s = t > 0 ? sMax[t - 1] : 0;
    for (int i = i0; i < i1; ++i) {
        s = max(s, start_in_range(starts, i, N));
        ordered[i] = s;
        if (starts[i] != s) bad = CANOPY_DEVERR_LENGTH;
    }
    if (bad) raise_err(err, bad);
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

// (the bounds are for the register counts, 128 and 168; R = 1 with 168 takes
// 77 us for 256 tokens of 32 states instead of 60, R = 2 with 128 as long as
// with 168 where blocks are many and 5 % longer where they are few)
template <typename InT, typename OutT, int D, int R>
__global__ void __launch_bounds__(NT, R == 1 ? 4 : 3) scan_kernel(const InT* __restrict__ q, const InT* __restrict__ k,
                                                  const InT* __restrict__ v, const float* __restrict__ g,
                                                  const float* __restrict__ beta, const float* S0, float* S_new,
                                                  const int32_t* __restrict__ starts, OutT* __restrict__ o, int N,
                                                  int HV, int ratio, float scale, int32_t* __restrict__ err) {
    using Raw4 = typename Four<InT>::type;
    constexpr int C4 = D / 32;             // float4 chunks per lane and row
    constexpr int ROWS = 16 * R;           // state rows per CTA
    constexpr int PER = TB * D / 4 / NT;   // float4 chunks of a block's q (and k) per thread
    static_assert(PER >= 1 && D % ROWS == 0, "staging");
    __shared__ float4 sQ[2][TB][D / 4], sK[2][TB][D / 4];
    __shared__ float sV[2][TB][ROWS];
    __shared__ float2 sGB[2][TB];  // g, beta
    const int h = blockIdx.y, b = blockIdx.z, t = threadIdx.x;
    const int gl = t & 7, row = (t >> 3) * R, r0 = blockIdx.x * ROWS;
    const int H = HV / ratio, hk = h / ratio;
    pdl_wait();
    pdl_trigger();  // after the wait: the next kernel may rely on everything before this one
    int lo = start_in_range(starts, b, N), hi = max(start_in_range(starts, b + 1, N), lo), bad = 0;

    const size_t at = ((size_t(b) * HV + h) * D + r0 + row) * D;
    float4 s[R][C4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < C4; ++c)
            s[r][c] = S0 ? *reinterpret_cast<const float4*>(S0 + at + r * D + (c * 8 + gl) * 4)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
    // The block from token n0 into registers, as it is: whatever looks at a
    // value (the conversion to fp32, the check of a gate) waits for its load,
    // so that comes a block later.  Tokens past the end are not read.
    Raw4 nq[PER], nk[PER];
    constexpr int VP = TB * ROWS / NT;
    InT nv[VP];
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
        for (int e = 0; e < VP; ++e) {
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
    // With the sequence's bounds as they are given, and again in the rare case
    // that an earlier start is larger; looked at once the first reads are out
    // (before them it took 200 single tokens from 180 to 208 us).
#pragma unroll 1
    for (bool again = true; again;) {
        if (lo < hi) fetch(lo);
        const int s = first_token(starts, b, gridDim.z, N, lo);
        again = s != lo;
        lo = s;
        hi = max(hi, s);
    }
    if (starts[b] != lo || starts[b + 1] != hi) bad |= CANOPY_DEVERR_LENGTH;
    int buf = 0;
    for (int n0 = lo; n0 < hi; n0 += TB, buf ^= 1) {
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int i = t + e * NT;
            sQ[buf][i / (D / 4)][i % (D / 4)] = to_f4(nq[e]);
            sK[buf][i / (D / 4)][i % (D / 4)] = to_f4(nk[e]);
        }
#pragma unroll
        for (int e = 0; e < VP; ++e) sV[buf][(t + e * NT) / ROWS][(t + e * NT) % ROWS] = to_f(nv[e]);
        if (t < TB) {
            if (!decay_ok(ng, nb)) {
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
                float4 kk[C4];
                float u[R], so[R];
#pragma unroll
                for (int c = 0; c < C4; ++c) kk[c] = sK[buf][n][c * 8 + gl];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < C4; ++c) {
                        part[0] += s[r][c].x * kk[c].x;
                        part[1] += s[r][c].y * kk[c].y;
                        part[2] += s[r][c].z * kk[c].z;
                        part[3] += s[r][c].w * kk[c].w;
                    }
                    u[r] = (part[0] + part[1]) + (part[2] + part[3]);
                }
#pragma unroll
                for (int x = 4; x; x >>= 1)
#pragma unroll
                    for (int r = 0; r < R; ++r) u[r] += __shfl_xor_sync(0xffffffffu, u[r], x);
                const float a = gb.x;
#pragma unroll
                for (int r = 0; r < R; ++r) u[r] = gb.y * (sV[buf][n][row + r] - a * u[r]);
                float part[R][4] = {};
#pragma unroll
                for (int c = 0; c < C4; ++c) {
                    const float4 qq = sQ[buf][n][c * 8 + gl];
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        s[r][c].x = a * s[r][c].x + u[r] * kk[c].x;
                        s[r][c].y = a * s[r][c].y + u[r] * kk[c].y;
                        s[r][c].z = a * s[r][c].z + u[r] * kk[c].z;
                        s[r][c].w = a * s[r][c].w + u[r] * kk[c].w;
                        part[r][0] += s[r][c].x * qq.x;
                        part[r][1] += s[r][c].y * qq.y;
                        part[r][2] += s[r][c].z * qq.z;
                        part[r][3] += s[r][c].w * qq.w;
                    }
                }
#pragma unroll
                for (int r = 0; r < R; ++r) so[r] = (part[r][0] + part[r][1]) + (part[r][2] + part[r][3]);
#pragma unroll
                for (int x = 4; x; x >>= 1)
#pragma unroll
                    for (int r = 0; r < R; ++r) so[r] += __shfl_xor_sync(0xffffffffu, so[r], x);
                float mine = so[0];  // lane r of the eight stores row r's
#pragma unroll
                for (int r = 1; r < R; ++r) mine = gl == r ? so[r] : mine;
                if (gl < R && n < m) store_out(op + size_t(n) * HV * D + gl, scale * mine);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < C4; ++c) *reinterpret_cast<float4*>(S_new + at + r * D + (c * 8 + gl) * 4) = s[r][c];
    if (bad && blockIdx.x == 0) raise_err(err, bad);
}

template <typename InT, typename OutT, int D, int R>
cudaError_t launch_rows(const void* q, const void* k, const void* v, const float* g, const float* beta,
                        const float* S0, float* S_new, const int32_t* starts, void* o, int N, int B, int H, int HV,
                        float scale, int32_t* err, cudaStream_t st) {
    // With more blocks than SMs but at most two for each, shared memory that
    // is not used keeps a third from an SM: 64 states 31 us instead of 41.
    constexpr int kTwoPerSM = 42 * 1024;
    static OncePerDevice attrs;
    const cudaError_t e = attrs([] { return allow_smem(scan_kernel<InT, OutT, D, R>, kTwoPerSM); });
    if (e != cudaSuccess) return e;
    const size_t blocks = size_t(D / (16 * R)) * HV * B;
    const int unused = D == 128 && blocks > kSMs && blocks <= 2 * kSMs ? kTwoPerSM : 0;
    return launch_pdl(scan_kernel<InT, OutT, D, R>, dim3(D / (16 * R), HV, B), dim3(NT), unused, st,
                      static_cast<const InT*>(q), static_cast<const InT*>(k), static_cast<const InT*>(v), g, beta, S0,
                      S_new, starts, static_cast<OutT*>(o), N, HV, HV / H, scale, err);
}

template <typename InT, typename OutT, int D>
cudaError_t launch(const void* q, const void* k, const void* v, const float* g, const float* beta, const float* S0,
                   float* S_new, const int32_t* starts, void* o, int N, int B, int H, int HV, float scale,
                   int32_t* err, cudaStream_t st) {
    const auto rows = size_t(D / 16) * HV * B <= kSMs ? launch_rows<InT, OutT, D, 1> : launch_rows<InT, OutT, D, 2>;
    return rows(q, k, v, g, beta, S0, S_new, starts, o, N, B, H, HV, scale, err, st);
}

}  // namespace scan

cudaError_t launch_order_starts(const int32_t* starts, int N, int B, int32_t* ordered, int32_t* err,
                                cudaStream_t st) {
    return launch_pdl(scan::order_starts_kernel, dim3(1), dim3(scan::kOrderThreads), 0, st, starts, N, B, ordered,
                      err);
}

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
