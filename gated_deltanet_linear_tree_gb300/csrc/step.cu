// One token of every stream: the recurrent form of the layer.
//
// canopy page (projects.dotslasha.me/p/canopy.md), "The gated delta rule",
// per stream b and value head h, with the state S [dv][dk]:
//     S_new = g S (I - beta k k^T) + beta v k^T,   o = scale S_new q.
// Row r of the state meets the others nowhere:
//     u_r = beta (v_r - g S_r.k),  S_new,r = g S_r + u_r k,
//     o_r = scale (g S_r.q + u_r k.q),
// so that both products of the old row are formed in one pass and the row is
// read and written once.  Eight lanes share a row (dk / 8 entries each,
// three-step shuffle reductions) and a CTA of 128 threads takes 16 rows.
// S_new may be S: a thread writes only what it has read itself.
//
// Bound by HBM: 128 KB per (stream, value head) and nothing twice.  With 32
// value heads and bf16 q/k/v 200 streams take 119.6 us (7.05 TB/s, 1.04 of the
// measured copy bandwidth), 16 streams 11.5 us (0.86) and one 2.1 us.  d = 32 has
// the same blocks, each with 4 KB to move: 200 streams 14.2 us (0.54), 2,000
// 130 us (0.60).
#include "common.cuh"

namespace canopy {

namespace st1 {

constexpr int ROWS = 16;  // state rows per CTA

template <typename InT, typename OutT, int D>
__global__ void __launch_bounds__(128) step_kernel(const InT* __restrict__ q, const InT* __restrict__ k,
                                                   const InT* __restrict__ v, const float* __restrict__ g,
                                                   const float* __restrict__ beta, const float* S, float* S_new,
                                                   OutT* __restrict__ o, int HV, int ratio, float scale,
                                                   int32_t* __restrict__ err) {
    constexpr int C4 = D / 32;  // float4 chunks per lane
    const int h = blockIdx.y, b = blockIdx.z, t = threadIdx.x;
    const int gl = t & 7, r = blockIdx.x * ROWS + (t >> 3);
    const int hk = (ratio == 1) ? h : h / ratio;  // the key head this value head reads
    pdl_wait();
    pdl_trigger();  // after the wait: the next kernel may rely on everything before this one

    const size_t unit = size_t(b) * HV + h;
    const size_t row = (unit * D + r) * D, key = (size_t(b) * (HV / ratio) + hk) * D;
    float4 s[C4], kk[C4], qq[C4];
#pragma unroll
    for (int c = 0; c < C4; ++c) s[c] = *reinterpret_cast<const float4*>(S + row + (c * 8 + gl) * 4);
#pragma unroll
    for (int c = 0; c < C4; ++c) kk[c] = load4(k + key + (c * 8 + gl) * 4);
#pragma unroll
    for (int c = 0; c < C4; ++c) qq[c] = load4(q + key + (c * 8 + gl) * 4);
    const float vv = to_f(v[unit * D + r]);
    float a = g[unit], be = beta[unit];
    if (!decay_ok(a, be)) {
        if (err && t == 0 && blockIdx.x == 0) raise_err(err, CANOPY_DEVERR_GATE);
        a = 1.f;
        be = 0.f;
    }
    float sk = 0.f, sq = 0.f, kq = 0.f;
#pragma unroll
    for (int c = 0; c < C4; ++c) {
        sk += s[c].x * kk[c].x + s[c].y * kk[c].y + s[c].z * kk[c].z + s[c].w * kk[c].w;
        sq += s[c].x * qq[c].x + s[c].y * qq[c].y + s[c].z * qq[c].z + s[c].w * qq[c].w;
        kq += kk[c].x * qq[c].x + kk[c].y * qq[c].y + kk[c].z * qq[c].z + kk[c].w * qq[c].w;
    }
#pragma unroll
    for (int m = 4; m; m >>= 1) {
        sk += __shfl_xor_sync(0xffffffffu, sk, m);
        sq += __shfl_xor_sync(0xffffffffu, sq, m);
        kq += __shfl_xor_sync(0xffffffffu, kq, m);
    }
    const float u = be * (vv - a * sk);
#pragma unroll
    for (int c = 0; c < C4; ++c) {
        s[c].x = a * s[c].x + u * kk[c].x;
        s[c].y = a * s[c].y + u * kk[c].y;
        s[c].z = a * s[c].z + u * kk[c].z;
        s[c].w = a * s[c].w + u * kk[c].w;
        *reinterpret_cast<float4*>(S_new + row + (c * 8 + gl) * 4) = s[c];
    }
    if (gl == 0) store_out(o + unit * D + r, scale * (a * sq + u * kq));
}

template <typename InT, typename OutT, int D>
cudaError_t launch(const void* q, const void* k, const void* v, const float* g, const float* beta, const float* S,
                   float* S_new, void* o, int B, int H, int HV, float scale, int32_t* err, cudaStream_t st) {
    return launch_pdl(step_kernel<InT, OutT, D>, dim3(D / ROWS, HV, B), dim3(128), 0, st, static_cast<const InT*>(q),
                      static_cast<const InT*>(k), static_cast<const InT*>(v), g, beta, S, S_new,
                      static_cast<OutT*>(o), HV, HV / H, scale, err);
}

}  // namespace st1

cudaError_t launch_step(const void* q, const void* k, const void* v, int in_bf16, const float* g, const float* beta,
                        const float* S, float* S_new, int B, int H, int HV, int d, void* o, int o_bf16, float scale,
                        int32_t* err, cudaStream_t st) {
    using bf = __nv_bfloat16;
#define CANOPY_STEP(IT, OT, D) return st1::launch<IT, OT, D>(q, k, v, g, beta, S, S_new, o, B, H, HV, scale, err, st)
    if (d == 128) {
        if (in_bf16) {
            if (o_bf16) CANOPY_STEP(bf, bf, 128);
            CANOPY_STEP(bf, float, 128);
        }
        if (o_bf16) CANOPY_STEP(float, bf, 128);
        CANOPY_STEP(float, float, 128);
    }
    if (in_bf16) {
        if (o_bf16) CANOPY_STEP(bf, bf, 32);
        CANOPY_STEP(bf, float, 32);
    }
    if (o_bf16) CANOPY_STEP(float, bf, 32);
    CANOPY_STEP(float, float, 32);
#undef CANOPY_STEP
}

}  // namespace canopy
