// Which node of every stream's draft tree the target's probabilities accept,
// from given random numbers.
//
// A stream walks down from its root.  At node i, with the target's row p_i
// and the draft's row q_i, the children are tried in index order against
// the row r of mass Z (r = p_i, Z = 1 at first): child c with token x is
// accepted if u_c Z q_i(x) < r(x), and the walk goes on from it.  A refused
// child leaves
//     r <- max(r - Z q_i, 0),   Z <- sum_x r(x).
// Without draft probabilities the candidates are the draft's fixed choice:
// q_i is 1 at the child's token, accepted if u_c Z < r(x), and a refused one
// leaves r(x) <- 0, Z <- max(Z - r(x), 0).  Where no child is accepted the
// next token is drawn from r / Z as the first x with the largest r(x) / e(x),
// e(x) given exponential variates (the largest of the independent races
// r(x) / e(x) is x with probability r(x) / Z, so Z is not needed); where r
// is zero throughout, from p_i.  Tokens come out distributed as the
// target's, whatever the draft.
//
// Every product and difference is rounded by itself (no fused multiply-add)
// and the sums are of integers (r in units of 2^-46, rounded down), so that
// the result does not depend on the order of threads or of a sum.
#include "common.cuh"

namespace canopy {

namespace acc {

constexpr int NT = 1024;

struct Best {
    float s;
    int x;
};

// The better of two candidates: the larger score, then the lower index.
__device__ inline Best better(Best a, Best b) {
    return (b.s > a.s || (b.s == a.s && b.x < a.x)) ? b : a;
}

template <typename PT>
__global__ void __launch_bounds__(NT) accept_kernel(const PT* __restrict__ p, const PT* __restrict__ q,
                                                    const int32_t* __restrict__ tokens,
                                                    const int32_t* __restrict__ parent,
                                                    const int32_t* __restrict__ lengths, const float* __restrict__ u,
                                                    const float* __restrict__ noise, int T, int V,
                                                    int32_t* __restrict__ accepted, int32_t* __restrict__ out,
                                                    int32_t* __restrict__ count, int32_t* __restrict__ err) {
    __shared__ int sParent[kMaxT], sTok[kMaxT];
    __shared__ float sR[kMaxT], sQ[kMaxT], sU[kMaxT];
    __shared__ float sZ[kMaxT];      // Z before each refusal at the current node
    __shared__ int sRefused[kMaxT];  // the refused tokens of the current node
    __shared__ unsigned long long sSum;
    __shared__ Best sBest[NT / 32];
    const int b = blockIdx.x, t = threadIdx.x;
    pdl_wait();
    pdl_trigger();  // after the wait: the next kernel may rely on everything before this one
    int bad = 0;
    const int n = stream_len(lengths, b, T, &bad);
    const size_t nodes = size_t(b) * T;
    if (t < n) {
        int pa = parent[nodes + t];
        if (!((t == 0) ? (pa == -1) : (pa >= 0 && pa < t))) {
            bad |= CANOPY_DEVERR_TREE;
            pa = (t == 0) ? -1 : 0;
        }
        const int x = tokens[nodes + t];
        float r = 0.f, qx = 0.f;
        if (t > 0) {
            if (x >= 0 && x < V) {
                r = to_f(p[(nodes + pa) * V + x]);
                if (q) qx = to_f(q[(nodes + pa) * V + x]);
            } else {
                bad |= CANOPY_DEVERR_TOKEN;
            }
        }
        sParent[t] = pa;
        sTok[t] = x;
        sR[t] = r;
        sQ[t] = q ? qx : 1.f;
        sU[t] = u[nodes + t];
    }
    if (t < T) out[nodes + t] = -1;
    if (bad && err) raise_err(err, bad);
    __syncthreads();
    if (n == 0) {
        if (t == 0) {
            accepted[b] = -1;
            count[b] = 0;
        }
        return;
    }

    // The walk; every thread follows it on the same shared values.
    int cur = 0, taken = 0, refused = 0;
    float Z = 1.f;
    for (int c = 1; c < n; ++c) {  // children come after their node, siblings in order
        if (sParent[c] != cur) continue;
        const float r = sR[c];
        if (__fmul_rn(__fmul_rn(sU[c], Z), sQ[c]) < r) {
            if (t == 0) out[nodes + taken] = sTok[c];
            cur = c;
            ++taken;
            refused = 0;
            Z = 1.f;
            continue;
        }
        __syncthreads();  // sR is read by all before it changes
        if (t == 0) {
            sZ[refused] = Z;
            sRefused[refused] = sTok[c];
            sSum = 0;
        }
        if (t > c && t < n && sParent[t] == cur) {
            if (q) sR[t] = fmaxf(__fsub_rn(sR[t], __fmul_rn(Z, sQ[t])), 0.f);
            else if (sTok[t] == sTok[c]) sR[t] = 0.f;
        }
        ++refused;
        __syncthreads();
        if (q) {
            const PT* pr = p + (nodes + cur) * V;
            const PT* qr = q + (nodes + cur) * V;
            unsigned long long sum = 0;
            for (int x = t; x < V; x += NT) {
                float rx = to_f(pr[x]);
                const float qx = to_f(qr[x]);
                for (int m = 0; m < refused; ++m) rx = fmaxf(__fsub_rn(rx, __fmul_rn(sZ[m], qx)), 0.f);
                sum += static_cast<unsigned long long>(__float2ll_rz(rx * 70368744177664.f));  // 2^46
            }
#pragma unroll
            for (int m = 16; m; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
            if ((t & 31) == 0) atomicAdd(&sSum, sum);
            __syncthreads();
            Z = __ll2float_rn(static_cast<long long>(sSum)) * 1.4210854715202004e-14f;  // 2^-46
        } else {
            Z = fmaxf(__fsub_rn(Z, r), 0.f);
        }
    }

    // The next token: from r, and where r is zero throughout from p.
    const PT* pr = p + (nodes + cur) * V;
    const PT* qr = q ? q + (nodes + cur) * V : nullptr;
    for (int pass = 0; pass < 2; ++pass) {
        Best best = {0.f, V};
        for (int x = t; x < V; x += NT) {
            float rx = to_f(pr[x]);
            if (pass == 0) {
                if (q) {
                    const float qx = refused ? to_f(qr[x]) : 0.f;
                    for (int m = 0; m < refused; ++m) rx = fmaxf(__fsub_rn(rx, __fmul_rn(sZ[m], qx)), 0.f);
                } else {
                    for (int m = 0; m < refused; ++m) rx = (x == sRefused[m]) ? 0.f : rx;
                }
            }
            best = better(best, Best{__fdiv_rn(rx, noise[size_t(b) * V + x]), x});
        }
#pragma unroll
        for (int m = 16; m; m >>= 1) {
            const Best o = {__shfl_xor_sync(0xffffffffu, best.s, m), __shfl_xor_sync(0xffffffffu, best.x, m)};
            best = better(best, o);
        }
        __syncthreads();
        if ((t & 31) == 0) sBest[t >> 5] = best;
        __syncthreads();
        best = sBest[0];
        for (int w = 1; w < NT / 32; ++w) best = better(best, sBest[w]);
        if (t == 0) {
            out[nodes + taken] = best.x < V ? best.x : 0;
            accepted[b] = cur;
            count[b] = taken + 1;
        }
        if (best.s > 0.f) break;
    }
}

}  // namespace acc

cudaError_t launch_accept(const void* p, const void* q, int bf16, const int32_t* tokens, const int32_t* parent,
                          const int32_t* lengths, const float* u, const float* noise, int T, int B, int V,
                          int32_t* accepted, int32_t* out, int32_t* count, int32_t* err, cudaStream_t st) {
    if (bf16)
        return launch_pdl(acc::accept_kernel<__nv_bfloat16>, dim3(B), dim3(acc::NT), 0, st,
                          static_cast<const __nv_bfloat16*>(p), static_cast<const __nv_bfloat16*>(q), tokens, parent,
                          lengths, u, noise, T, V, accepted, out, count, err);
    return launch_pdl(acc::accept_kernel<float>, dim3(B), dim3(acc::NT), 0, st, static_cast<const float*>(p),
                      static_cast<const float*>(q), tokens, parent, lengths, u, noise, T, V, accepted, out, count,
                      err);
}

}  // namespace canopy
