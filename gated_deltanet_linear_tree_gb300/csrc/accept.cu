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
//
// A cluster of up to 16 blocks takes a stream, a slice of the vocabulary
// each.  Every block walks by itself on the same numbers (one probability
// per node and row, gathered for all nodes at once), so that blocks meet
// only for a mass that a later sibling needs and for the final draw.  What
// has to be read is the last node's rows and the noise, once: 4 to 12 bytes
// per token of the vocabulary and stream.
//
// Bound by latency up to 65,536 tokens: two dependent reads before the walk,
// the rows' read after it, and a meeting of the cluster (about 1 us) for each
// mass and for the draw.  A chain of 8 over 32,000 tokens takes 6.0 to 6.7 us, 48
// ragged trees of 33 nodes over 50,021 tokens with draft rows 21 to 23 (up to
// four masses one after the other).  Over more a block's slice is longer and its
// tiles are read one after the other: 16 trees of 64 nodes without draft rows
// take 9.1 us over 65,536 tokens and 12.8 to 13.8 over 131,072 (17 MB); with draft
// rows over 151,936, where no slice is held and each mass reads both rows again,
// 32 us, and 36 with bf16 rows.
// Slices of 4,096 tokens for 256 threads measured best: 512 threads or
// slices twice as long took 1.1 to 1.5 times as long.
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"

namespace canopy {

namespace acc {

namespace cg = cooperative_groups;

constexpr int NT = 256;
constexpr int TILE = 8;                  // elements of a thread that are in flight together
constexpr int kTileTokens = NT * TILE;
constexpr int kSlice = 2 * kTileTokens;  // tokens of a block's slice, where that many blocks do
constexpr int kMaxHeld = 3 * kSlice;     // tokens of a slice that fit in shared memory
constexpr int kSMs = 152;
constexpr int kMaxCluster = 16;          // (beyond 8 a kernel has to ask)
constexpr int WORDS = kMaxT / 32;        // of a set of nodes

// A score > 0 and its token as one key whose order is: larger score, then
// lower token.  0 stands for none.
__device__ inline unsigned long long key_of(float s, int x) {
    return s > 0.f ? (static_cast<unsigned long long>(__float_as_uint(s)) << 32) | (0xFFFFFFFFu - x) : 0ull;
}
__device__ inline unsigned long long larger(unsigned long long a, unsigned long long b) { return a > b ? a : b; }

// The floors of sums of values in [0, 1] in units of 2^-46, each value
// rounded down: r + 1 rounded towards zero carries floor(2^23 r) in its
// significand, and what is left, times 2^23, the next 23 bits in the same
// way.  (Conversions to 64-bit integers are a slow pipe.)
struct Units {
    uint32_t hi = 0, lo = 0;  // sums of the bit patterns, modulo 2^32; up to 2^8 values
    int count = 0;
    __device__ void add(float r) {
        const float s = __fadd_rz(r, 1.f);
        const float t = __fadd_rz(__fmul_rn(__fsub_rn(r, __fsub_rn(s, 1.f)), 8388608.f), 1.f);
        hi += __float_as_uint(s);
        lo += __float_as_uint(t);
        ++count;
    }
    __device__ unsigned long long total() const {
        const uint32_t base = uint32_t(count) * 0x3F800000u;
        return (static_cast<unsigned long long>(hi - base) << 23) + (lo - base);
    }
};

// The token with the largest r / e of a thread's elements, given in
// ascending order.  Quotients to a few units in the last place decide all
// but near ties and values near the ends of the range; the exact ones are
// apart from the loop's code.
__device__ __noinline__ bool exactly_ahead(float r1, float e1, float r, float e) {
    return __fdiv_rn(r1, e1) > __fdiv_rn(r, e);
}
struct Race {
    float r = 0.f, e = 1.f, est = 0.f;
    int x = 0;
    __device__ void enter(float r1, float e1, int x1) {
        constexpr float kTiny = 0x1p-100f, kNear = 0x1p-19f;
        float y;
        asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(e1));
        const float est1 = r1 * y;
        bool ahead = est1 > est * (1.f + kNear);
        if (((!ahead && est1 >= est * (1.f - kNear)) || fminf(e1, e) < kTiny || fmaxf(est1, est) < kTiny) && r1 > 0.f)
            ahead = exactly_ahead(r1, e1, r, e);
        if (ahead) {
            r = r1;
            e = e1;
            est = est1;
            x = x1;
        }
    }
    __device__ unsigned long long key() const { return key_of(__fdiv_rn(r, e), x); }
};

constexpr int kNone = 0;     // no child is accepted
constexpr int kPending = -1; // the first is refused and its later siblings wait for Z

struct Shared {
    unsigned long long part[2][kMaxCluster];  // of every block of the cluster: sums or keys, two rounds
    unsigned long long warp[NT / 32];
    float4 node[kMaxT];                       // per node: r and q_i at its token, its uniform number, the token
    uint32_t kids[kMaxT * WORDS];             // the children of every node, as a set of nodes
    int next[kMaxT];                          // per node: its accepted child, or one of
    float z[kMaxT];                           // Z before each refusal at the current node
    int cur, refused, more;                   // where the walk stands; more: a mass is wanted
};

// hold: the block's slice of r and q_i at the current node stays in shared
// memory from one refusal to the next, 8 bytes per token.  (In registers it
// left one block of 512 threads to an SM: 49 us for 48 streams of 50,021
// tokens, 24 us like this.)
template <typename PT>
__global__ void __launch_bounds__(NT, 4) accept_kernel(const PT* __restrict__ p, const PT* __restrict__ q,
                                                       const int32_t* __restrict__ tokens,
                                                       const int32_t* __restrict__ parent,
                                                       const int32_t* __restrict__ lengths,
                                                       const float* __restrict__ u, const float* __restrict__ noise,
                                                       int T, int V, int slice, int hold,
                                                       int32_t* __restrict__ accepted, int32_t* __restrict__ out,
                                                       int32_t* __restrict__ count, int32_t* __restrict__ err) {
    __shared__ Shared sh;
    extern __shared__ float4 sRow[];  // hold: r, then q, of the slice's tiles, [tile][4 elements][thread]
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = blockIdx.x, blocks = gridDim.x, b = blockIdx.y;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int x0 = rank * slice, x1 = min(V, x0 + slice);  // this block's tokens
    cluster.barrier_arrive();  // (waited for below: a block's memory is written by others only once it runs)
    pdl_wait();
    pdl_trigger();  // after the wait: the next kernel may rely on everything before this one
    int bad = 0;
    const int n = stream_len(lengths, b, T, &bad), words = (n + 31) >> 5;
    const size_t nodes = size_t(b) * T;
    const float* e = noise + size_t(b) * V;
    int pa = -1, token = 0;
    float un = 0.f;
    if (t < n) {
        pa = parent[nodes + t];
        token = tokens[nodes + t];
        un = u[nodes + t];
    }
    // the noise is read whatever is accepted: have it on its way during the walk
    for (int x = x0 + t * 32; x < x1; x += NT * 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(e + x));
    for (int j = t; j < n * words; j += NT) sh.kids[j] = 0;
    __syncthreads();
    if (t < n) {
        if (!((t == 0) ? (pa == -1) : (pa >= 0 && pa < t))) {
            bad |= CANOPY_DEVERR_TREE;
            pa = (t == 0) ? -1 : 0;
        }
        float r = 0.f, qx = q ? 0.f : 1.f;
        if (t > 0) {
            if (token >= 0 && token < V) {
                r = to_f(p[(nodes + pa) * V + token]);
                if (q) qx = to_f(q[(nodes + pa) * V + token]);
            } else {
                bad |= CANOPY_DEVERR_TOKEN;
            }
            atomicOr(&sh.kids[pa * words + (t >> 5)], 1u << (t & 31));
        }
        sh.node[t] = make_float4(r, qx, un, __int_as_float(token));
    }
    if (bad && err && rank == 0) raise_err(err, bad);
    cluster.barrier_wait();
    if (n == 0) {
        if (rank == 0) {
            if (t < T) out[nodes + t] = -1;
            if (t == 0) {
                accepted[b] = -1;
                count[b] = 0;
            }
        }
        return;
    }
    __syncthreads();

    // What happens at a node does not depend on how the walk gets there, so
    // every node has a thread for it, as far as it goes without the rows.
    if (!q) {
        // r is gone where an earlier sibling (refused by then) has the same token
        bool gone = false;
        const int first = t < n && t > 0 ? pa * words : 0;
        for (int w = 0; t < n && t > 0 && w <= (t >> 5); ++w) {
            uint32_t set = sh.kids[first + w] & (w == (t >> 5) ? (1u << (t & 31)) - 1 : ~0u);
            for (; set; set &= set - 1)
                gone |= __float_as_int(sh.node[32 * w + __ffs(set) - 1].w) == token;
        }
        __syncthreads();
        if (gone) sh.node[t].x = 0.f;
        __syncthreads();
    }
    if (t < n) {
        int next = kNone;
        float z = 1.f;
        for (int w = t >> 5; w < words && next == kNone; ++w)
            for (uint32_t set = sh.kids[t * words + w]; set && next == kNone; set &= set - 1) {
                const int j = 32 * w + __ffs(set) - 1;
                const float4 nd = sh.node[j];
                if (__fmul_rn(__fmul_rn(nd.z, z), nd.y) < nd.x) {
                    next = j;
                } else if (!q) {
                    z = fmaxf(__fsub_rn(z, nd.x), 0.f);
                } else {
                    bool later = (set & (set - 1)) != 0;
                    for (int v = w + 1; v < words; ++v) later |= sh.kids[t * words + v] != 0;
                    if (later) next = kPending;
                }
            }
        sh.next[t] = next;
    }
    __syncthreads();

    // A value of every block (given by its warp 0), from every block into
    // every block: lane k of warp 0 gets block k's (0 beyond the last).
    int round = 0;
    auto exchange = [&](unsigned long long mine) {
        if (t < blocks) *cluster.map_shared_rank(&sh.part[round][rank], t) = mine;
        cluster.sync();
        const unsigned long long got = t < blocks ? sh.part[round][t] : 0ull;
        round ^= 1;
        return got;
    };

    // r of tile i's elements at `node` after its first m refusals; elements
    // past the slice have r = 0
    int held = -1, applied = 0;  // the node whose rows are held, and the refusals that they carry
    float4* const heldR = sRow + t;
    float4* const heldQ = sRow + (hold ? (slice + kTileTokens - 1) / kTileTokens * (TILE / 4) * NT : 0) + t;
    auto residual = [&](float (&rx)[TILE], int i, int node, int m) {
        float qx[TILE];
        const bool have = held == node;
        const int xt = x0 + i * kTileTokens + t;
        if (have) {
#pragma unroll
            for (int c = 0; c < TILE / 4; ++c) {
                const float4 a = heldR[(i * (TILE / 4) + c) * NT], d = heldQ[(i * (TILE / 4) + c) * NT];
                rx[4 * c] = a.x; rx[4 * c + 1] = a.y; rx[4 * c + 2] = a.z; rx[4 * c + 3] = a.w;
                qx[4 * c] = d.x; qx[4 * c + 1] = d.y; qx[4 * c + 2] = d.z; qx[4 * c + 3] = d.w;
            }
        } else {
            const PT* pr = p + (nodes + node) * V;
            const PT* qr = q + (nodes + node) * V;
#pragma unroll
            for (int k = 0; k < TILE; ++k) rx[k] = xt + k * NT < x1 ? to_f(pr[xt + k * NT]) : 0.f;
            if (m) {
#pragma unroll
                for (int k = 0; k < TILE; ++k) qx[k] = xt + k * NT < x1 ? to_f(qr[xt + k * NT]) : 0.f;
            }
        }
        for (int j = have ? applied : 0; j < m; ++j) {
            const float z = sh.z[j];
#pragma unroll
            for (int k = 0; k < TILE; ++k) rx[k] = fmaxf(__fsub_rn(rx[k], __fmul_rn(z, qx[k])), 0.f);
        }
        if (hold && m) {
#pragma unroll
            for (int c = 0; c < TILE / 4; ++c) {
                heldR[(i * (TILE / 4) + c) * NT] =
                    make_float4(rx[4 * c], rx[4 * c + 1], rx[4 * c + 2], rx[4 * c + 3]);
                if (!have)
                    heldQ[(i * (TILE / 4) + c) * NT] =
                        make_float4(qx[4 * c], qx[4 * c + 1], qx[4 * c + 2], qx[4 * c + 3]);
            }
        }
    };
    const int tiles = (x1 - x0 + kTileTokens - 1) / kTileTokens;

    // The walk, by warp 0.  It pauses where a refused child has a later
    // sibling and Z has to be summed.
    int cur = 0, refused = 0, taken = 0, c = 0;
    float Z = 1.f;
    bool more = false;  // child c of cur is refused, and its mass is in Z now
    while (true) {
        if (warp == 0) {
            while (true) {
                if (!more) {
                    const int next = sh.next[cur];
                    if (next > 0) {
                        if (rank == 0 && lane == 0) out[nodes + taken] = __float_as_int(sh.node[next].w);
                        cur = next;
                        ++taken;
                        continue;
                    }
                    c = cur;
                    refused = 0;
                    Z = 1.f;
                    if (next == kNone && !q) break;
                }
                // cur's next child after c
                more = false;
                int w = (c + 1) >> 5;
                uint32_t set = w < words ? sh.kids[cur * words + w] & (~0u << ((c + 1) & 31)) : 0u;
                while (!set && ++w < words) set = sh.kids[cur * words + w];
                if (!set) break;
                c = 32 * w + __ffs(set) - 1;
                const float4 nd = sh.node[c];
                if (__fmul_rn(__fmul_rn(nd.z, Z), nd.y) < nd.x) {
                    if (rank == 0 && lane == 0) out[nodes + taken] = __float_as_int(nd.w);
                    cur = c;
                    ++taken;
                    continue;
                }
                if (lane == 0) sh.z[refused] = Z;
                ++refused;
                for (int v = 0; v < words; ++v) {  // what is left at the later siblings' tokens
                    const int j = 32 * v + lane;
                    if (j > c && (sh.kids[cur * words + v] >> lane & 1)) {
                        sh.node[j].x = fmaxf(__fsub_rn(sh.node[j].x, __fmul_rn(Z, sh.node[j].y)), 0.f);
                        more = true;
                    }
                }
                more = __any_sync(0xffffffffu, more);
                break;
            }
            if (lane == 0) {
                sh.cur = cur;
                sh.refused = refused;
                sh.more = more;
            }
        }
        __syncthreads();
        if (!sh.more) break;
        // Z = sum of r over the vocabulary, in units of 2^-46
        unsigned long long sum = 0;
#pragma unroll 1
        for (int i = 0; i < tiles; ++i) {
            float rx[TILE];
            residual(rx, i, sh.cur, sh.refused);
            Units units;
#pragma unroll
            for (int k = 0; k < TILE; ++k) units.add(rx[k]);
            sum += units.total();
        }
        if (hold) {
            held = sh.cur;
            applied = sh.refused;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) sh.warp[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            sum = sh.warp[lane & (NT / 32 - 1)];
#pragma unroll
            for (int o = NT / 64; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        sum = exchange(sum);
        if (warp == 0) {
#pragma unroll
            for (int o = kMaxCluster / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            sum = __shfl_sync(0xffffffffu, sum, 0);
            Z = __ll2float_rn(static_cast<long long>(sum)) * 1.4210854715202004e-14f;  // 2^-46
        }
    }
    if (warp == 0 && rank == 0) {  // the walk is over; what follows the accepted tokens
        for (int j = lane; j < T; j += 32)
            if (j > taken) out[nodes + j] = -1;
        if (lane == 0) {
            accepted[b] = cur;
            count[b] = taken + 1;
        }
    }

    // The next token: from r, and where r is zero throughout from p.
    for (int pass = 0; pass < 2; ++pass) {
        const int m = pass == 0 ? sh.refused : 0;
        if (pass == 1) held = -1;
        Race race;
#pragma unroll 1
        for (int i = 0; i < tiles; ++i) {
            const int xt = x0 + i * kTileTokens + t;
            float rx[TILE], ex[TILE];
#pragma unroll
            for (int k = 0; k < TILE; ++k) ex[k] = xt + k * NT < x1 ? e[xt + k * NT] : 1.f;
            residual(rx, i, sh.cur, q ? m : 0);
            if (!q) {
                // all of the last node's children are refused
                for (int w = 0; w < words && pass == 0; ++w)
                    for (uint32_t set = sh.kids[sh.cur * words + w]; set; set &= set - 1) {
                        const int x = __float_as_int(sh.node[32 * w + __ffs(set) - 1].w);
#pragma unroll
                        for (int k = 0; k < TILE; ++k) rx[k] = xt + k * NT == x ? 0.f : rx[k];
                    }
            }
#pragma unroll
            for (int k = 0; k < TILE; ++k) race.enter(rx[k], ex[k], xt + k * NT);
        }
        unsigned long long best = race.key();
#pragma unroll
        for (int o = 16; o; o >>= 1) best = larger(best, __shfl_xor_sync(0xffffffffu, best, o));
        __syncthreads();  // sh.warp is free
        if (lane == 0) sh.warp[warp] = best;
        __syncthreads();
        if (warp == 0) {
            best = sh.warp[lane & (NT / 32 - 1)];
#pragma unroll
            for (int o = NT / 64; o; o >>= 1) best = larger(best, __shfl_xor_sync(0xffffffffu, best, o));
        }
        best = exchange(best);
        if (warp == 0) {
#pragma unroll
            for (int o = kMaxCluster / 2; o; o >>= 1) best = larger(best, __shfl_xor_sync(0xffffffffu, best, o));
            if (rank == 0 && lane == 0 && (best || pass == 1))
                out[nodes + taken] = best ? static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best)) : 0;
            if (lane == 0) sh.more = best == 0;
        }
        __syncthreads();
        if (!sh.more) break;
    }
}

template <typename PT>
cudaError_t launch(const void* p, const void* q, const int32_t* tokens, const int32_t* parent, const int32_t* lengths,
                   const float* u, const float* noise, int T, int B, int V, int32_t* accepted, int32_t* out,
                   int32_t* count, int32_t* err, cudaStream_t st) {
    static OncePerDevice attrs;
    const cudaError_t e = attrs([] {
        const cudaError_t e = cudaFuncSetAttribute(accept_kernel<PT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        return e != cudaSuccess ? e : allow_smem(accept_kernel<PT>, kMaxHeld * 8);
    });
    if (e != cudaSuccess) return e;
    // As many blocks as full slices take, whatever their number: with the next
    // power of two 48 streams of 50,021 tokens take 23.6 us for 22.3, 100 of them
    // 37 for 33, eight (all at once either way) 11.2 for 11.8.
    const int blocks = std::min(kMaxCluster, (V - 1) / kSlice + 1);
    // Longer slices are held too where every block has an SM for itself: four
    // streams of 131,072 tokens 18.2 -> 15.6 us, of 151,936 15.9 -> 15.4; 48 streams
    // would take 57 us for 44, two or three blocks to an SM.
    const int slice = (V - 1) / blocks + 1;
    const bool hold = q && T > 2 && slice <= (size_t(B) * blocks <= kSMs ? kMaxHeld : kSlice);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks, B);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = hold ? size_t(slice + kTileTokens - 1) / kTileTokens * kTileTokens * 8 : 0;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = blocks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, accept_kernel<PT>, static_cast<const PT*>(p), static_cast<const PT*>(q), tokens,
                              parent, lengths, u, noise, T, V, slice, hold, accepted, out, count, err);
}

}  // namespace acc

cudaError_t launch_accept(const void* p, const void* q, int bf16, const int32_t* tokens, const int32_t* parent,
                          const int32_t* lengths, const float* u, const float* noise, int T, int B, int V,
                          int32_t* accepted, int32_t* out, int32_t* count, int32_t* err, cudaStream_t st) {
    if (bf16)
        return acc::launch<__nv_bfloat16>(p, q, tokens, parent, lengths, u, noise, T, B, V, accepted, out, count, err,
                                          st);
    return acc::launch<float>(p, q, tokens, parent, lengths, u, noise, T, B, V, accepted, out, count, err, st);
}

}  // namespace canopy
