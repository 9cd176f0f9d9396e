// The layer over packed prompts in 64-token chunks on tcgen05 tensor cores
// (bf16 q/k/v, dk = dv = 128; fp32 states and accumulation).
//
// canopy page (projects.dotslasha.me/p/canopy.md), "The gated delta rule"
// and "The tree closed form" on a chain: within a chunk, with l_i the sum of
// log2 g up to token i and S the state before it,
//     G_ij = beta_i 2^(l_i - l_j) k_i.k_j (j < i),  C_ij = 2^(l_i - l_j) q_i.k_j (j <= i),
//     W = (I + G)^-1,  M = C W,  R = beta (V - 2^l K S^T),
//     U = W R,  o = scale (2^l Q S^T + M R),
//     S <- 2^l_last S + sum_j 2^(l_last - l_j) u_j k_j^T.
// M and W do not depend on the state.  A first launch forms them for every
// (chunk, value head) at once; a second walks each sequence's chunks in
// order, and there a chunk is three dependent products:
//     [X_Q; X_K] = [Q; K] S^T,   [o; U] = [M; W] R,   S += K^T (2^(l_last - l) U).
// Value columns never meet, so the second launch splits a state's 128 value
// columns into chains of 32.
//
// Precision.  q, k and v are exact bf16; S, R, U, M and W enter their
// products as three bf16 parts that hold the 24 bits of an fp32 value.  The
// right operand's parts stand side by side along N, so that the left operand
// is read once for all of them (16 of K take 46 to 56 cycles for N = 32 to 96,
// 64 for 128 and 96 for 192, and the first is seen after 470), and
// products of parts below 2^-24 of the result are left out, the same ones in
// every shape of a block (below), so that a sequence comes out the same beside
// any others.  (U without W's third part, 2^-18 of its entries off the unit
// diagonal, saves the quarter of a state 250 cycles a chunk and left the state
// up to 6e-6 of its rms off on aligned keys.)  All accumulation is fp32 and S
// itself stays in fp32 across chunks.
//
// Measured (32 value heads of 16 key heads, both launches in a loop): one
// sequence of 16,384 tokens 688 us, of which the walk 545; sixteen of 8,191
// together 229 (81 and 150); eight of 32,768 together 890 to 950, by how
// uneven they are.  The first launch is held by the shared-memory and fp32
// pipes, the walk by the latency of its three products a chunk: with fewer heads
// one sequence takes nearly as long (16,384 tokens of 16, 8 and 4 value heads
// 626, 585 and 565 us, the walk on 64, 32 and 16 SMs).
//
// Chunk slots: with s_b the first token of sequence b, its chunk c is slot
// s_b / 64 + b + c; these never collide, and there are at most N / 64 + B of
// them.
#include "common.cuh"

namespace canopy {

bool make_bf16_row_map(CUtensorMap* m, const void* base, int B, int T, int H, int rows);

namespace pfc {

constexpr int D = 128;            // dk = dv
constexpr int C = 64;             // tokens per chunk
constexpr int QK_BYTES = 32768;   // [Q; K]: 2 atoms of 64 keys x 128 rows x 128 B
constexpr int MW_PART = 16384;    // [M; W]: 128 rows x 128 B
constexpr int MW_BYTES = 3 * MW_PART;
constexpr int GATE_FLOATS = 192;  // 2^l, beta and the decay to the chunk's end, 64 each

__host__ __device__ inline size_t slot_count(int N, int B) { return size_t(N / C) + B; }

constexpr int kMaxRanked = 127;  // sequences that the walk is planned for
constexpr int kSMs = 152;

// Blocks per head that the walk may take beyond one per sequence: about as
// many in all as there are SMs (one without a walk costs its start).
__host__ __device__ inline int more_blocks(int HV) { return HV > kSMs / 4 ? 4 : HV < kSMs / 12 ? 12 : kSMs / HV; }

// The walk's rows, longest first: the sequence, how many blocks share a state
// of it, and its first block; one more for where they end.
struct Row {
    int32_t seq, parts, first, unused;
};

struct WsView {
    int32_t* err;
    Row* rows;
    uint8_t* mw;   // [slot][HV] images of MW_BYTES
    float* gates;  // [slot][HV][GATE_FLOATS]
};

__host__ __device__ inline size_t ws_bytes(int N, int B, int HV) {
    return 256 + ordered_bytes(B) + (kMaxRanked + 1) * sizeof(Row) +
           slot_count(N, B) * HV * (MW_BYTES + GATE_FLOATS * 4);
}
inline WsView ws_view(void* base, int N, int B, int HV) {
    uint8_t* p = static_cast<uint8_t*>(base);
    WsView w;
    w.err = reinterpret_cast<int32_t*>(p);
    w.rows = reinterpret_cast<Row*>(p + 256 + ordered_bytes(B));
    w.mw = p + 256 + ordered_bytes(B) + (kMaxRanked + 1) * sizeof(Row);
    w.gates = reinterpret_cast<float*>(w.mw + slot_count(N, B) * HV * MW_BYTES);
    return w;
}

__device__ inline uint32_t bits(float x) { return __float_as_uint(x); }
__device__ inline uint32_t pack_top(float lo, float hi) { return __byte_perm(bits(lo), bits(hi), 0x7632); }

// fp32 pairs in one 64-bit register.
__device__ inline uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ inline uint64_t pack2(uint32_t x, uint32_t y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
    return r;
}
__device__ inline float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ inline uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ inline uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ inline uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Two fp32 values as three packed bf16 pairs that sum to them exactly (for
// normal parts; each part is the top 16 bits of what is left).
__device__ inline uint64_t rest(uint64_t v, uint32_t packed) {  // v less the pair's bf16 values
    const uint64_t minus1 = 0xBF800000BF800000ull;
    return fma2(pack2(packed << 16, packed & 0xFFFF0000u), minus1, v);
}
__device__ inline void split3(uint64_t v, uint32_t& h, uint32_t& m, uint32_t& l) {
    const float2 x = unpack2(v);
    h = pack_top(x.x, x.y);
    const uint64_t v1 = rest(v, h);
    const float2 y = unpack2(v1);
    m = pack_top(y.x, y.y);
    const float2 z = unpack2(rest(v1, m));
    l = pack_top(z.x, z.y);
}

// Shared-memory matrix descriptor.  K-major 128-byte swizzle: sbo = 1024.
// MN-major: rows of one K index, w bytes of the MN dimension each, in the
// w-byte swizzle; sbo between groups of 8 K indices, lbo between w-byte
// groups of the MN dimension.
__device__ inline uint64_t sdesc(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t swizzle_code) {
    return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(lbo >> 4) << 16) | (uint64_t(sbo >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(swizzle_code) << 61);
}
constexpr uint32_t kMajorA = 1u << 15, kMajorB = 1u << 16;  // instruction descriptor: operand is MN-major

__device__ inline void prefetch_map(const CUtensorMap* m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

__device__ inline void bulk_store(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(reinterpret_cast<uint64_t>(dst)),
                 "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}

// ---------------------------------------------------------------------------
// M, W and the gates of one (chunk, value head): 128 threads, a row of
// [C; I] each.
//
// Decays are products of the gates, no logs (an error of 2^-24 a step, as near
// as logs and their differences come), and underflow to zero quietly: running
// products from the row's own token back in the 32 columns of its own half;
// before those, the product up to there times that from the column to the end
// of its 16 (formed once per head).
//
// The substitution x (I + G) = x0 goes by halves of 32 columns, with
// G = [G00 0; G10 G11]:  x1 (I + G11) = x0_1,  x0 (I + G00) = x0_0 - x1 G10.
// Rows of the first 32 tokens have no x1: their threads take half the columns
// of x1 G10 for the row 32 tokens on.
// All threads read the same row of G at a time.  The kernel's shared memory
// is one array at a fixed, aligned place, so that these addresses are
// constants, or uniform: a 128-bit read at such an address is one pass of the
// shared-memory pipe, at an address in a register it is four, even where all
// threads give the same one (measured: 18,000 cycles of substitution per block
// with four blocks on the SM, now 7,500).

struct PrepSmem {
    static constexpr int QK = 0;                     // later the [M; W] image, over all that follows up to GATE
    static constexpr int P = 68, PW = 52;            // row pitches in floats (no two rows of a store on one bank)
    static constexpr int ROWC = QK;                  // float [64][P]: rows of C, then x1 of M (over Q and K)
    static constexpr int ROWW = ROWC + C * P * 4;    // float [64][PW]: x1 of W, and 16 sums
    static constexpr int G = QK + QK_BYTES;          // float [64][P]
    static constexpr int GATE = G + C * P * 4;       // float [2][64]: g of each head
    static constexpr int BE = GATE + 2 * C * 4;      // float [2][64]: beta
    static constexpr int TAIL = BE + 2 * C * 4;      // float [2][64]: the decay from each token to the end of its 16
    static constexpr int ALL = TAIL + 2 * C * 4;     // float [2][4]: the decay over each 16 tokens
    static constexpr int BAR = ALL + 2 * 4 * 4;      // u64 [2]
    static constexpr int SLOT = BAR + 16;
    static constexpr int TOTAL = SLOT + 8;
    static_assert(BAR % 8 == 0 && GATE >= MW_BYTES && ROWW + C * PW * 4 <= G, "layout");
    static_assert(TOTAL + 1024 <= 56 * 1024, "four blocks per SM");
};

// x (I + G) = x0 for W columns, from the last one down: x[j] -= x[i] G[i][j]
// for j < i, two columns per instruction; G's rows are P floats apart.
template <int W>
__device__ inline void solve(uint64_t (&x)[W / 2], const float* G) {
#pragma unroll
    for (int i = W - 1; i >= 1; --i) {
        const float2 x2 = unpack2(x[i / 2]);
        const float xi = -((i & 1) ? x2.y : x2.x);
        const uint64_t xx = pack2(xi, xi);
        const ulonglong2* row = reinterpret_cast<const ulonglong2*>(G + i * PrepSmem::P);
#pragma unroll
        for (int j4 = 0; j4 < (i + 3) / 4; ++j4) {
            const ulonglong2 g = row[j4];
            x[2 * j4] = fma2(xx, g.x, x[2 * j4]);
            if (4 * j4 + 2 < i) x[2 * j4 + 1] = fma2(xx, g.y, x[2 * j4 + 1]);
        }
    }
}

// z -= y G for 16 columns and the rows of G that y[0 .. 3] belong to.
__device__ inline void take4(uint64_t (&z)[8], const float (&y)[4], const float* G) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const uint64_t yy = pack2(-y[u], -y[u]);
        const ulonglong2* row = reinterpret_cast<const ulonglong2*>(G + u * PrepSmem::P);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const ulonglong2 g = row[j];
            z[2 * j] = fma2(yy, g.x, z[2 * j]);
            z[2 * j + 1] = fma2(yy, g.y, z[2 * j + 1]);
        }
    }
}
// The same for 32 rows, y in shared memory.  Not unrolled: G's addresses stay
// uniform, and with the loop's 800 instructions in line four blocks at
// different places took 9 % of their instructions from beyond the SM's cache,
// 4 % without (the launch for 32,768 tokens 296 against 283 us).
__device__ inline void take32(uint64_t (&z)[8], const float* y, const float* G) {
#pragma unroll 1
    for (int k = 0; k < 32; k += 4) {
        const float4 y4 = *reinterpret_cast<const float4*>(y + k);
        const float yy[4] = {y4.x, y4.y, y4.z, y4.w};
        take4(z, yy, G + k * PrepSmem::P);
    }
}

template <int V>
__device__ inline void read_row(uint64_t (&x)[V], const float* p) {
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
        const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(p + 4 * j);
        x[2 * j] = y.x;
        x[2 * j + 1] = y.y;
    }
}
template <int V>
__device__ inline void write_row(float* p, const uint64_t (&x)[V]) {
#pragma unroll
    for (int j = 0; j < V / 2; ++j) *reinterpret_cast<ulonglong2*>(p + 4 * j) = make_ulonglong2(x[2 * j], x[2 * j + 1]);
}

// The same with the first two parts rounded (ties away), so that they alone
// are within 2^-18.
__device__ inline float near16(float x) { return __uint_as_float((__float_as_uint(x) + 0x8000u) & 0xFFFF0000u); }
__device__ inline void split3_near(float x, float y, uint32_t& h, uint32_t& m, uint32_t& l) {
    const float hx = near16(x), hy = near16(y), x1 = x - hx, y1 = y - hy, mx = near16(x1), my = near16(y1);
    h = pack_top(hx, hy);
    m = pack_top(mx, my);
    l = pack_top(x1 - mx, y1 - my);
}

// Columns 32 half .. + 31 of row `row` of the image's three parts.
__device__ inline void put_half_row(uint8_t* image, int row, int half, const uint64_t (&x)[16]) {
    uint8_t* dst = image + row * 128;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t h[4], m[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 y = unpack2(x[4 * c + e]);
            split3_near(y.x, y.y, h[e], m[e], l[e]);
        }
        const int off = ((4 * half + c) ^ (row & 7)) << 4;
        *reinterpret_cast<uint4*>(dst + off) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(dst + off + MW_PART) = make_uint4(m[0], m[1], m[2], m[3]);
        *reinterpret_cast<uint4*>(dst + off + 2 * MW_PART) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}

// The walk's plan, by one block of 128 threads.  Sequences are walked by four
// blocks per state (quarters), or by one, the longest of them by four and the
// next by two: so many of either as give the least estimate for the launch,
// the largest of the longest walk, (m + 1) times the walk at place 152 m + 1 by
// length (of 152 m + 1 walks some SM has m + 1) and, where they are more than
// the SMs, the work spread over the SMs and a third of a mean walk (what is
// uneven at the end).  The longest walks start first.
constexpr int kWalkCycles = 5000;  // per walk, and
constexpr int kQuarterCycles = 4250, kHalfCycles = 5700, kWholeCycles = 8300;  // per chunk

__device__ inline void plan_walk(const int32_t* starts, int nseq, int N, int HV, int quarters, Row* rows) {
    __shared__ int sLen[128], sSorted[128], sCount[128];
    __shared__ unsigned long long sBest;
    const int tid = threadIdx.x;
    if (tid == 0) sBest = ~0ull;
    sLen[tid] = tid <= nseq ? start_in_range(starts, tid, N) : 0;
    __syncthreads();
    int lo = 0;
    for (int k = 0; k <= tid; ++k) lo = max(lo, sLen[k]);
    const int len = tid < nseq ? max(sLen[tid + 1] - lo, 0) : 0, chunks = (len + C - 1) / C;
    __syncthreads();
    sLen[tid] = len;
    __syncthreads();
    int rank = 0;
    for (int k = 0; k < nseq; ++k) rank += sLen[k] > len || (sLen[k] == len && k < tid);
    if (tid < nseq) sSorted[rank] = chunks;
    __syncthreads();
    // thread by thread: the first nq sequences in quarters, those up to nsplit in halves
    const int more = more_blocks(HV);
    int nq = 0, nsplit = tid;
    for (; 3 * nq <= more && nsplit > more - 3 * nq; ++nq) nsplit -= more - 3 * nq + 1;
    nsplit += nq;
    if (!quarters && 3 * nq <= more && nsplit <= nseq) {
        int i = 0, j = nq, k = nsplit, walks = 0, m = 0;
        float most = 0.f, work = 0.f;
        while (i < nq || j < nsplit || k < nseq) {  // each kind in descending order
            const float quarter = i < nq ? float(sSorted[i]) * kQuarterCycles + kWalkCycles : -1.f;
            const float half = j < nsplit ? float(sSorted[j]) * kHalfCycles + kWalkCycles : -1.f;
            const float whole = k < nseq ? float(sSorted[k]) * kWholeCycles + kWalkCycles : -1.f;
            const float cycles = fmaxf(quarter, fmaxf(half, whole));
            int count = HV;
            if (cycles == quarter) ++i, count *= 4;
            else if (cycles == half) ++j, count *= 2;
            else ++k;
            work += cycles * count;
            walks += count;
            for (; walks > kSMs * m; ++m) most = fmaxf(most, float(m + 1) * cycles);
        }
        if (walks > kSMs) most = fmaxf(most, work / kSMs + 0.35f * work / float(walks));
        if (tid > 0) most *= 1.04f;  // (and it has to be worth it)
        atomicMin(&sBest, static_cast<unsigned long long>(most) << 16 | nq << 8 | nsplit);
    }
    __syncthreads();
    nq = quarters ? nseq : int(sBest >> 8 & 255);
    nsplit = int(sBest & 255);
    auto parts = [&](int r) { return r < nq ? 4 : r < nsplit ? 2 : 1; };
    auto cycles = [&](int r, int n) {
        return float(n) * (parts(r) == 4 ? kQuarterCycles : parts(r) == 2 ? kHalfCycles : kWholeCycles);
    };
    int place = 0;
    if (tid < nseq) {
        const float mine = cycles(rank, chunks);
        for (int k = 0; k < nseq; ++k) {
            const float other = cycles(k, sSorted[k]);
            place += other > mine || (other == mine && k < rank);
        }
        sCount[place] = parts(rank) * HV;
    }
    __syncthreads();
    int first = 0;
    for (int k = 0; k < (tid < nseq ? place : nseq); ++k) first += sCount[k];
    if (tid < nseq) rows[place] = {tid, parts(rank), first, 0};
    else if (tid == nseq) rows[nseq] = {-1, 0, first, 0};
}

__global__ void __launch_bounds__(128, 4)
    prep_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const float* __restrict__ g, const float* __restrict__ beta, const int32_t* __restrict__ starts,
                int N, int B, int HV, int ratio, int heads, int quarters, WsView ws) {
    using P = PrepSmem;
    extern __shared__ __align__(1024) uint8_t sm[];
    float* sG = reinterpret_cast<float*>(sm + P::G);
    float* sGate = reinterpret_cast<float*>(sm + P::GATE);
    float* sBe = reinterpret_cast<float*>(sm + P::BE);
    float* sTail = reinterpret_cast<float*>(sm + P::TAIL);
    float* sAll = reinterpret_cast<float*>(sm + P::ALL);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + P::BAR);
    uint32_t* sTmem = reinterpret_cast<uint32_t*>(sm + P::SLOT);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int per_slot = HV / heads, slot = blockIdx.x / per_slot, h = (blockIdx.x - slot * per_slot) * heads;
    // Tile row r is token (r & 63) ^ flip, of Q for r < 64 and of K beyond:
    // the two warps with the long rows sit on the SM's schedulers 1 and 3 in
    // even blocks, 0 and 2 in odd ones.
    const int flip = (blockIdx.x & 1) * 32;

    if (tid == 0) {
        mbar_init(&bars[0], 1);
        mbar_init(&bars[1], 1);
        fence_mbar_init();
        prefetch_map(&tmQ);
        prefetch_map(&tmK);
    }
    pdl_wait();
    if (blockIdx.x == 0 && B <= kMaxRanked) plan_walk(starts, B, N, HV, quarters, ws.rows);
    // The sequence whose chunk this slot is: the last b with s_b / 64 + b <= slot.
    // With s the running maximum of the starts, the first sequence past the slot
    // is the least max(i, slot + 1 - starts[i] / 64) of all i.
    int past = B;
    for (int b0 = 0; b0 < past; b0 += 128) {
        int least = past;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = b0 + 32 * u + (tid & 31);
            if (i < B) least = min(least, max(i, slot + 1 - start_in_range(starts, i, N) / C));
        }
        past = __reduce_min_sync(0xffffffffu, least);
    }
    const int b = max(past - 1, 0);
    int s0, s1, bad = 0;
    sequence(starts, b, B, N, s0, s1, &bad);
    const int n0 = s0 + C * (slot - (s0 / C + b));
    const int valid = min(C, s1 - n0);  // tokens of this chunk
    if (valid <= 0 || n0 < s0) return;

    if (tid == 0) {
        const int hk = h / ratio;
        mbar_expect_tx(&bars[0], QK_BYTES);
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // 32 tokens of 64 keys: (half, atom)
            const int off = ((32 * (e & 1)) ^ flip) * 128 + (e >> 1) * 16384;
            tma_load_4d(sm + P::QK + off, &tmQ, &bars[0], 64 * (e >> 1), hk, n0 + 32 * (e & 1), 0);
            tma_load_4d(sm + P::QK + off + 8192, &tmK, &bars[0], 64 * (e >> 1), hk, n0 + 32 * (e & 1), 0);
        }
    }
    if (warp == 3) {
        tmem_alloc(sTmem, 64);
        tmem_relinquish();
        tc_fence_before();
    }
    if (tid < C * heads) {  // token tid & 63 of head h + tid / 64; tokens past the end decay and write nothing
        const int n = tid & (C - 1);
        float a = 1.f, be = 0.f;
        if (n < valid) {
            a = g[size_t(n0 + n) * HV + h + tid / C];
            be = beta[size_t(n0 + n) * HV + h + tid / C];
            if (!decay_ok(a, be)) {
                bad |= CANOPY_DEVERR_GATE;
                a = 1.f;
                be = 0.f;
            }
        }
        sGate[tid] = a;
        sBe[tid] = be;
        const int n16 = n & 15;
#pragma unroll
        for (int step = 1; step < 16; step *= 2) {  // a: g of this token and those after it in its 16
            const float y = __shfl_down_sync(0xffffffffu, a, step, 16);
            if (n16 + step < 16) a *= y;
        }
        const float y = __shfl_down_sync(0xffffffffu, a, 1, 16);
        sTail[tid] = n16 < 15 ? y : 1.f;
        if (n16 == 0) sAll[tid >> 4] = a;
    }
    if (bad) raise_err(ws.err, bad);
    __syncthreads();
    // After the wait (the next kernel may rely on everything before this one)
    // and after the allocation: a block of the second launch may take the
    // whole tensor memory and then waits for this kernel.
    pdl_trigger();
    tc_fence_after();
    const uint32_t tmem = *sTmem;
    if (tid == 0 && mbar_wait(&bars[0], 0)) {
        const uint32_t aQK = smem_u32(sm + P::QK);
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
            mma_bf16_ss(tmem, sdesc_sw128(aQK + (ks >> 2) * 16384 + (ks & 3) * 32),
                        sdesc_sw128(aQK + (ks >> 2) * 16384 + 8192 + (ks & 3) * 32), idesc_bf16(128, 64), ks != 0);
        mma_commit(&bars[1]);
    }
    __syncwarp();
    const bool ok = __syncthreads_and(mbar_wait(&bars[1], 0));
    tc_fence_after();

    if (ok) {
        // Row i of C (2^(l_i - l_j) q_i.k_j, j <= i) or G (times beta, j < i).
        const int i = (tid & 63) ^ flip;
        const bool krow = tid >= C;
        const bool live = i < valid;
#pragma unroll 1
        for (int hh = 0; hh < heads; ++hh) {
            const size_t at = size_t(slot) * HV + h + hh;
            const float *gate = sGate + hh * C, *tail = sTail + hh * C, *all = sAll + hh * 4;
            float* rowp = (krow ? sG : reinterpret_cast<float*>(sm + P::ROWC)) + i * P::P;
            float d = krow ? sBe[hh * C + i] : 1.f;  // beta g_{j+1} .. g_i
            const int own = i >= 32 ? 2 : 0;         // the row's half begins at 16 tokens times this
#pragma unroll 1
            for (int kb = own + 1; kb >= own; --kb) {
                uint32_t a[16];
                tmem_ld16(tmem + (uint32_t(warp * 32) << 16) + ((16 * kb) ^ flip), a);
                tmem_wait_ld();
                const int last = i - 16 * kb;  // the row's own column in this 16
                const int lim = !live ? -1 : krow ? last - 1 : last;
#pragma unroll
                for (int u4 = 3; u4 >= 0; --u4) {
                    const float4 g4 = *reinterpret_cast<const float4*>(gate + 16 * kb + 4 * u4);
                    const float gg[4] = {g4.x, g4.y, g4.z, g4.w};
                    float y[4];
#pragma unroll
                    for (int u = 3; u >= 0; --u) {
                        y[u] = 4 * u4 + u <= lim ? d * __uint_as_float(a[4 * u4 + u]) : 0.f;
                        if (4 * u4 + u <= last) d *= gg[u];
                    }
                    *reinterpret_cast<float4*>(rowp + 16 * kb + 4 * u4) = make_float4(y[0], y[1], y[2], y[3]);
                }
            }
            // In the half before the row's own, every column is before the row.
            // (The half after it is not read.)
#pragma unroll 1
            for (int kb = own - 1; kb >= 0; --kb) {
                uint32_t a[16];
                tmem_ld16(tmem + (uint32_t(warp * 32) << 16) + ((16 * kb) ^ flip), a);
                tmem_wait_ld();
#pragma unroll
                for (int u4 = 0; u4 < 4; ++u4) {
                    const float4 t4 = *reinterpret_cast<const float4*>(tail + 16 * kb + 4 * u4);
                    const float tt[4] = {t4.x, t4.y, t4.z, t4.w};
                    float y[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) y[u] = live ? d * tt[u] * __uint_as_float(a[4 * u4 + u]) : 0.f;
                    *reinterpret_cast<float4*>(rowp + 16 * kb + 4 * u4) = make_float4(y[0], y[1], y[2], y[3]);
                }
                d *= all[kb];
            }
            float end = tail[i];  // g_{i+1} .. g_63
#pragma unroll
            for (int m = 1; m < 4; ++m)
                if (16 * m > i) end *= all[m];
            float* gates = ws.gates + at * GATE_FLOATS;
            gates[krow ? C + i : i] = krow ? sBe[hh * C + i] : d;
            if (krow) gates[2 * C + i] = end;
            __syncthreads();
            // Row i of M (from c_i), or of W (from the unit row e_i).
            const bool upper = i >= 32;
            float* up = (krow ? reinterpret_cast<float*>(sm + P::ROWW) : reinterpret_cast<float*>(sm + P::ROWC)) +
                        (i | 32) * (krow ? P::PW : P::P);  // the row itself, or 32 tokens on
            float *sX1 = up + (krow ? 0 : 32), *sSum = up + (krow ? 32 : 0);
            uint64_t x[16];
            if (krow) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    x[j] = pack2(2 * j == (i & 31) ? 1.f : 0.f, 2 * j + 1 == (i & 31) ? 1.f : 0.f);
            } else {
                read_row(x, rowp + (i & 32));
            }
            if (upper) {
                solve<32>(x, sG + 32 * P::P + 32);
                write_row(sX1, x);
            } else {
                solve<32>(x, sG);
            }
            __syncthreads();
            uint64_t z[8] = {};
            if (!krow) read_row(z, upper ? rowp + 16 : sSum);
            if (upper) {
                uint64_t y[8] = {}, part[8];
                take32(z, sX1, sG + 32 * P::P + 16);
                solve<16>(z, sG + 16 * P::P + 16);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 z0 = unpack2(z[2 * k]), z1 = unpack2(z[2 * k + 1]);
                    const float zz[4] = {z0.x, z0.y, z1.x, z1.y};
                    take4(y, zz, sG + (16 + 4 * k) * P::P);
                }
                __syncthreads();
                read_row(part, sSum);
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = add2(y[j], part[j]);
                solve<16>(y, sG);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[j] = y[j];
                    x[8 + j] = z[j];
                }
            } else {
                take32(z, sX1, sG + 32 * P::P);
                write_row(sSum, z);
                __syncthreads();
            }
            uint64_t x1[16] = {};
            if (upper) read_row(x1, sX1);
            __syncthreads();  // everything before the image is done with
            const int row = (i >> 4) * 32 + (i & 15) + (krow ? 16 : 0);
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                put_half_row(sm + P::QK, row, half, x);
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = x1[j];
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncthreads();
            if (tid == 0) {
                bulk_store(ws.mw + at * MW_BYTES, sm + P::QK, MW_BYTES);
                bulk_commit();
                if (hh + 1 < heads) bulk_wait_read<0>();
                else bulk_wait<0>();
            }
            if (hh + 1 < heads) __syncthreads();  // the image is read: its place is free
        }
    } else if (tid == 0) {
        raise_err(ws.err, CANOPY_DEVERR_TIMEOUT);
        mbar_wait(&bars[0], 0);
    }
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc(tmem, 64);
    }
}

// ---------------------------------------------------------------------------
// The walk over a sequence's chunks for NCH chains of NV value columns each
// of one head.  A chain has eight compute warps (TMEM quadrant w & 3, columns
// half w >> 2) and a warp that issues its products; the chains read the same
// [Q; K] and [M; W] tiles, which one more warp copies in.
//
// The tiles' rows alternate by 16 tokens: Q (M), K (W), Q, K, ..., so that
// each TMEM quadrant holds 16 token rows of X_Q (o) and 16 of X_K (U), and
// the rows of K, on the critical path, are shared by the SM's four
// schedulers.  A warp reads 16 of its lanes at a time with all its threads:
// thread t has rows t / 4 and t / 4 + 8, columns 2 (t % 4), + 1 of every 8.

constexpr int WARPS = 8;         // compute warps per chain

enum { CB_X, CB_OU, CB_DS, CB_S, CB_R, CB_U, CB_N };  // a chain's barriers (from CB_S on: its warps arrive)
enum { PB_QK = 0, PB_QKE = 2, PB_MW = 4, PB_MWE = 6, PB_LO = 8, PB_LOE, PB_N };  // tiles: full and empty

// Three shapes of a block:
//   <32, 1>  a quarter of a state: one chain, where there are few states, or
//            one sequence that the others wait for, and a chunk's latency
//            counts (16 warps of 8 columns were no faster);
//   <32, 2>  half a state: two chains half a chunk apart, one's products
//            beside the other's register work;
//   <64, 2>  a whole state: [Q; K] and [M; W] are read once for all of it, and
//            a product is hardly longer for 192 columns than for 96.  What
//            does not fit twice shares its place: R and U the shared memory
//            of S, o and U the tensor memory of X, [M; W] has one buffer, and
//            S itself is in tensor memory.
// A chunk takes about 4,150, 5,400 to 5,900 and 8,200 cycles in them.
template <int NV_, int NCH_>
struct Shape {
    static constexpr int NV = NV_, NCH = NCH_;
    static constexpr int HN = NV * 4 / WARPS;     // value columns of a compute thread
    static constexpr int ROW = NV * 2;            // bytes of one K index of a B operand part
    static constexpr int SPART = D * ROW;         // one part of S
    static constexpr int RPART = C * ROW;         // one part of R (and U)
    static constexpr uint32_t SWIZZLE = NV == 64 ? 2 : 4;  // rows of 128 or 64 bytes, the swizzle of that width
    static constexpr bool TIGHT = NV == 64;
    // TMEM columns of a chain: [X_Q; X_K] and later K^T U in three groups,
    // [o; U] in three, S
    static constexpr uint32_t TX = 0, TO = TIGHT ? 0 : 3 * NV, TS = 3 * NV;
    static constexpr uint32_t COLS = TIGHT ? 4 * NV : 6 * NV;
    static_assert(NCH * COLS <= 512, "tensor memory");
    // shared memory: [Q; K] twice; parts 0 and 1 of [M; W] (twice, or once), part 2
    static constexpr int MW_BUFS = TIGHT ? 1 : 2;
    static constexpr int QK = 0, MW = QK + 2 * QK_BYTES, LO = MW + MW_BUFS * 2 * MW_PART;
    static constexpr int S = LO + MW_PART;
    static constexpr int R = TIGHT ? S : S + NCH * 3 * SPART;  // and U
    static constexpr int CHAIN_R = TIGHT ? 3 * SPART : 3 * RPART;  // from one chain's R to the next's
    static constexpr int BAR = TIGHT ? S + NCH * 3 * SPART : R + NCH * 3 * RPART;
    static constexpr int SLOT = BAR + (PB_N + NCH * CB_N) * 8;
    static constexpr int TOTAL = SLOT + 8;
    static_assert(TOTAL <= 227 * 1024, "shared memory");
};

// 16 TMEM lanes x HN columns: for e = 0, 1 (rows) and c < HN / 8 (groups of 8
// columns) x[(HN / 8) e + c] is the pair at row t / 4 + 8 e, columns
// 8 c + 2 (t % 4); GROUPS column groups, NV apart, summed.
__device__ inline void tmem_ld_16x256b_x2(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
template <typename P, int GROUPS>
__device__ inline void sum_rows16(uint32_t taddr, uint64_t (&x)[P::HN / 4]) {
#pragma unroll
    for (int c2 = 0; c2 < P::HN / 16; ++c2) {
        uint32_t a[GROUPS][8];
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) tmem_ld_16x256b_x2(taddr + g * P::NV + 16 * c2, a[g]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 4 * c + 2 * e;
                uint64_t y = pack2(a[GROUPS - 1][r], a[GROUPS - 1][r + 1]);
#pragma unroll
                for (int g = GROUPS - 2; g >= 0; --g) y = add2(pack2(a[g][r], a[g][r + 1]), y);
                x[P::HN / 8 * e + 2 * c2 + c] = y;
            }
    }
}

// Byte offset of group c of 8 columns of K index k in a part of a B operand.
template <typename P>
__device__ inline int part_offset(int k, int c) {
    return k * P::ROW + ((c ^ (P::NV == 64 ? k & 7 : (k >> 1) & 3)) << 4);
}

// The same values as three parts of a B operand whose K index is the token:
// k0 is the first of the 16 tokens, c0 the first group of 8 columns.
template <typename P>
__device__ inline void put_rows16(uint8_t* base, int k0, int c0, int lane, const uint64_t (&x)[P::HN / 4]) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int c = 0; c < P::HN / 8; ++c) {
            const int k = k0 + (lane >> 2) + 8 * e;
            uint32_t h, m, l;
            split3(x[P::HN / 8 * e + c], h, m, l);
            uint8_t* p = base + part_offset<P>(k, c0 + c) + (lane & 3) * 4;
            *reinterpret_cast<uint32_t*>(p) = h;
            *reinterpret_cast<uint32_t*>(p + P::RPART) = m;
            *reinterpret_cast<uint32_t*>(p + 2 * P::RPART) = l;
        }
}

// Group c of 8 columns of K index k as three parts of a B operand.
template <typename P>
__device__ inline void put_part8(uint8_t* base, int k, int c, const uint64_t* x) {
    uint32_t h[4], m[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split3(x[e], h[e], m[e], l[e]);
    uint8_t* p = base + part_offset<P>(k, c);
    *reinterpret_cast<uint4*>(p) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(p + P::SPART) = make_uint4(m[0], m[1], m[2], m[3]);
    *reinterpret_cast<uint4*>(p + 2 * P::SPART) = make_uint4(l[0], l[1], l[2], l[3]);
}

__device__ inline void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ inline void tmem_put8(uint32_t taddr, const uint64_t* x) {
    uint32_t r[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 y = unpack2(x[e]);
        r[2 * e] = bits(y.x);
        r[2 * e + 1] = bits(y.y);
    }
    tmem_st8(taddr, r);
}
// 8 columns of this lane, summed over the accumulator's three groups.
template <typename P>
__device__ inline void sum8(uint32_t taddr, uint64_t (&x)[4]) {
    uint32_t a[8], b[8], d[8];
    tmem_ld8(taddr, a);
    tmem_ld8(taddr + P::NV, b);
    tmem_ld8(taddr + 2 * P::NV, d);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 4; ++e)
        x[e] = add2(pack2(a[2 * e], a[2 * e + 1]),
                    add2(pack2(b[2 * e], b[2 * e + 1]), pack2(d[2 * e], d[2 * e + 1])));
}

// This block's place in the plan.
struct Turn {
    int seq, parts, index;  // index among the sequence's blocks
};
__device__ inline Turn take_turn(const Row* rows, int nseq, int per_seq) {
    __shared__ Turn sTurn;
    const int tid = threadIdx.x, item = blockIdx.x;
    if (nseq > kMaxRanked) return {item / per_seq, 1, item % per_seq};
    if (tid == 0) sTurn.seq = -1;
    __syncthreads();
    if (tid < nseq) {
        const Row r = rows[tid];
        if (item >= r.first && item < rows[tid + 1].first) sTurn = {r.seq, r.parts, item - r.first};
    }
    __syncthreads();
    return sTurn;
}

struct WalkArgs {
    const __nv_bfloat16* v;
    const float* S0;
    float* S_new;
    const int32_t* starts;
    int N, B, HV, ratio;
    float scale;
    WsView ws;
};

// Value columns v0 .. v0 + NV NCH - 1 of head h of sequence b.
template <typename P, typename OutT>
__device__ __forceinline__ void walk(const CUtensorMap& tmQ, const CUtensorMap& tmK, const WalkArgs& args, OutT* o,
                                     int b, int h, int v0, uint8_t* sm) {
    const __nv_bfloat16* const v = args.v;
    const float* const S0 = args.S0;
    float* const S_new = args.S_new;
    const int N = args.N, HV = args.HV, ratio = args.ratio;
    const float scale = args.scale;
    const WsView& ws = args.ws;
    constexpr int NV = P::NV, NCH = P::NCH, HN = P::HN;
    constexpr uint32_t kCols = 512;
    constexpr int kComputeWarps = WARPS * NCH;
    uint64_t* pb = reinterpret_cast<uint64_t*>(sm + P::BAR);
    uint32_t* sTmem = reinterpret_cast<uint32_t*>(sm + P::SLOT);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        prefetch_map(&tmQ);
        prefetch_map(&tmK);
        for (int i = 0; i < PB_N; ++i)
            mbar_init(&pb[i], (i >= PB_QKE && i < PB_MW) || (i >= PB_MWE && i < PB_LO) || i == PB_LOE ? NCH : 1);
        for (int c = 0; c < NCH; ++c)
            for (int i = 0; i < CB_N; ++i)
                mbar_init(&pb[PB_N + c * CB_N + i], i < CB_S ? 1 : WARPS);
        fence_mbar_init();
    }
    if (warp == kComputeWarps) {
        tmem_alloc(sTmem, kCols);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    int lo, hi, bad = 0;
    sequence(args.starts, b, args.B, N, lo, hi, &bad);
    const int nc = (hi - lo + C - 1) / C;
    const size_t slot0 = size_t(lo / C) + b;
    bool ok = true;
    pdl_trigger();  // after the wait and the allocation

    if (warp == kComputeWarps + NCH) {
        // ---- copies -----------------------------------------------------------
        if (lane == 0) {
            const int hk = h / ratio;
            int qk_n = 0, mw_n = 0, lo_n = 0;  // copies issued
            for (int t = 0; t < nc; ++t) {
                const int s = t & 1, n = lo + C * t;
                const uint32_t freed = ((t >> 1) & 1) ^ 1;  // a fresh barrier passes for parity 1
                const uint8_t* image = ws.mw + ((slot0 + t) * HV + h) * MW_BYTES;
                uint8_t* qk = sm + P::QK + s * QK_BYTES;
                if (!(ok = mbar_wait(&pb[PB_QKE + s], freed))) break;
                mbar_expect_tx(&pb[PB_QK + s], QK_BYTES);
#pragma unroll
                for (int e = 0; e < 8; ++e) {  // 16 tokens of 64 keys: (tokens, atom)
                    uint8_t* dst = qk + (e & 3) * 4096 + (e >> 2) * 16384;
                    tma_load_4d(dst, &tmQ, &pb[PB_QK + s], 64 * (e >> 2), hk, n + 16 * (e & 3), 0);
                    tma_load_4d(dst + 2048, &tmK, &pb[PB_QK + s], 64 * (e >> 2), hk, n + 16 * (e & 3), 0);
                }
                ++qk_n;
                const int ms = P::MW_BUFS == 2 ? s : 0;
                if (!(ok = mbar_wait(&pb[PB_MWE + ms], P::MW_BUFS == 2 ? freed : (t & 1) ^ 1))) break;
                mbar_expect_tx(&pb[PB_MW + ms], 2 * MW_PART);
                bulk_load(sm + P::MW + ms * 2 * MW_PART, image, 2 * MW_PART, &pb[PB_MW + ms]);
                ++mw_n;
                if (!(ok = mbar_wait(&pb[PB_LOE], (t & 1) ^ 1))) break;
                mbar_expect_tx(&pb[PB_LO], MW_PART);
                bulk_load(sm + P::LO, image + 2 * MW_PART, MW_PART, &pb[PB_LO]);
                ++lo_n;
            }
            if (!ok) {  // the copies in flight land before the block ends
                raise_err(ws.err, CANOPY_DEVERR_TIMEOUT);
                for (int e = max(0, qk_n - 2); e < qk_n; ++e) mbar_wait(&pb[PB_QK + (e & 1)], (e >> 1) & 1);
                for (int e = max(0, mw_n - P::MW_BUFS); e < mw_n; ++e) {
                    if (P::MW_BUFS == 2) mbar_wait(&pb[PB_MW + (e & 1)], (e >> 1) & 1);
                    else mbar_wait(&pb[PB_MW], e & 1);
                }
                if (lo_n) mbar_wait(&pb[PB_LO], (lo_n - 1) & 1);
            }
        }
    } else if (warp > kComputeWarps + NCH) {
        // (a block with more warps than this shape has)
    } else if (warp >= kComputeWarps) {
        // ---- the chain's products -----------------------------------------------
        if (lane == 0) {
            const int ch = warp - kComputeWarps;
            uint64_t* cb = pb + PB_N + ch * CB_N;
            const uint32_t tmem = *sTmem + ch * P::COLS;
            const uint32_t aS = smem_u32(sm + P::S + ch * 3 * P::SPART), aR = smem_u32(sm + P::R + ch * P::CHAIN_R);
            const uint32_t aLo = smem_u32(sm + P::LO);
            constexpr uint32_t i3 = idesc_bf16(128, 3 * NV) | kMajorB, i2 = idesc_bf16(128, 2 * NV) | kMajorB,
                               i1 = idesc_bf16(128, NV) | kMajorB;
            for (int t = 0; t < nc; ++t) {
                const int s = t & 1;
                const uint32_t par = t & 1, fpar = (t >> 1) & 1;
                const uint32_t aQK = smem_u32(sm + P::QK + s * QK_BYTES);
                const int ms = P::MW_BUFS == 2 ? s : 0;
                const uint32_t aMW = smem_u32(sm + P::MW + ms * 2 * MW_PART);
                if (!(ok = mbar_wait(&pb[PB_QK + s], fpar))) break;
                if (NCH > 1) {
                    // Half a chunk between the chains, so that one's products
                    // run beside the other's register work: the second starts
                    // a chunk once the first has its X, the first the next
                    // one once the second has its X.
                    uint64_t* other = pb + PB_N + (1 - ch) * CB_N;
                    if ((ch || t) && !(ok = mbar_wait(&other[CB_X], ch ? par : par ^ 1))) break;
                }
                if (!(ok = mbar_wait(&cb[CB_S], par))) break;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    mma_bf16_ss(tmem + P::TX, sdesc(aQK + (ks >> 2) * 16384 + (ks & 3) * 32, 0, 1024, 2),
                                sdesc(aS + ks * 16 * P::ROW, P::SPART, 8 * P::ROW, P::SWIZZLE), i3, ks != 0);
                mma_commit(&cb[CB_X]);
                if (!(ok = mbar_wait(&pb[PB_MW + ms], P::MW_BUFS == 2 ? fpar : par))) break;
                if (!(ok = mbar_wait(&pb[PB_LO], par))) break;
                if (!(ok = mbar_wait(&cb[CB_R], par))) break;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_bf16_ss(tmem + P::TO, sdesc(aMW + ks * 32, 0, 1024, 2),
                                sdesc(aR + ks * 16 * P::ROW, P::RPART, 8 * P::ROW, P::SWIZZLE), i3, ks != 0);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_bf16_ss(tmem + P::TO, sdesc(aMW + MW_PART + ks * 32, 0, 1024, 2),
                                sdesc(aR + ks * 16 * P::ROW, P::RPART, 8 * P::ROW, P::SWIZZLE), i2, 1);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_bf16_ss(tmem + P::TO, sdesc(aLo + ks * 32, 0, 1024, 2),
                                sdesc(aR + ks * 16 * P::ROW, P::RPART, 8 * P::ROW, P::SWIZZLE), i1, 1);
                mma_commit(&cb[CB_OU]);
                mma_commit(&pb[PB_MWE + ms]);
                mma_commit(&pb[PB_LOE]);
                if (!(ok = mbar_wait(&cb[CB_U], par))) break;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_bf16_ss(tmem + P::TX, sdesc(aQK + 2048 + ks * 4096, 16384, 1024, 2),
                                sdesc(aR + ks * 16 * P::ROW, P::RPART, 8 * P::ROW, P::SWIZZLE),
                                i3 | kMajorA, ks != 0);
                mma_commit(&cb[CB_DS]);
                mma_commit(&pb[PB_QKE + s]);
            }
            if (!ok) raise_err(ws.err, CANOPY_DEVERR_TIMEOUT);
        }
    } else {
        // ---- the chain's state, R, U and o ----------------------------------------
        const int ch = warp / WARPS, quad = warp & 3, part = (warp % WARPS) >> 2, c0 = part * (HN / 8);
        uint64_t* cb = pb + PB_N + ch * CB_N;
        uint8_t* sS = sm + P::S + ch * 3 * P::SPART;
        uint8_t* sR = sm + P::R + ch * P::CHAIN_R;
        const uint32_t taddr = *sTmem + ch * P::COLS + (uint32_t(quad * 32) << 16) + part * HN;
        const int krow = quad * 32 + lane;          // key row of S^T
        const int col = v0 + ch * NV + part * HN;   // first value column of this warp
        const int i0 = quad * 16 + (lane >> 2);     // this thread's token rows: i0, i0 + 8
        const int cp = 2 * (lane & 3);              // and column pairs: cp, cp + 8, ...
        const size_t sbase = ((size_t(b) * HV + h) * D + col) * D + krow;
        // S: this lane's key row, HN columns, in registers or (tight) in
        // tensor memory, and always as the next chunk's operand
        uint64_t S[P::TIGHT ? 4 : HN / 2];
        auto held = [&](int g) -> uint64_t* { return S + (P::TIGHT ? 0 : 4 * g); };  // columns 8 g .. 8 g + 7
#pragma unroll
        for (int g = 0; g < HN / 8; ++g) {
            uint64_t* x = held(g);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                x[c] = S0 ? pack2(S0[sbase + size_t(8 * g + 2 * c) * D], S0[sbase + size_t(8 * g + 2 * c + 1) * D])
                          : 0ull;
            put_part8<P>(sS, krow, c0 + g, x);
            if (P::TIGHT) tmem_put8(taddr + P::TS + 8 * g, x);
        }
        if (P::TIGHT) tmem_wait_st();
        if (bad && tid == 0) raise_err(ws.err, bad);

        // chunk t's values and gates for this thread's tokens, one chunk ahead
        constexpr int G8 = HN / 8, NP = 2 * G8;  // column pairs per row, and in all
        uint32_t nv[NP];
        float ng[2], nb[2], nd[2], nlast = 1.f;
        const float* gates = ws.gates + (slot0 * HV + h) * GATE_FLOATS;
        const __nv_bfloat16* vp = v + (size_t(lo + i0) * HV + h) * D + col + cp;
        auto fetch = [&](int t) {
            nlast = gates[C - 1];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                ng[e] = gates[i0 + 8 * e];
                nb[e] = gates[C + i0 + 8 * e];
                nd[e] = gates[2 * C + i0 + 8 * e];
                const bool live = lo + C * t + i0 + 8 * e < hi;
#pragma unroll
                for (int c = 0; c < G8; ++c)
                    nv[G8 * e + c] =
                        live ? __ldg(reinterpret_cast<const uint32_t*>(vp + size_t(8 * e) * HV * D + 8 * c)) : 0u;
            }
            gates += size_t(HV) * GATE_FLOATS;
            vp += size_t(C) * HV * D;
        };
        uint64_t oq[NP];  // 2^l X_Q, then o
        auto store_o = [&](int t) {
            OutT* dst = o + (size_t(lo + C * t + i0) * HV + h) * D + col + cp;
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int c = 0; c < G8; ++c) {
                    const float2 f = unpack2(oq[G8 * e + c]);
                    OutT* p = dst + size_t(8 * e) * HV * D + 8 * c;
                    if (lo + C * t + i0 + 8 * e < hi) {
                        if constexpr (sizeof(OutT) == 4) {
                            *reinterpret_cast<float2*>(p) = f;
                        } else {
                            const __nv_bfloat162 f2 = __floats2bfloat162_rn(f.x, f.y);
                            *reinterpret_cast<__nv_bfloat162*>(p) = f2;
                        }
                    }
                }
        };
        if (nc > 0) fetch(0);
        for (int t = 0; t < nc; ++t) {
            const uint32_t par = t & 1;
            const int left = hi - (lo + C * t);  // tokens from this chunk's first on
            // S is in place as the B operand of the chunk's first product
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&cb[CB_S]);
            const float last = nlast;
            uint64_t x[NP], ga[2], be[2], de[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                ga[e] = pack2(ng[e], ng[e]);
                be[e] = pack2(-nb[e] * ng[e], -nb[e] * ng[e]);
                de[e] = pack2(nd[e], nd[e]);
#pragma unroll
                for (int c = 0; c < G8; ++c)  // beta v
                    x[G8 * e + c] =
                        mul2(pack2(nb[e], nb[e]), pack2(nv[G8 * e + c] << 16, nv[G8 * e + c] & 0xFFFF0000u));
            }
            if (t + 1 < nc) fetch(t + 1);

            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&cb[CB_X], par)))) break;
            tc_fence_after();
            uint64_t y[NP];
            sum_rows16<P, 3>(taddr + (16u << 16) + P::TX, y);
            // R = beta (v - 2^l X_K)
#pragma unroll
            for (int r = 0; r < NP; ++r) x[r] = fma2(be[r / G8], y[r], x[r]);
            if (left < C) {
                // rows past the sequence are zero, and so are their keys in
                // the last product's operand
#pragma unroll
                for (int r = 0; r < NP; ++r)
                    if (i0 + 8 * (r / G8) >= left) x[r] = 0ull;
                if (part < 2) {
                    uint8_t* z = sm + P::QK + (t & 1) * QK_BYTES + part * 16384 + quad * 4096 + 2048;
                    for (int r = lane >> 3; r < 16; r += 4)
                        if (quad * 16 + r >= left)
                            *reinterpret_cast<uint4*>(z + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
            }
            put_rows16<P>(sR, quad * 16, c0, lane, x);
            fence_proxy_async_smem();
            sum_rows16<P, 3>(taddr + P::TX, oq);  // (the last product goes where X is)
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&cb[CB_R]);
#pragma unroll
            for (int r = 0; r < NP; ++r) oq[r] = mul2(ga[r / G8], oq[r]);

            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&cb[CB_OU], par)))) break;
            tc_fence_after();
            sum_rows16<P, 3>(taddr + (16u << 16) + P::TO, x);
#pragma unroll
            for (int r = 0; r < NP; ++r) x[r] = mul2(de[r / G8], x[r]);
            put_rows16<P>(sR, quad * 16, c0, lane, x);  // U, where R was
            fence_proxy_async_smem();
            __syncwarp();
            if (P::TIGHT) {  // (the last product goes where o is)
                sum_rows16<P, 3>(taddr + P::TO, x);
                tc_fence_before();
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(&cb[CB_U]);
            if (!P::TIGHT) sum_rows16<P, 3>(taddr + P::TO, x);
            {
                const uint64_t sc = pack2(scale, scale);
#pragma unroll
                for (int r = 0; r < NP; ++r) oq[r] = mul2(sc, add2(x[r], oq[r]));
            }
            store_o(t);

            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&cb[CB_DS], par)))) break;
            tc_fence_after();
            const uint64_t ll = pack2(last, last);
#pragma unroll
            for (int g = 0; g < HN / 8; ++g) {
                uint64_t* y8 = held(g);
                uint64_t ds[4];
                if (P::TIGHT) {
                    uint32_t r[8];
                    tmem_ld8(taddr + P::TS + 8 * g, r);
                    sum8<P>(taddr + P::TX + 8 * g, ds);
#pragma unroll
                    for (int c = 0; c < 4; ++c) y8[c] = pack2(r[2 * c], r[2 * c + 1]);
                } else {
                    sum8<P>(taddr + P::TX + 8 * g, ds);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) y8[c] = fma2(ll, y8[c], ds[c]);
                put_part8<P>(sS, krow, c0 + g, y8);
                if (P::TIGHT) tmem_put8(taddr + P::TS + 8 * g, y8);
            }
            if (P::TIGHT) tmem_wait_st();
        }
#pragma unroll
        for (int g = 0; g < HN / 8; ++g) {
            uint64_t* x = held(g);
            if (P::TIGHT) {
                uint32_t r[8];
                tmem_ld8(taddr + P::TS + 8 * g, r);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 4; ++c) x[c] = pack2(r[2 * c], r[2 * c + 1]);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float2 z = unpack2(x[c]);
                S_new[sbase + size_t(8 * g + 2 * c) * D] = z.x;
                S_new[sbase + size_t(8 * g + 2 * c + 1) * D] = z.y;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kComputeWarps) {
        tc_fence_after();
        tmem_dealloc(*sTmem, kCols);
    }
}

template <typename OutT>
__global__ void __launch_bounds__(32 * (WARPS + 2), 1)
    walk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, const WalkArgs args,
                OutT* __restrict__ o) {
    extern __shared__ __align__(1024) uint8_t sm[];
    pdl_wait();
    const Turn turn = take_turn(args.ws.rows, args.B, 4 * args.HV);
    walk<Shape<32, 1>>(tmQ, tmK, args, o, turn.seq, turn.index >> 2, (turn.index & 3) * 32, sm);
}

template <typename OutT>
__global__ void __launch_bounds__(32 * (2 * WARPS + 3), 1)
    walk_many_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const WalkArgs args, OutT* __restrict__ o) {
    extern __shared__ __align__(1024) uint8_t sm[];
    pdl_wait();
    const Turn turn = take_turn(args.ws.rows, args.B, args.HV);
    if (turn.seq < 0) return;  // fewer walks than there might be
    if (turn.parts == 1) walk<Shape<64, 2>>(tmQ, tmK, args, o, turn.seq, turn.index, 0, sm);
    else if (turn.parts == 2) walk<Shape<32, 2>>(tmQ, tmK, args, o, turn.seq, turn.index >> 1, (turn.index & 1) * 64, sm);
    else walk<Shape<32, 1>>(tmQ, tmK, args, o, turn.seq, turn.index >> 2, (turn.index & 3) * 32, sm);
}

template <typename OutT>
cudaError_t launch_walk(bool many, const CUtensorMap& mq, const CUtensorMap& mk, const WalkArgs& args, OutT* o,
                        cudaStream_t st) {
    static constexpr int one = Shape<32, 1>::TOTAL, half = Shape<32, 2>::TOTAL, whole = Shape<64, 2>::TOTAL;
    static constexpr int two = half > whole ? half : whole;  // of the shapes that meet in one launch
    static_assert(two >= one, "shared memory");
    static OncePerDevice attrs;
    const cudaError_t e = attrs([] {
        const cudaError_t e = allow_smem(walk_kernel<OutT>, one);
        return e != cudaSuccess ? e : allow_smem(walk_many_kernel<OutT>, two);
    });
    if (e != cudaSuccess) return e;
    const unsigned states = unsigned(args.B) * args.HV;
    if (many)
        return launch_pdl(walk_many_kernel<OutT>, dim3(states + (args.B <= kMaxRanked ? more_blocks(args.HV) * args.HV : 0)),
                          dim3(32 * (2 * WARPS + 3)), two, st, mq, mk, args, o);
    return launch_pdl(walk_kernel<OutT>, dim3(states * 4), dim3(32 * (WARPS + 2)), one, st, mq, mk, args, o);
}

}  // namespace pfc

// (chunk, value head) pairs from which two value heads of a key head share a
// block of the first launch.  With 1,312 pairs of 16 key heads it takes 30.3 us
// with heads alone and 31.2 in twos, with 1,568 35.2 and 34.6, with 2,080 44.5
// and 40.3, with 4,128 81.8 and 77.6.
constexpr size_t kPairFrom = 1400;

// States (sequences times value heads) from which not every one is walked in
// quarters: those fill the SMs up to 38.  Sequences of 2,048 tokens on
// average, one even and three uneven batches, in us, quarters against the
// plan's mixture: 48 states of three sequences 176/158/150/146 and
// 136/167/139/137, 64 of two 183/185/179/170 and 142/154/183/176, 80 of five
// 264/216/225/223 and 207/230/213/209, 96 of three 271/271/271/264 and
// 215/256/197/210, 96 of twelve 275/336/255/253 and 218/346/278/263.
bool many_states(int B, int HV) { return size_t(B) * HV > 38; }

size_t prefill_chunk_ws_bytes(int N, int B, int HV) { return pfc::ws_bytes(N, B, HV); }

cudaError_t launch_prefill_chunk(const void* q, const void* k, const void* v, const float* g, const float* beta,
                                 const float* S0, float* S_new, const int32_t* starts, int N, int B, int H, int HV,
                                 void* o, int o_bf16, float scale, void* workspace, cudaStream_t st) {
    CUtensorMap pq, pk, mq, mk;
    if (!make_bf16_row_map(&pq, q, 1, N, H, 32) || !make_bf16_row_map(&pk, k, 1, N, H, 32) ||
        !make_bf16_row_map(&mq, q, 1, N, H, 16) || !make_bf16_row_map(&mk, k, 1, N, H, 16))
        return cudaErrorInvalidValue;
    const pfc::WsView ws = pfc::ws_view(workspace, N, B, HV);
    const int smem = pfc::PrepSmem::TOTAL;
    static OncePerDevice attrs;
    cudaError_t e = attrs([=] { return allow_smem(pfc::prep_kernel, smem); });
    if (e != cudaSuccess) return e;
    // Two value heads of one key head share a block, its [Q; K] and their
    // product, where there are many blocks all the same.
    const bool many = many_states(B, HV);
    const size_t pairs = pfc::slot_count(N, B) * HV;
    const int heads = (HV / H) % 2 == 0 && pairs >= kPairFrom ? 2 : 1;
    e = launch_pdl(pfc::prep_kernel, dim3(unsigned(pairs / heads)), dim3(128), smem, st, pq, pk, g, beta, starts, N, B,
                   HV, HV / H, heads, !many, ws);
    if (e != cudaSuccess) return e;
    const pfc::WalkArgs args = {static_cast<const __nv_bfloat16*>(v), S0, S_new, starts, N, B, HV, HV / H, scale, ws};
    return o_bf16 ? pfc::launch_walk(many, mq, mk, args, static_cast<__nv_bfloat16*>(o), st)
                  : pfc::launch_walk(many, mq, mk, args, static_cast<float*>(o), st);
}

}  // namespace canopy
