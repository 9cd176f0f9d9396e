// The accepted path's keys and values, moved together in the cache's pages.
//
// The nodes of a draft tree lie behind the stream's tokens in index order, node
// i at place context + i.  The accepted node's root path n_0 = 0 < n_1 < ... <
// n_m stays: node n_k moves to place context + k, and the stream's new length is
// context + m + 1.  In place: n_k >= k, so a move never writes a place that a
// later node of the path still lies at, and within a batch of moves all rows are
// read before any is written.  A block per stream, key head and cache.  Latency:
// 2.7 us in a graph for a few streams, 5 for 48 trees of 64 nodes (8 key heads),
// whose few kilobytes a block take no more.
#include "common.cuh"

namespace canopy {
namespace cc {

constexpr int NT = 256;

struct Args {
    const int32_t *accepted, *parent, *lengths, *table, *context;
    int32_t *context_new, *err;
    uint4 *kc, *vc;
    int T, B, HKV, vecs;  // vecs: 16-byte words a row
    int pages, log_page, max_pages;
};

__global__ void __launch_bounds__(NT) commit_kernel(const Args a) {
    __shared__ int par[kMaxT], path[kMaxT], len;
    __shared__ int64_t to[kMaxT], fro[kMaxT];  // rows in the pages, without the head; -1: stays
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.y, tid = threadIdx.x;
    const bool lead = blockIdx.x == 0;
    int bad = 0;
    const int T = stream_len(a.lengths, b, a.T, &bad);
    if (tid < T) {
        const int p = a.parent[size_t(b) * a.T + tid];
        const bool ok = tid == 0 ? p == -1 : p >= 0 && p < tid;
        if (!ok) bad |= CANOPY_DEVERR_TREE;
        par[tid] = tid == 0 ? -1 : ok ? p : 0;
    }
    int node = a.accepted[b], ctx = a.context[b];
    if (node < -1 || node >= T) {
        bad |= CANOPY_DEVERR_ACCEPTED;
        node = -1;
    }
    if (ctx < 0 && node >= 0) {
        bad |= CANOPY_DEVERR_LENGTH;
        node = -1;
    }
    __syncthreads();
    if (tid == 0) {
        int m = 0;
        for (int n = node; n >= 0; n = par[n]) path[m++] = n;  // from the accepted node up
        len = m;
        if (lead) a.context_new[b] = ctx + m;
    }
    __syncthreads();
    if (tid < len) {
        auto row = [&](int64_t pos) -> int64_t {
            const int64_t entry = pos >> a.log_page;
            const int page = entry < a.max_pages ? a.table[int64_t(b) * a.max_pages + entry] : -1;
            if (page >= 0 && page < a.pages)
                return ((int64_t(page) * a.HKV) << a.log_page) + (pos & ((1 << a.log_page) - 1));
            bad |= CANOPY_DEVERR_PAGE;
            return -1;
        };
        const int n = path[len - 1 - tid];
        const int64_t f = row(int64_t(ctx) + n), t = row(int64_t(ctx) + tid);
        fro[tid] = f;
        to[tid] = n == tid || f < 0 ? -1 : t;
    }
    if (bad && lead && a.err) raise_err(a.err, bad);
    __syncthreads();
    const int h = blockIdx.x >> 1;
    uint4* cache = blockIdx.x & 1 ? a.vc : a.kc;
    constexpr int U = 4;
    const int words = len * a.vecs;
    for (int e0 = 0; e0 < words; e0 += U * NT) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = e0 + u * NT + tid;
            if (e < words && to[e / a.vecs] >= 0)
                x[u] = cache[(fro[e / a.vecs] + (int64_t(h) << a.log_page)) * a.vecs + e % a.vecs];
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = e0 + u * NT + tid;
            if (e < words && to[e / a.vecs] >= 0)
                cache[(to[e / a.vecs] + (int64_t(h) << a.log_page)) * a.vecs + e % a.vecs] = x[u];
        }
        __syncthreads();
    }
}

}  // namespace cc

cudaError_t launch_cache_commit(const int32_t* accepted, const int32_t* parent, const int32_t* lengths, void* kc,
                                void* vc, int bf16, const int32_t* table, int pages, int log_page, int max_pages,
                                const int32_t* context, int T, int B, int HKV, int d, int32_t* context_new,
                                int32_t* err, cudaStream_t st) {
    const cc::Args a = {accepted, parent, lengths, table, context, context_new, err, static_cast<uint4*>(kc),
                        static_cast<uint4*>(vc), T, B, HKV, d * (bf16 ? 2 : 4) / 16, pages, log_page, max_pages};
    return launch_pdl(cc::commit_kernel, dim3(2 * HKV, B), dim3(cc::NT), 0, st, a);
}

}  // namespace canopy
