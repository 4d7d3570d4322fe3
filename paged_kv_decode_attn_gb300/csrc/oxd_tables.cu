// Block tables and token maps built on the GPU from request lengths (oxd_build_tables).
//
// Three prefix sums over the requests (pages, new tokens, pages to take from the free
// list) and then copies: request b's pages go to indices[indptr[b]..), its new tokens to
// the token maps from qo_indptr[b] on. One launch of one cluster: every CTA scans all
// requests (a tile of 1024 at a time, a thread a request; 12 bytes of each, from L2 but
// for the first reader) and so needs nothing from another, and the cluster's warps share
// the copies: a request's by several warps where there are fewer requests than warps.
// The state (held, taken) may be updated in place: it is written behind a cluster
// barrier that every CTA passes after it has read it.
//
// In a graph 64 requests' step takes 4.1 us, 8 prompts 4.6 (one launch's latencies; 6.8 as
// calls, by the host's time), 1024 requests of 128..16384 tokens 13.1, of 512 pages each 10:
// 16 SMs' instructions, where the bytes would take 0.6 of the whole GPU's. For 1024 requests
// that is a hundredth of the decode step that such tables are for; for one request the
// tables take about as long as it (5.2).
#include <algorithm>
#include <atomic>

#include "oxd_internal.h"
#include "oxd_ptx.cuh"

namespace oxd {
namespace {

constexpr int kTabThreads = 1024;
constexpr int kTabWarps = kTabThreads / 32;
constexpr int kMostTabCtas = 16;
constexpr int kDeviceNoPages = 6;

struct Request {
    int need;     // pages of its tables
    int first;    // where they start in `indices`
    int len, fresh;  // tokens, and how many of them are new
    int token0;   // where those start in the token maps
    int held;     // pages its row lists
    int free0;    // where the pages that it takes start in the free list
};

__device__ __forceinline__ int warp_scan(int x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

__global__ void __launch_bounds__(kTabThreads, 1)
    build_tables_kernel(const __grid_constant__ TablesParams p) {
    __shared__ Request req[kTabThreads];
    __shared__ int sums[3][kTabWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_ctas = gridDim.x, cta = blockIdx.x;  // (the grid is one cluster)
    // launched as a programmatic dependent: nothing in global memory before this
    grid_dependency_wait();
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (cta == 0 && threadIdx.x == 0) *p.last_epoch = p.epoch;
    const int ps = 1 << p.page_shift;
    auto fail = [&](int code) { record_status(p.status, p.epoch, code); };

    // pages of the free list already taken; a count outside it: there are none
    int taken = p.num_free > 0 ? *p.taken : 0;
    const bool bad_taken = taken < 0 || taken > p.num_free;
    if (bad_taken && cta == 0 && threadIdx.x == 0) fail(kDeviceBadPosition);
    const int n_free = bad_taken ? 0 : p.num_free;
    int carry[3] = {0, 0, bad_taken ? 0 : taken};

    for (int b0 = 0; b0 < p.batch; b0 += kTabThreads) {
        const int b = b0 + threadIdx.x;
        Request r = {};
        int lack = 0, held_now = 0;
        if (b < p.batch) {
            const int len = p.lengths[b], fresh = p.new_tokens != nullptr ? p.new_tokens[b] : 0;
            const int held = p.held[b];
            const bool ok = len >= 0 && fresh >= 0 && fresh <= len &&
                            len <= static_cast<int64_t>(p.row_pages) << p.page_shift &&
                            held >= 0 && held <= p.row_pages;
            if (!ok && cta == 0) fail(kDeviceBadPosition);
            r.len = ok ? len : 0;
            r.fresh = ok ? fresh : 0;
            r.held = ok ? held : 0;
            held_now = held;
            r.need = (r.len + ps - 1) >> p.page_shift;
            lack = max(r.need - r.held, 0);
        }
        // ---- exclusive prefix sums
        const int x[3] = {r.need, r.fresh, lack};
        int before[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int s = warp_scan(x[k], lane);
            if (lane == 31) sums[k][warp] = s;
            before[k] = s - x[k];
        }
        __syncthreads();
        int total[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int s = warp_scan(sums[k][lane], lane);
            before[k] += carry[k] + (warp > 0 ? __shfl_sync(0xffffffffu, s, warp - 1) : 0);
            total[k] = __shfl_sync(0xffffffffu, s, 31);
        }
        r.first = before[0];
        r.token0 = before[1];
        r.free0 = before[2];
        req[threadIdx.x] = r;
        // every CTA has read this tile's state, and req is complete
        if (n_ctas > 1)
            cluster_sync_all();
        else
            __syncthreads();
        if (cta == 0 && b < p.batch) {
            p.indptr[b] = min(r.first, p.num_indices);
            p.last_page_len[b] = r.need > 0 ? r.len - ((r.need - 1) << p.page_shift) : 0;
            if (p.qo_indptr != nullptr) p.qo_indptr[b] = min(r.token0, p.num_tokens);
            const int got = min(lack, max(n_free - r.free0, 0));
            p.held_out[b] = held_now + got;
            if (got < lack) fail(kDeviceNoPages);
            if (r.first + r.need > p.num_indices ||
                (p.qo_indptr != nullptr && r.token0 + r.fresh > p.num_tokens))
                fail(kDeviceBadPosition);
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) carry[k] += total[k];

        // ---- the tile's copies: `k` warps a request
        const int n_warps = n_ctas * kTabWarps, w = cta * kTabWarps + warp;
        const int n = min(p.batch - b0, kTabThreads);
        const int k = max(n_warps / n, 1);
        for (int i = w / k; i < n; i += n_warps / k) {
            const Request q = req[i];
            const int seg = (w % k) * 32 + lane, stride = k * 32;
            int32_t* row = p.rows + static_cast<size_t>(b0 + i) * p.row_pages;
            // pages that it has after this step (the free list may end before its need)
            const int have = min(q.need, q.held + max(n_free - q.free0, 0));
            // page j of the request: what its row lists, or the next free page
            auto page_of = [&](int j) {
                if (j < q.held) return row[j];
                const int at = q.free0 + j - q.held;
                return at < n_free ? p.free_pages[at] : -1;
            };
            // pages [dead0, dead1) are out of every new token's sight: behind the sinks, before
            // the first token that a new token's window holds
            const int seen = q.len - max(q.fresh, 1) + 1 - p.window;
            const int dead0 = (p.sinks + ps - 1) >> p.page_shift;
            const int dead1 = p.window > 0 ? max(dead0, max(seen, 0) >> p.page_shift) : dead0;
            auto dead = [&](int j) {
                return static_cast<unsigned>(j - dead0) < static_cast<unsigned>(dead1 - dead0);
            };
            const int fits = min(q.need, max(p.num_indices - q.first, 0));  // entries written
            // (kAhead loads in flight: a request's pages are one chain otherwise; more of them
            // are more code, which the small calls fetch for nothing)
            constexpr int kAhead = 4;
            int32_t* to = p.indices + q.first;
            for (int j0 = seg; j0 < q.need; j0 += kAhead * stride) {
                int pages[kAhead];
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    const int j = j0 + a * stride;
                    pages[a] = j < q.need ? page_of(j) : -1;
                }
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    const int j = j0 + a * stride;
                    if (j >= q.held && j < have) {
                        // (what the free list says, a page or not: the row must not go on
                        // listing what it held there before)
                        row[j] = pages[a];
                        if (pages[a] < 0 || pages[a] >= p.num_pages)
                            fail(kDeviceBadPage);
                        else if (p.refcount != nullptr)
                            p.refcount[pages[a]] = 1;
                    }
                    if (j < fits) to[j] = dead(j) ? -1 : pages[a];
                }
            }
            if (p.token_request != nullptr)
                for (int t = seg; t < q.fresh && q.token0 + t < p.num_tokens; t += stride) {
                    const int pos = q.len - q.fresh + t;
                    p.token_request[q.token0 + t] = b0 + i;
                    p.positions[q.token0 + t] = pos;
                    if (p.slots != nullptr) {
                        const int page = page_of(pos >> p.page_shift);
                        p.slots[q.token0 + t] =
                            page < 0 ? -1
                                     : (static_cast<int64_t>(page) << p.page_shift) + (pos & (ps - 1));
                    }
                }
        }
        __syncthreads();  // req and sums are free again
    }
    if (cta == 0 && threadIdx.x == 0) {
        p.indptr[p.batch] = min(carry[0], p.num_indices);
        if (p.qo_indptr != nullptr) p.qo_indptr[p.batch] = min(carry[1], p.num_tokens);
        if (p.num_free > 0) *p.taken_out = bad_taken ? taken : min(carry[2], p.num_free);
    }
    // entries of the token maps behind the last new token
    if (p.token_request != nullptr)
        for (int t = carry[1] + cta * kTabThreads + threadIdx.x; t < p.num_tokens;
             t += n_ctas * kTabThreads) {
            p.token_request[t] = -1;
            p.positions[t] = -1;
            if (p.slots != nullptr) p.slots[t] = -1;
        }
}

}  // namespace

cudaError_t launch_build_tables(const TablesParams& p, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
    if (bit == 0 || !(done.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(build_tables_kernel,
                                 cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    // a CTA for every 4096 entries, and no more than two requests a warp: 1024 requests of
    // one page on one CTA take 33 us, on 16 5
    const int64_t entries = static_cast<int64_t>(p.num_indices) + p.num_tokens;
    int ctas = 1;
    while (ctas < kMostTabCtas &&
           (ctas * int64_t{4096} < entries || ctas * 2 * kTabWarps < p.batch))
        ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kTabThreads);
    cfg.stream = stream;
    // (the kernel waits for the one before it: what that saves is its launch, 2 us of the
    // smallest calls)
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, build_tables_kernel, p);
}

}  // namespace oxd
