// What the two window decode kernels share (oxd_window_decode.cu for bf16 pages,
// oxd_window_quant.cu for 4-bit ones): which cached tokens a request's query sees,
// and the merge of the states of a CTA's warps and of a cluster's CTAs.
#pragma once

#include <algorithm>
#include <atomic>
#include <mutex>

#include "oxd_internal.h"
#include "oxd_ptx.cuh"

namespace oxd {
namespace {

constexpr int kWinWarps = 4;
constexpr int kWinThreads = kWinWarps * 32;

// The tokens that a request's query (its last token, at position L - 1) sees: the
// first `front` ones (sinks outside the window), then those from `lo` on; `count`
// in all. Visible token v is token v, or v + lo - front from `front` on: chunks of
// visible tokens have no masked ones but past the end of the last.
struct Visible {
    int first;  // offset of the request's first page in `indices`
    int count, front, lo;
    bool bad;   // a table entry outside its bounds: nothing is seen
};

__device__ __forceinline__ Visible visible_tokens(const WindowParams& p, int b) {
    Visible v;
    const int e0 = __ldg(p.indptr + b), e1 = __ldg(p.indptr + b + 1);
    const int last = __ldg(p.last_page_len + b);
    const int pages = e1 - e0;
    v.first = e0;
    v.bad = e0 < 0 || e1 < e0 || e1 > p.num_indices ||
            (pages > 0 && (last < 1 || last > 1 << p.page_shift)) ||
            pages > kMaxWindowTokens >> p.page_shift;
    const int len = v.bad || pages == 0 ? 0 : ((pages - 1) << p.page_shift) + last;
    v.lo = max(len - p.window, 0);
    v.front = p.sinks;
    if (v.lo <= p.sinks) v.lo = v.front = 0;  // the window reaches the sinks: one range
    v.count = v.front + len - v.lo;
    return v;
}

__device__ __forceinline__ uint32_t map_rank(uint32_t local, uint32_t rank) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    return remote;
}

// A cluster's CTAs exchange their states through a region of each: row r of the
// group belongs to rank r % C, which gets the state of rank s at [s][r / C], the
// values f32 [128] and after all of them the log2-sums. (A multiple of 16 bytes:
// one region may follow another.)
__host__ __device__ constexpr int exchange_rows(int rows, int ctas) {
    return (rows + ctas - 1) / ctas * ctas;
}
__host__ __device__ constexpr int exchange_bytes(int rows, int ctas) {
    return ctas > 1 ? (exchange_rows(rows, ctas) * (kHeadDim + 1) * 4 + 15) / 16 * 16 : 0;
}

__device__ __forceinline__ void store_row(const WindowParams& p, size_t row, float4 o, float lse2,
                                          int lane) {
    uint2 w;
    w.x = pack_bf16x2(o.x, o.y);
    w.y = pack_bf16x2(o.z, o.w);
    *reinterpret_cast<uint2*>(p.out + row * kHeadDim + lane * 4) = w;
    if (lane == 0 && p.lse != nullptr) p.lse[row] = lse2 * kLn2;
}

// States (values normalised, log2-sums) of one row weighted together.
struct RowMerge {
    float top = -INFINITY, sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void add(float4 v, float weight) {
        o.x = fmaf(v.x, weight, o.x);
        o.y = fmaf(v.y, weight, o.y);
        o.z = fmaf(v.z, weight, o.z);
        o.w = fmaf(v.w, weight, o.w);
    }
    // The weighted mean, and the log2 of the sum of weights `top` is counted from.
    __device__ __forceinline__ float finish() {
        const float inv = sum != 0.f ? 1.f / sum : 0.f;
        o.x *= inv;
        o.y *= inv;
        o.z *= inv;
        o.w *= inv;
        return sum != 0.f ? top + __log2f(sum) : -INFINITY;
    }
};

// Merges the states that the CTA's warps have dumped and, over a cluster, those of
// its CTAs; writes out and lse of rows [row0, row0 + rows). Every thread of every CTA
// of the cluster calls it, after a barrier behind the dumps (and, over a cluster, a
// cluster barrier since the start).
//   dumps   row r of warp w: 128 f32 at dumps + w * dump_stride + r * 512, the float4
//           at column 4 c stored at c ^ (r & 7); not read where red_l is 0
//   red_m   [warp][red_stride] reference of the row's weights (log2), `offset` above
//           the log2 a weight of 1 stands for; red_l their sums
//   w0, nw  the warps that hold these rows' states
//   xchg    the exchange region's address, of `rows` rows
__device__ __forceinline__ void merge_states(const WindowParams& p, const uint8_t* dumps,
                                             int dump_stride, const float* red_m,
                                             const float* red_l, int red_stride, float offset,
                                             int w0, int nw, size_t row0, int rows, uint8_t* xchg,
                                             int warp, int n_warps, int lane) {
    const int C = p.splits;
    const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int xrows = exchange_rows(rows, C) / C;  // rows a rank owns
    for (int r = warp; r < rows; r += n_warps) {
        RowMerge m;
        for (int w = w0; w < w0 + nw; ++w) m.top = fmaxf(m.top, red_m[w * red_stride + r]);
        const float mu = m.top == -INFINITY ? 0.f : m.top;
        for (int w = w0; w < w0 + nw; ++w) {
            const float l = red_l[w * red_stride + r];
            if (l == 0.f) continue;  // the warp had no token
            const float f = fast_exp2(red_m[w * red_stride + r] - mu);
            m.sum = fmaf(l, f, m.sum);
            m.add(*reinterpret_cast<const float4*>(dumps + w * dump_stride + r * (kHeadDim * 4) +
                                                   ((lane ^ (r & 7)) << 4)),
                  f);
        }
        const float lse2 = m.finish() - offset;
        if (C == 1) {
            store_row(p, row0 + r, m.o, lse2, lane);
        } else {
            const int at = rank * xrows + r / C;
            const uint32_t to = map_rank(smem_addr(xchg), r % C);
            st_cluster_v4(to + (at * kHeadDim + lane * 4) * 4, m.o);
            if (lane == 0) st_cluster_f32(to + (C * xrows * kHeadDim + at) * 4, lse2);
        }
    }
    if (C == 1) return;
    cluster_sync_all();
    const float* vals = reinterpret_cast<const float*>(xchg);
    const float* sums = vals + C * xrows * kHeadDim;
    for (int i = warp; i * C + rank < rows; i += n_warps) {
        RowMerge m;
        for (int s = 0; s < C; ++s) m.top = fmaxf(m.top, sums[s * xrows + i]);
        const float mu = m.top == -INFINITY ? 0.f : m.top;
        for (int s = 0; s < C; ++s) {
            const float z = sums[s * xrows + i];
            if (z == -INFINITY) continue;
            const float f = fast_exp2(z - mu);
            m.sum += f;
            m.add(*reinterpret_cast<const float4*>(vals + (s * xrows + i) * kHeadDim + lane * 4), f);
        }
        const float lse2 = m.finish();
        store_row(p, row0 + i * C + rank, m.o, lse2, lane);
    }
}

// ------------------------------------------------------------------ launching

// How many clusters of c CTAs of a kernel are resident at once, by c; filled once a
// device, with the kernel's attributes set.
struct WindowOccupancy {
    int clusters[kMaxWindowSplits + 1];
};
constexpr int kMaxDevices = 64;

// `which`: the kernel's number among a file's; smem(c): its shared memory in clusters
// of c CTAs, at most `most_smem`.
template <class Smem>
cudaError_t window_kernel_ready(void (*kernel)(WindowParams), int which, int most_smem, Smem smem,
                                const WindowOccupancy** out) {
    static std::atomic<bool> done[3][kMaxDevices];
    static WindowOccupancy table[3][kMaxDevices];
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
    *out = &table[which][dev];
    if (done[which][dev].load(std::memory_order_acquire)) return cudaSuccess;
    std::lock_guard<std::mutex> lk(mu);
    if (done[which][dev].load(std::memory_order_relaxed)) return cudaSuccess;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  most_smem)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) !=
            cudaSuccess)
        return e;
    for (int c = 1; c <= kMaxWindowSplits; ++c) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(c);
        cfg.blockDim = dim3(kWinThreads);
        cfg.dynamicSmemBytes = smem(c);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(c);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if ((e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) != cudaSuccess) return e;
        table[which][dev].clusters[c] = n;
    }
    done[which][dev].store(true, std::memory_order_release);
    return cudaSuccess;
}

// CTAs a stream. As many as still leave all of them resident at once (a cluster sits in
// one GPC, so that fewer large ones fit), each with at least a chunk a warp (`least`
// tokens); more than eight only for four chunks a warp: 16 requests x 1 head of 8192 over
// bf16 take 25 us with 8 and 19 with 12.
// Where that is one, streams of 4096 tokens and more are cut in two all the same, so that
// the last to start end sooner and the SMs are filled more evenly (bf16: 64 x 8 heads of
// 4096 164 -> 158 us). Over 4 bits, where a stream's end costs more of its time, that pays
// up to two waves of the GPU, if the last of them fills at most 85 % of their room (320
// streams of 4096 57 -> 46 us, 440 58 -> 55, 1024 of mixed lengths 202 -> 193; but 608
// 60 -> 66, 1216 115 -> 126): `ends_cost`.
// 4096 is on the safe side: two CTAs against one by window and streams of that length,
//          512 streams   640          800          1000         1600
//   bf16 1024  47/44     60/63        69/67        86/78        129/122 us
//   bf16 2048  83/83     107/118      124/127      156/150      241/236
//   bf16 4096  156/159   203/232      237/248      298/294      466/464
//   bf16 8192  302/316   398/451      466/491      586/581      925/922
//   4 bits 1024  23/19   28/32        33/33        37/34        54/50
//   4 bits 2048  36/34   48/59        52/60        60/61        90/90
//   4 bits 4096  59/60   83/110       92/112       105/114      161/169
//   4 bits 8192  105/114 154/213      172/216      198/219      304/330
// (at 2048 two would gain where a second wave is nearly empty and lose elsewhere; below,
// they lose).
inline int window_splits(const WindowParams& p, const WindowOccupancy& occ, int64_t streams,
                         int least, bool ends_cost, int max_splits) {
    const int64_t most = std::min<int64_t>(
        static_cast<int64_t>(p.window) + p.sinks,
        static_cast<int64_t>(p.num_indices) << p.page_shift);
    const int cap =
        max_splits > 0 ? std::min(max_splits, kMaxWindowSplits) : kMaxWindowSplits;
    int c = 1;
    for (int i = 2; i <= cap; ++i)
        if (occ.clusters[i] >= streams && most >= int64_t{i} * least * (i > 8 ? 4 : 1)) c = i;
    if (c > 1 || cap == 1 || most < 4096) return c;
    const int64_t room = std::max(occ.clusters[1], 1), waves = (streams + room - 1) / room;
    return ends_cost && (waves > 2 || streams * 20 > room * waves * 17) ? 1 : 2;
}

inline cudaError_t window_launch(void (*kernel)(WindowParams), const WindowParams& p,
                                 int64_t streams, int smem, cudaStream_t stream, bool pdl) {
    const int64_t grid = streams * p.splits;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kWinThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (p.splits > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(p.splits);
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace
}  // namespace oxd
