// Decode with a sliding window over a 4-bit paged cache for sm_103a
// (oxd_quant_window_decode): as oxd_window_decode.cu, 144 bytes a token and KV head.
//
// A warp streams chunks of 32 visible tokens (a lane looks one up) through a private
// ring by cp.async: 16-byte pieces of the codes, 8 bytes of scales a token. What it
// does with a chunk is the 4-bit decode's (oxd_decode_quant_state.cuh): tokens as the
// M dimension of mma.sync, one N tile of 8 query heads. A larger group is cut into
// parts of 8 heads, CTAs of their own that start together and find each other's rows
// in L2. In NHD pools a CTA takes two KV heads where there are many (64 bytes of codes a
// head: half a 128-byte line).
//
// 256 requests U{128..16384} x 8 heads, groups of 8, window 4096: 197 us, 81 % of the copy
// rate; between the ends of streams it runs at 94 % (of which 572 instructions a chunk take
// 56 % of the issue slots), a CTA's start and end cost 8 us of one wave. In a graph 8 requests
// x 8 heads of 1024 tokens take 7.4 us, one request 5.5 (latencies; 7.8 and 6.0 as calls).
// Larger groups pay for every part, which unpacks and converts the codes again: 64 x 8 heads
// of 4096 tokens 60 us with groups of 8, 105 with 16, 202 with 32 (floor 45).
#include <algorithm>

#include "oxd_decode_quant_state.cuh"
#include "oxd_internal.h"
#include "oxd_ptx.cuh"
#include "oxd_window.cuh"

namespace oxd {
namespace {

constexpr int kRows = 8;  // query heads of a part

struct QW {
    static constexpr int kSlots = 2;  // of a warp's ring
    static constexpr int kCtas = 4;   // resident a SM
    // slot: K codes | V codes | K scales | V scales of 32 tokens. 16-byte piece i of
    // a token's codes sits at piece i ^ (token / 2 % 4).
    static constexpr int kVOff = kChunk * kCodeBytes;
    static constexpr int kKsOff = 2 * kVOff;
    static constexpr int kVsOff = kKsOff + kChunk * kScaleBytes;
    static constexpr int kSlotBytes = kVsOff + kChunk * kScaleBytes;
    static constexpr int kRingBytes = kSlots * kSlotBytes;
    static constexpr int kQOff = kWinWarps * kRingBytes;  // fragments [head][group][lane]
    static constexpr int kQHeadBytes = kRows * kHeadDim * 2;
    static constexpr int kRawOff = kQOff + 2 * kQHeadBytes;
    static constexpr int kScOff = kRawOff + 2 * kQHeadBytes;  // logit scales [head][kRows]
    static constexpr int kRedOff = kScOff + 2 * kRows * 4;
    static constexpr int kXchgOff = kRedOff + 2 * kWinWarps * kRows * 4;
    static_assert(kRows * kHeadDim * 4 <= kRingBytes, "a warp's state fits its ring");
    static_assert(kXchgOff % 16 == 0 && kQOff % 16 == 0, "16-byte accesses");
};

__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// One warp's stream of chunks, the refilling side: lane t looks up token t of a chunk;
// the page index of the next chunk to copy is read a chunk ahead.
struct Stream {
    Visible vis;
    int head;
    int next, step, end;  // next chunk to copy, and how far this warp's are apart
    int page;

    __device__ __forceinline__ int token(int c, int lane) const {
        const int v = min(c * kChunk + lane, vis.count - 1);  // the last once more past it
        return v < vis.front ? v : v - vis.front + vis.lo;
    }
    __device__ __forceinline__ void look_up(const WindowParams& p, int lane) {
        if (next < end)
            page = __ldg(p.indices + vis.first + (token(next, lane) >> p.page_shift));
    }
    __device__ __forceinline__ void refill(const WindowParams& p, uint32_t slot, int lane) {
        if (next < end) {
            // An index outside the pool is recorded and replaced by page 0.
            const bool bad = page < 0 || static_cast<int64_t>(page) >= p.num_pages;
            if (__any_sync(0xffffffffu, bad) && lane == 0)
                record_status(p.status, p.epoch, kDeviceBadPage);
            const uint32_t pg = bad ? 0u : static_cast<uint32_t>(page);
            const uint32_t at = token(next, lane) & ((1 << p.page_shift) - 1);
            const uint32_t H = p.num_kv_heads;
            // (a pool has fewer than 2^32 rows)
            const uint32_t srow = ((pg * H + head) << p.page_shift) + at;
            const uint32_t row =
                p.layout == 0 ? ((pg << p.page_shift) + at) * H + head : srow;
            cp_async8(slot + QW::kKsOff + lane * kScaleBytes,
                      p.k_scales + static_cast<size_t>(srow) * kRowScales);
            cp_async8(slot + QW::kVsOff + lane * kScaleBytes,
                      p.v_scales + static_cast<size_t>(srow) * kRowScales);
            const uint32_t dst =
                slot + (lane >> 2) * kCodeBytes + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
#pragma unroll
            for (int i = 0; i < kChunk / 8; ++i) {  // eight tokens of K and of V
                const uint32_t r = __shfl_sync(0xffffffffu, row, i * 8 + (lane >> 2));
                const size_t off = static_cast<size_t>(r) * kCodeBytes + (lane & 3) * 16;
                cp_async16(dst + i * 8 * kCodeBytes, p.k + off);
                cp_async16(dst + QW::kVOff + i * 8 * kCodeBytes, p.v + off);
            }
            next += step;
            look_up(p, lane);
        }
        cp_async_commit();
    }
};

__global__ void __launch_bounds__(kWinThreads, QW::kCtas)
    window_quant_kernel(const __grid_constant__ WindowParams p) {
    extern __shared__ __align__(128) uint8_t base[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (p.splits > 1) cluster_arrive();  // (the others are there once all have)
    // as a programmatic dependent: nothing in global memory before this
    grid_dependency_wait();
    if (threadIdx.x == 0) {
        if (blockIdx.x == 0) *p.last_epoch = p.epoch;
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    // stream: request, KV heads, part of the group, the last fastest
    int stream = blockIdx.x / p.splits;
    const int rank = blockIdx.x - stream * p.splits;
    const int parts = (p.group + kRows - 1) / kRows;
    const int part = stream % parts;
    stream /= parts;
    const int head_groups = p.num_kv_heads / p.heads;
    const int b = stream / head_groups;
    const int h0 = (stream - b * head_groups) * p.heads;
    const int rows = min(kRows, p.group - part * kRows);
    const int wl2 = p.heads == 2 ? 1 : 2;  // log2 of the warps a head has
    const int hd = warp >> wl2, w = warp & ((1 << wl2) - 1);

    // query rows, 16 bytes a thread and head, on their way while the tables are read and
    // the first chunks asked for (with the merge of two heads side by side: 256 requests
    // 202 -> 197 us, one 7.9 -> 6.8, 5.5 with a KV head a CTA)
    auto row0 = [&](int head) {
        return static_cast<size_t>(b) * p.num_qo_heads + (h0 + head) * p.group + part * kRows;
    };
    uint4 qv[2];
#pragma unroll
    for (int head = 0; head < 2; ++head)
        if (head < p.heads && threadIdx.x < rows * 16)
            qv[head] = __ldg(reinterpret_cast<const uint4*>(p.q + row0(head) * kHeadDim) +
                             threadIdx.x);

    Stream in;
    in.head = h0 + hd;
    in.vis = visible_tokens(p, b);
    if (in.vis.bad && threadIdx.x == 0) record_status(p.status, p.epoch, kDeviceBadPosition);
    const int n_chunks = (in.vis.count + kChunk - 1) / kChunk;
    const int c0 = static_cast<int>(static_cast<int64_t>(n_chunks) * rank / p.splits) + w;
    in.end = static_cast<int>(static_cast<int64_t>(n_chunks) * (rank + 1) / p.splits);
    in.next = c0;
    in.step = 1 << wl2;
    in.page = 0;
    in.look_up(p, lane);

    const uint32_t ring = smem_addr(base) + warp * QW::kRingBytes;
    for (int i = 0; i < QW::kSlots; ++i) in.refill(p, ring + i * QW::kSlotBytes, lane);
#pragma unroll
    for (int head = 0; head < 2; ++head)
        if (head < p.heads && threadIdx.x < rows * 16)
            *reinterpret_cast<uint4*>(base + QW::kRawOff + head * QW::kQHeadBytes +
                                      threadIdx.x * 16) = qv[head];
    // (convert_query has a thread read the 16 bytes of a head that it wrote)
    float* sc = reinterpret_cast<float*>(base + QW::kScOff);
    for (int head = 0; head < p.heads; ++head)
        convert_query<1>(base + QW::kRawOff + head * QW::kQHeadBytes, rows, p.scale_log2,
                         base + QW::kQOff + head * QW::kQHeadBytes, sc + head * kRows);
    __syncthreads();

    State<QW> st;
    st.set_lane(lane);
    st.init(smem_addr(base) + QW::kQOff + hd * QW::kQHeadBytes, sc + hd * kRows, lane);
    int slot = 0;
    for (int c = c0; c < in.end; c += in.step) {
        cp_async_wait<QW::kSlots - 1>();
        __syncwarp();  // every lane's copies of the chunk have landed
        const uint32_t chunk = ring + slot * QW::kSlotBytes;
        const int left = in.vis.count - c * kChunk;
        if (left >= kChunk)
            st.template consume<false>(chunk, left, lane);
        else
            st.template consume<true>(chunk, left, lane);
        __syncwarp();
        in.refill(p, chunk, lane);
        slot = slot + 1 == QW::kSlots ? 0 : slot + 1;
    }
    cp_async_wait<0>();
    __syncwarp();

    float* red_m = reinterpret_cast<float*>(base + QW::kRedOff);
    float* red_l = red_m + kWinWarps * kRows;
    st.dump(reinterpret_cast<float*>(base + warp * QW::kRingBytes), red_m + warp * kRows,
            red_l + warp * kRows, lane);
    __syncthreads();
    if (p.splits > 1) cluster_wait();
    // (a head's rows by the warps that streamed it)
    merge_states(p, base, QW::kRingBytes, red_m, red_l, kRows, kPOffset, hd << wl2, 1 << wl2,
                 row0(hd), rows, base + QW::kXchgOff + hd * exchange_bytes(rows, p.splits), w,
                 1 << wl2, lane);
}

}  // namespace

cudaError_t launch_window_quant(WindowParams p, int max_splits, cudaStream_t stream, bool pdl) {
    // (rows rounded up to a multiple of the CTAs are fewer than this, bytes to 16)
    constexpr int kMostSmem = QW::kXchgOff + 2 * (kRows + kMaxWindowSplits) * (kHeadDim + 1) * 4;
    const WindowOccupancy* occ = nullptr;
    const cudaError_t e = window_kernel_ready(
        window_quant_kernel, 0, kMostSmem,
        [](int c) { return QW::kXchgOff + 2 * exchange_bytes(kRows, c); }, &occ);
    if (e != cudaSuccess) return e;
    const int64_t streams =
        static_cast<int64_t>(p.batch) * p.num_kv_heads * ((p.group + kRows - 1) / kRows);
    // two KV heads a CTA (NHD) only where the CTAs of one would not all be resident: 76
    // requests x 8 heads of 1024 tokens 24.1 us with two, 21.0 with one, 152 36.4 and 38.8
    p.heads = p.layout == 0 && p.num_kv_heads % 2 == 0 && streams > occ->clusters[1] ? 2 : 1;
    p.splits = window_splits(p, *occ, streams / p.heads, kWinWarps / p.heads * kChunk, true,
                             max_splits);
    return window_launch(window_quant_kernel, p, streams / p.heads,
                         QW::kXchgOff + p.heads * exchange_bytes(std::min(kRows, p.group), p.splits),
                         stream, pdl);
}

}  // namespace oxd
