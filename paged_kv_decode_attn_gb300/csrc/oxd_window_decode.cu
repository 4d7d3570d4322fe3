// Decode with a sliding window over bf16 pages for sm_103a (oxd_window_decode).
//
// For every query row q of a group, over the tokens t that its request's last token
// sees (the last `window` ones and the first `sinks`):
//   x_t = sm_scale q . k_t,  out = sum_t softmax(x)_t v_t,  lse = ln sum_t exp(x_t)
// 512 bytes a token and KV head, about window + sinks tokens whatever the request's
// length: the work is bounded before the lengths are known, so there is no plan, the
// lengths are read here and a captured call follows them.
//
//   * a stream (request, KV head) is one CTA's, or a cluster's: each CTA takes an equal
//     share of the visible tokens and the states are merged through shared memory;
//   * each of a CTA's four warps streams its own 16-token chunks through a private ring
//     of slots, K and V in turn, that it refills by 16-byte cp.async (16 lanes a row; a
//     slot as soon as it is read). The copies go by token, not
//     by page: a chunk starts at any visible token, so the window's edges, the sinks and
//     pages cost no masked tokens, and rows outside the window are never read;
//   * the tokens are the M dimension of mma.sync m16n8k16 (S^T = K Q^T, O^T = V^T P^T),
//     so 8 heads are one N tile and one read of K and V serves up to 16; a larger group
//     is two parts, CTAs of their own that start together and find the rows in L2;
//   * the running maximum is raised only when a score passes it by 2^8, so most chunks
//     need one warp vote and no reduction or rescaling. Weights are rounded to bf16, V's
//     type, for the product on the tensor cores (half a step, 2^-8 of a weight; the sum
//     of weights is not rounded).
//
// HBM bounds it where there is work for all SMs: 256 requests U{128..16384} x 8 heads,
// groups of 8, window 4096, 547 us with other inputs from call to call, 528 to 537 with the
// same ones (7.15 TB/s of reads; a copy, half of it writes, runs at 6.77); 64 x 8 heads of up
// to 512 tokens 23.7 us, 83 % of the copy rate (one wave: 3 us of it a CTA's start and end).
// One request x 8 heads of 1024 tokens 5.6 us, 5.2 in a graph: the chain tables, page index,
// rows, cluster merge. Groups of 17 to 32, in two parts that both copy and read all rows: 16
// x 1 head of 8256 tokens 20.4 us, 49 % (copies, fragments and waits a byte are doubled, over
// 10 warps a SM), 64 x 8 heads of 4096 212, 75 %.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>

#include "oxd_internal.h"
#include "oxd_ptx.cuh"
#include "oxd_window.cuh"

namespace oxd {
namespace {

constexpr int kChunk = 16;  // tokens a warp takes at a time
constexpr int kRowBytes = kHeadDim * 2;
constexpr int kSlotBytes = kChunk * kRowBytes;  // K or V of a chunk
constexpr float kLazy = 8.f;  // log2: how far a score may pass the running maximum

template <int kTiles_>  // N tiles of 8 query heads
struct WCfg {
    static constexpr int kTiles = kTiles_;
    // Slots of a warp's ring, K and V of its chunks in turn, and the resident CTAs a SM
    // that they leave. (Four slots: one CTA fewer, 16 x 1 head of 32 rows 19.1 -> 22.2 us;
    // whole chunks as slots, two of them: 64 x 8 heads of 512 tokens 23.3 -> 27.0.)
    static constexpr int kSlots = 3;
    static constexpr int kCtas = kTiles == 1 ? 4 : 3;
    static constexpr int kRingBytes = kSlots * kSlotBytes;
    static constexpr int kRows = 8 * kTiles;
    static_assert(kRows * kHeadDim * 4 <= kRingBytes, "a warp's state fits its ring");
    // query fragments [k step][tile][lane] of 8 bytes; one tile keeps them in registers
    static constexpr int kQOff = kWinWarps * kRingBytes;
    static constexpr int kQBytes = kTiles > 1 ? 8 * kTiles * 32 * 8 : 0;
    static constexpr int kRedOff = kQOff + kQBytes;  // references and sums of the warps' rows
    static constexpr int kXchgOff = kRedOff + 2 * kWinWarps * kRows * 4;
    static_assert(kXchgOff % 16 == 0, "exchanged rows");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
// D = A * B + D, m16n8k16, bf16 inputs, f32 accumulate.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

// One warp's stream of chunks, the refilling side. Lane t % 16 looks up token t of a
// chunk; the page index of the next chunk to copy is read a chunk ahead.
struct Stream {
    Visible vis;
    int head;
    int next, end;  // next chunk to copy (every fourth is this warp's), end of the CTA's share
    int page;       // page index of this lane's token of it
    uint32_t row;   // its row in the pools, once its K is under way

    __device__ __forceinline__ int token(int c, int lane) const {
        const int v = min(c * kChunk + (lane & 15), vis.count - 1);  // the last once more past it
        return v < vis.front ? v : v - vis.front + vis.lo;
    }
    __device__ __forceinline__ void look_up(const WindowParams& p, int lane) {
        if (next < end)
            page = __ldg(p.indices + vis.first + (token(next, lane) >> p.page_shift));
    }
    // Copies the next K or V into `slot`, if there is one; always one more copy group.
    template <bool kV>
    __device__ __forceinline__ void refill(const WindowParams& p, uint32_t slot, int lane) {
        if (next < end) {
            if constexpr (!kV) {
                // An index outside the pool is recorded and replaced by page 0.
                const bool bad = page < 0 || static_cast<int64_t>(page) >= p.num_pages;
                if (__any_sync(0xffffffffu, bad) && lane == 0)
                    record_status(p.status, p.epoch, kDeviceBadPage);
                const uint32_t pg = bad ? 0u : static_cast<uint32_t>(page);
                const uint32_t at = token(next, lane) & ((1 << p.page_shift) - 1);
                const uint32_t H = p.num_kv_heads;
                // (a pool has fewer than 2^32 rows)
                row = p.layout == 0 ? ((pg << p.page_shift) + at) * H + head
                                    : ((pg * H + head) << p.page_shift) + at;
            }
            const int col = lane & 15;
            const uint8_t* src = (kV ? p.v : p.k) + col * 16;
#pragma unroll
            for (int i = 0; i < kChunk / 2; ++i) {
                const int t = 2 * i + (lane >> 4);
                cp_async16(slot + t * kRowBytes + ((col ^ (t & 7)) << 4),
                           src + static_cast<size_t>(__shfl_sync(0xffffffffu, row, t)) * kRowBytes);
            }
            if constexpr (kV) {
                next += kWinWarps;
                look_up(p, lane);
            }
        }
        cp_async_commit();
    }
};

template <class C>
struct State {
    uint32_t qf[C::kTiles == 1 ? 8 : 1][2];  // one tile's query fragments
    uint32_t q_addr;                         // several tiles' (this lane's), 256 bytes a tile
    float m[C::kTiles][2], l[C::kTiles][2];  // heads 2 tq, 2 tq + 1 of each tile
    float acc[8][C::kTiles][4];              // [16 columns][tile]

    uint32_t pb[C::kTiles][2];               // P^T of the chunk

    // The weights of one chunk from its K at `slot`; its first `left` tokens count.
    __device__ __forceinline__ void scores(uint32_t slot, int left, float scale_log2, int lane) {
        const int g = lane >> 2;
        const int r = lane & 7, mi = lane >> 3;
        // ---- S^T = K Q^T, even and odd steps apart (two chains of dependent MMAs)
        float s[C::kTiles][4], s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int n = 0; n < C::kTiles; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
        const uint32_t krow = slot + ((mi & 1) * 8 + r) * kRowBytes;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            uint32_t a[4];
            ldsm_x4(krow + (((2 * ks + (mi >> 1)) ^ r) << 4), a);
            if constexpr (C::kTiles == 1) {
                mma_bf16(ks & 1 ? s2 : s[0], a, qf[ks][0], qf[ks][1]);
            } else {
#pragma unroll
                for (int n = 0; n < C::kTiles; ++n) {
                    const uint2 b = lds64(q_addr + (ks * C::kTiles + n) * 256);
                    mma_bf16(s[n], a, b.x, b.y);
                }
            }
        }
        // ---- online softmax in the log2 domain
#pragma unroll
        for (int n = 0; n < C::kTiles; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = (C::kTiles == 1 ? s[n][e] + s2[e] : s[n][e]) * scale_log2;
                s[n][e] = g + (e >> 1) * 8 < left ? x : -INFINITY;
            }
        }
        bool raise = false;
#pragma unroll
        for (int n = 0; n < C::kTiles; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                raise = raise || fmaxf(s[n][j], s[n][2 + j]) > m[n][j] + kLazy;
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int n = 0; n < C::kTiles; ++n) {
                float al[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = fmaxf(s[n][j], s[n][2 + j]);
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                    const float top = fmaxf(m[n][j], x);
                    al[j] = fast_exp2(m[n][j] - top);
                    m[n][j] = top;
                    l[n][j] *= al[j];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    acc[i][n][0] *= al[0];
                    acc[i][n][1] *= al[1];
                    acc[i][n][2] *= al[0];
                    acc[i][n][3] *= al[1];
                }
            }
        }
#pragma unroll
        for (int n = 0; n < C::kTiles; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = fast_exp2(s[n][e] - m[n][e & 1]);
            l[n][0] += s[n][0] + s[n][2];
            l[n][1] += s[n][1] + s[n][3];
            // P^T as the B operand: tokens along K, heads along N
            pb[n][0] = transpose_8x8(pack_bf16x2(s[n][0], s[n][1]));
            pb[n][1] = transpose_8x8(pack_bf16x2(s[n][2], s[n][3]));
        }
    }

    // O^T += V^T P^T from the chunk's V at `slot` (tokens past the last are the last
    // once more, weight 0).
    __device__ __forceinline__ void values(uint32_t slot, int lane) {
        const int r = lane & 7, mi = lane >> 3;
        const uint32_t vrow = slot + ((mi >> 1) * 8 + r) * kRowBytes;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t a[4];
            ldsm_x4_trans(vrow + (((2 * i + (mi & 1)) ^ r) << 4), a);
#pragma unroll
            for (int n = 0; n < C::kTiles; ++n) mma_bf16(acc[i][n], a, pb[n][0], pb[n][1]);
        }
    }
};

template <class C>
__global__ void __launch_bounds__(kWinThreads, C::kCtas)
    window_decode_kernel(const __grid_constant__ WindowParams p) {
    extern __shared__ __align__(128) uint8_t base[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (p.splits > 1) cluster_arrive();  // (the others are there once all have)
    // as a programmatic dependent: nothing in global memory before this
    grid_dependency_wait();
    if (threadIdx.x == 0) {
        if (blockIdx.x == 0) *p.last_epoch = p.epoch;
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    // stream: request, KV head, part of the group, the last fastest
    int stream = blockIdx.x / p.splits;
    const int rank = blockIdx.x - stream * p.splits;
    const int parts = (p.group + C::kRows - 1) / C::kRows;
    const int part = stream % parts;
    stream /= parts;
    const int b = stream / p.num_kv_heads;
    const int G = min(C::kRows, p.group - part * C::kRows);  // rows of the part
    const int head = stream - b * p.num_kv_heads;

    // the query rows as B fragments: columns 16 ks + 2 tq, + 1, + 8, + 9 of head 8 n + g
    // (asked for before the tables, on which they do not depend: 8 requests x 8 heads of
    // 1024 tokens 8.6 -> 8.3 us)
    State<C> st;
    const size_t row0 =
        static_cast<size_t>(b) * p.num_qo_heads + head * p.group + part * C::kRows;
    auto query = [&](int ks, int n, int ln) {
        const int g = n * 8 + (ln >> 2);
        if (g >= G) return make_uint2(0u, 0u);
        const uint32_t* src =
            reinterpret_cast<const uint32_t*>(p.q + (row0 + g) * kHeadDim) + ks * 8 + (ln & 3);
        return make_uint2(__ldg(src), __ldg(src + 4));
    };
    if constexpr (C::kTiles == 1) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            const uint2 w = query(ks, 0, lane);
            st.qf[ks][0] = w.x;
            st.qf[ks][1] = w.y;
        }
    } else {
#pragma unroll
        for (int i = warp; i < 8 * C::kTiles; i += kWinWarps)
            *reinterpret_cast<uint2*>(base + C::kQOff + (i * 32 + lane) * 8) =
                query(i / C::kTiles, i % C::kTiles, lane);
        st.q_addr = smem_addr(base) + C::kQOff + lane * 8;
    }

    Stream in;
    in.head = head;
    in.vis = visible_tokens(p, b);
    if (in.vis.bad && threadIdx.x == 0) record_status(p.status, p.epoch, kDeviceBadPosition);
    // this CTA's share of the chunks; the warps take them in turn
    const int n_chunks = (in.vis.count + kChunk - 1) / kChunk;
    const int c0 = static_cast<int>(static_cast<int64_t>(n_chunks) * rank / p.splits) + warp;
    in.end = static_cast<int>(static_cast<int64_t>(n_chunks) * (rank + 1) / p.splits);
    in.next = c0;
    in.page = 0;
    in.look_up(p, lane);

#pragma unroll
    for (int n = 0; n < C::kTiles; ++n) {
        st.m[n][0] = st.m[n][1] = -FLT_MAX;  // (a score of -inf keeps its weight of 0)
        st.l[n][0] = st.l[n][1] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            st.acc[i][n][0] = st.acc[i][n][1] = st.acc[i][n][2] = st.acc[i][n][3] = 0.f;
    }
    const uint32_t ring = smem_addr(base) + warp * C::kRingBytes;
    uint32_t slot = ring;  // of the next K or V
    auto advance = [&]() {
        slot += kSlotBytes;
        if (slot == ring + C::kRingBytes) slot = ring;
    };
    in.refill<false>(p, ring, lane);
    in.refill<true>(p, ring + kSlotBytes, lane);
    in.refill<false>(p, ring + 2 * kSlotBytes, lane);
    static_assert(C::kSlots == 3, "what is copied ahead, and into which slot");
    if constexpr (C::kTiles > 1) __syncthreads();

    // (a slot is refilled with what comes three further on: V behind K, K behind V)
    for (int c = c0; c < in.end; c += kWinWarps) {
        cp_async_wait<C::kSlots - 1>();
        __syncwarp();  // every lane's copies of K have landed
        st.scores(slot, in.vis.count - c * kChunk, p.scale_log2, lane);
        __syncwarp();
        in.refill<true>(p, slot, lane);
        advance();
        cp_async_wait<C::kSlots - 1>();
        __syncwarp();
        st.values(slot, lane);
        __syncwarp();
        in.refill<false>(p, slot, lane);
        advance();
    }
    cp_async_wait<0>();
    __syncwarp();

    // ---- the warps' states through their rings
    float* red_m = reinterpret_cast<float*>(base + C::kRedOff);
    float* red_l = red_m + kWinWarps * C::kRows;
    const int g = lane >> 2, tq = lane & 3;
    uint8_t* dump = base + warp * C::kRingBytes;
#pragma unroll
    for (int n = 0; n < C::kTiles; ++n) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float l = st.l[n][j];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const int row = n * 8 + 2 * tq + j;
            if (g == 0) {
                red_m[warp * C::kRows + row] = st.m[n][j];
                red_l[warp * C::kRows + row] = l;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int col = i * 16 + e * 8 + g;
                    *reinterpret_cast<float*>(dump + row * (kHeadDim * 4) +
                                              (((col >> 2) ^ (row & 7)) << 4) + (col & 3) * 4) =
                        st.acc[i][n][2 * e + j];
                }
        }
    }
    __syncthreads();
    if (p.splits > 1) cluster_wait();
    merge_states(p, base, C::kRingBytes, red_m, red_l, C::kRows, 0.f, 0, kWinWarps, row0, G,
                 base + C::kXchgOff, warp, kWinWarps, lane);
}

template <class C>
cudaError_t launch(WindowParams& p, int max_splits, cudaStream_t stream, bool pdl) {
    // (rows rounded up to a multiple of the CTAs are fewer than this, bytes to 16)
    constexpr int kMostSmem = C::kXchgOff + (C::kRows + kMaxWindowSplits) * (kHeadDim + 1) * 4;
    const int64_t streams = static_cast<int64_t>(p.batch) * p.num_kv_heads *
                            ((p.group + C::kRows - 1) / C::kRows);
    const WindowOccupancy* occ = nullptr;
    const cudaError_t e = window_kernel_ready(
        window_decode_kernel<C>, C::kTiles - 1, kMostSmem,
        [](int c) { return C::kXchgOff + exchange_bytes(C::kRows, c); }, &occ);
    if (e != cudaSuccess) return e;
    p.heads = 1;
    p.splits = window_splits(p, *occ, streams, kWinWarps * kChunk, false, max_splits);
    return window_launch(window_decode_kernel<C>, p, streams,
                         C::kXchgOff + exchange_bytes(std::min(C::kRows, p.group), p.splits),
                         stream, pdl);
}

}  // namespace

cudaError_t launch_window_decode(WindowParams p, int max_splits, cudaStream_t stream, bool pdl) {
    if (p.group <= 8) return launch<WCfg<1>>(p, max_splits, stream, pdl);
    return launch<WCfg<2>>(p, max_splits, stream, pdl);
}

}  // namespace oxd
