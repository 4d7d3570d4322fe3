// Decode attention over a 4-bit paged cache for sm_103a (oxd_quant_decode_run),
// groups of up to 8 query heads (oxd_decode_quant_wide.cu: larger ones).
//
// For every query row q of a group and the tokens t of its request
//   x_t = sm_scale * sum_c ks[t,c] (q_c . e2m1(kc[t,c])),  c the four groups of 32
//   out = sum_t softmax(x)_t vs[t,.] e2m1(vc[t,.]),  lse = ln sum_t exp(x_t)
// 144 bytes a token and KV head, 3.6 times fewer than bf16: at the rate HBM
// delivers them (about 42 codes a clock and SM) the codes' conversion and the
// products have to be lean, so
//   * each of a CTA's four warps streams its own 32-token chunks of the CTA's
//     work units through a private ring of shared-memory slots, which it refills
//     itself by 16-byte cp.async (9 a lane and chunk); no barrier between warps
//     until a unit ends. (A page of 16 tokens is 4 bulk copies of 1 KB and 128 B
//     a head, and a bulk copy with lane-wise operands costs about 20 issue
//     slots: refilled by TMA, the copies took 234 of 765 instructions a chunk,
//     and one producer warp a CTA could issue them at half HBM's rate.)
//   * the tokens are the M dimension of mma.sync m16n8k16 (S^T = K Q^T,
//     O^T = V^T P^T), so the unpacked codes are the A fragment as they come out
//     of shared memory, a group of up to 8 heads is one N tile, and neither
//     operand goes back through shared memory;
//   * codes become f16 pairs by cvt.f16x2.e2m1x2, exact. K's scales multiply
//     the F32 sums of each 32-column group (2 packed FMAs for 2 MMAs), V's scales
//     the f16 codes; P goes from the S^T accumulator to the P^T operand by
//     movmatrix;
//   * the running maximum is raised only when a score passes it by 2^4, so most
//     chunks need one warp vote and no reduction or rescaling. P is held in f16
//     as exp2(x - m + 10): at most 2^14, and full precision down to 2^-24 of
//     the largest weight.
// A unit's warp states are merged through the chunks the warps last read;
// split streams leave F32 partial states for the merge kernel, as in the bf16
// decode; a small batch is launched as clusters, one stream a cluster, whose
// first CTA merges the pieces' states from its shared memory.
//
// HBM bounds long streams: 8 heads x 8, 256 requests U{128..16384}, NHD, 414 us
// or 5.9 TB/s, 87 % of the copy rate (HND 403 us); between the ends of units the
// stream runs at 97 %. A unit's end costs 2.9 us (4 heads) to 3.6 (8), a part of
// what log-normal batches pay: 80 to 90 us, 66 to 75 %. One request of 512 tokens,
// 8 KV heads: 8.2 us, dependent latencies of one launch.
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "oxd_decode_quant.cuh"

namespace oxd {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = 32;  // tokens a warp takes at a time

template <int kPs>  // page size
struct QCfg {
    static constexpr int kRows = 8;    // query heads: one N tile
    static constexpr int kStages = 2;  // slots of a warp's ring
    // Resident CTAs a SM, which caps the registers at 128: most instances spill 24
    // to 48 bytes. (Three with 168 registers and longer rings: the same steady rate,
    // slower short streams.)
    static constexpr int kCtas = 4;
    static constexpr int kPageSize = kPs;
    static constexpr int kPagesPerChunk = kPs < kChunk ? kChunk / kPs : 1;
    static constexpr int kRun = 32 / kPagesPerChunk;  // chunks whose pages a window of 32 holds
    // slot: K codes | V codes | K scales | V scales of 32 tokens. 16-byte piece
    // i of a token's codes sits at piece i ^ (token / 2 % 4).
    static constexpr int kVOff = kChunk * kCodeBytes;
    static constexpr int kKsOff = 2 * kVOff;
    static constexpr int kVsOff = kKsOff + kChunk * kScaleBytes;
    static constexpr int kSlotBytes = kVsOff + kChunk * kScaleBytes;
    static_assert(8 * kHeadDim * 4 <= kSlotBytes, "a dumped 8-row state fits a slot");
    // query fragments of up to two heads: [head][group c][lane] 16 bytes,
    // and the next unit's query rows as they come from memory
    static constexpr int kQOff = kWarps * kStages * kSlotBytes;
    static constexpr int kQHeadBytes = kRows * kHeadDim * 2;
    static constexpr int kRawOff = kQOff + 2 * kQHeadBytes;
    static constexpr int kBarOff = kRawOff + 2 * kQHeadBytes;      // their mbarrier
    static constexpr int kScOff = kBarOff + 16;                    // logit scales [head][kRows]
    static constexpr int kRedOff = kScOff + 2 * kRows * 4;
    static constexpr int kFlagOff = kRedOff + 2 * kWarps * 8 * 4;  // dump offset of each warp, units
    static constexpr int kListOff = kFlagOff + 32;
    static constexpr int kSmemBytes = kListOff + kListed * 32;
    // A cluster launch adds the pieces' states in rank 0: [rank][kRows][128]
    // f32 values, then [rank][kRows] log2-sums.
    static constexpr int kClusterOff = (kSmemBytes + 15) / 16 * 16;
    static constexpr int kClusterSums = kClusterOff + kMaxClusterCtas * kRows * kHeadDim * 4;
    static constexpr int kSmemBytesCluster = kClusterSums + kMaxClusterCtas * kRows * 4;
    static_assert(kCtas * (kSmemBytes + 1024) <= 228 * 1024, "the CTAs fit a SM");
};

// Token of MMA row r (0..7) of an 8-token block: 2 <-> 3 and 6 <-> 7 trade
// places, so the four V rows that a quarter of a warp reads at once lie in
// different banks.
__device__ __forceinline__ int row_token(int r) { return r ^ ((r >> 1) & 1); }

using List = UnitList<true>;

// One warp's stream of chunks: the refilling side, up to kStages chunks ahead
// of the consuming one. The warp takes every fourth chunk of a unit (every
// second one where a unit covers two heads). The page
// indices of a run of its chunks sit in the lanes (`win`, the next run in
// `ahead`), and the next unit's first indices are read while the current
// unit's chunks are still being issued.
template <class C>
struct Stream {
    int wl2;                     // log2 of the warps that share a head
    int w, head;                 // this warp's place among them, and which head
    int u_end, unit;             // unit being issued
    int n_pages, n_chunks, first;
    int c;                       // this warp's next chunk of it
    int win_c, win, ahead;       // indices of the chunks from win_c on, and of the next run
    int nx_win;                  // unit + 1's first indices
    // this lane's addresses in page 0 of the unit's head: the 16-byte piece
    // lane % 4 of token lane / 4 of K and V, and the scales of tokens
    // 2 (lane % 16), + 1 of K (lanes 0..15) or V
    const uint8_t* k;
    const uint8_t* v;
    const uint8_t* sc;

    __device__ __forceinline__ int load_window(const int32_t* indices, int x_first, int x_chunks,
                                               int x_pages, int c0, int lane) const {
        const int cc = c0 + ((lane / C::kPagesPerChunk) << wl2);
        const int pg = cc * kChunk / C::kPageSize + lane % C::kPagesPerChunk;
        return cc < x_chunks && pg < x_pages ? __ldg(indices + x_first + pg) : 0;
    }
    // An index outside the pool is recorded and replaced by page 0.
    __device__ __forceinline__ int check(const DecodeParams& p, int i, int lane) const {
        const bool bad = i < 0 || static_cast<int64_t>(i) >= p.num_pages;
        if (__any_sync(0xffffffffu, bad) && lane == 0)
            record_status(p.status, p.epoch, kDeviceBadPage);
        return bad ? 0 : i;
    }
    // Enters `unit`, whose first indices are in nx_win.
    __device__ __forceinline__ void enter(const QuantDecodeParams& qp, const List& units,
                                          int lane) {
        const DecodeParams& p = qp.d;
        const Unit u = units.get(qp, unit);
        n_pages = u.n_pages;
        n_chunks = (u.valid + kChunk - 1) / kChunk;
        first = u.first;
        c = win_c = w;
        const int h = u.valid > 0 ? u.h + head : 0;
        const size_t row = row_index(p.layout, 0, (lane >> 2) % C::kPageSize, h, p.num_kv_heads, C::kPageSize);
        k = qp.k_codes + row * kCodeBytes + (lane & 3) * 16;
        v = qp.v_codes + row * kCodeBytes + (lane & 3) * 16;
        const int st = 2 * (lane & 15) % C::kPageSize;
        sc = reinterpret_cast<const uint8_t*>((lane < 16 ? qp.k_scales : qp.v_scales) +
                                              scale_index(0, st, h, p.num_kv_heads, C::kPageSize));
        win = check(p, nx_win, lane);
        ahead = load_window(p.indices, first, n_chunks, n_pages, w + (C::kRun << wl2), lane);
        load_next_window(qp, units, lane);
    }
    __device__ __forceinline__ void load_next_window(const QuantDecodeParams& qp,
                                                     const List& units, int lane) {
        if (unit + 1 < u_end) {
            const Unit x = units.get(qp, unit + 1);
            nx_win = load_window(qp.d.indices, x.first, (x.valid + kChunk - 1) / kChunk, x.n_pages, w, lane);
        }
    }
    // Issues the next chunk's copies into `slot`, if there is one; always one
    // more copy group. `slot` is the shared address, dst / sdst this lane's
    // offsets in it. Pages past the unit's last are read as page 0.
    __device__ __forceinline__ void refill(const QuantDecodeParams& qp, const List& units,
                                           uint32_t slot, uint32_t dst, uint32_t sdst,
                                           int lane) {
        const DecodeParams& p = qp.d;
        while (unit < u_end && c >= n_chunks) {
            ++unit;
            if (unit < u_end) enter(qp, units, lane);
        }
        if (unit < u_end) {
            if (c - win_c >= C::kRun << wl2) {
                win = check(p, ahead, lane);
                win_c += C::kRun << wl2;
                ahead = load_window(p.indices, first, n_chunks, n_pages, win_c + (C::kRun << wl2), lane);
            }
            const int w0 = ((c - win_c) >> wl2) * C::kPagesPerChunk;
            // bytes of one token and of a page
            const uint32_t tok = p.layout == 0 ? p.num_kv_heads * kCodeBytes : kCodeBytes;
            const uint32_t page_bytes = p.num_kv_heads * (C::kPageSize * kCodeBytes);
            const uint32_t half = C::kPageSize > kChunk ? (c & 1) * kChunk : 0;
#pragma unroll
            for (int i = 0; i < kChunk / 8; ++i) {  // eight tokens of K and of V
                const uint32_t page = __shfl_sync(0xffffffffu, win, w0 + i * 8 / C::kPageSize);
                const size_t off = static_cast<size_t>(page) * page_bytes +
                                   (half + i * 8 % C::kPageSize) * tok;
                cp_async16(slot + dst + i * 8 * kCodeBytes, k + off);
                cp_async16(slot + dst + C::kVOff + i * 8 * kCodeBytes, v + off);
            }
            const uint32_t page =
                __shfl_sync(0xffffffffu, win, w0 + 2 * (lane & 15) / C::kPageSize);
            cp_async16(slot + sdst, sc + static_cast<size_t>(page) * (page_bytes / 8) +
                                        half * kScaleBytes);
            c += 1 << wl2;
        }
        cp_async_commit();
    }
};

template <class C>
struct State {
    uint32_t q;   // this lane's query fragments, 512 bytes from group to group
    float sc[2];  // logit scale (log2) of heads 2 tq, 2 tq + 1, positive
    float mu[2], l[2];  // mu: 10 - the running maximum (inf: none yet)
    float acc[8][4];
    // This lane's offsets in a slot: its ldmatrix row and 16-byte chunk (chunk
    // c + 2 is 32 bytes away in the XOR), its K scales, and the codes and
    // scales of its two V tokens of an 8-token block. Eight tokens on, the
    // swizzle repeats, so everything else is a constant.
    uint32_t k_off, ks_off, v_off[2], vs_off[2];

    __device__ __forceinline__ void set_lane(int lane) {
        const int g = lane >> 2, tq = lane & 3;
        const int kt = ((lane >> 3) & 1) * 8 + row_token(lane & 7);
        k_off = kt * kCodeBytes + (((lane >> 4) ^ ((kt >> 1) & 3)) << 4);
        ks_off = C::kKsOff + row_token(g) * kScaleBytes;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = row_token(2 * tq + i);
            v_off[i] = C::kVOff + t * kCodeBytes + (((g >> 1) ^ ((t >> 1) & 3)) << 4) + (g & 1) * 8;
            vs_off[i] = C::kVsOff + t * kScaleBytes + (g >> 1) * 2;
        }
    }

    // q_addr, sc_row: the head's fragments and logit scales in shared memory.
    __device__ __forceinline__ void init(uint32_t q_addr, const float* sc_row, int lane) {
        q = q_addr + lane * 16;
        const float2 f = *reinterpret_cast<const float2*>(sc_row + 2 * (lane & 3));
        sc[0] = f.x;
        sc[1] = f.y;
        mu[0] = mu[1] = INFINITY;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    }

    // One chunk of 32 tokens at `chunk`, of which the first `left` are there.
    template <bool kPartial>
    __device__ __forceinline__ void consume(uint32_t chunk, int left, int lane) {
        const int tq = lane & 3;
        const int pg = row_token(lane >> 2);
        // ---- S^T = K Q^T
        float s[2][4];
        uint2 ks[2][2];  // [token block][row g, g + 8]: the four groups' f16 scales
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            ks[tb][0] = lds64(chunk + ks_off + tb * 16 * kScaleBytes);
            ks[tb][1] = lds64(chunk + ks_off + (tb * 16 + 8) * kScaleBytes);
        }
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
            uint32_t w[2][4];
#pragma unroll
            for (int tb = 0; tb < 2; ++tb)
                ldsm_x4(chunk + (k_off ^ (c << 4)) + tb * 16 * kCodeBytes, w[tb]);
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
                const int grp = c + cc;
                uint32_t a[2][4], b[2][4];
                float f[2][2];
#pragma unroll
                for (int tb = 0; tb < 2; ++tb) {
                    codes_to_f16(w[tb][2 * cc], a[tb]);
                    codes_to_f16(w[tb][2 * cc + 1], b[tb]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float2 two = f16x2_floats(c ? ks[tb][j].y : ks[tb][j].x);
                        f[tb][j] = cc ? two.y : two.x;
                    }
                }
                const uint4 qf = lds128(q + grp * 512);
#pragma unroll
                for (int tb = 0; tb < 2; ++tb) {
                    float t[4];
                    mma_f16_zero(t, a[tb][0], b[tb][0], a[tb][1], b[tb][1], qf.x, qf.y);
                    mma_f16(t, a[tb][2], b[tb][2], a[tb][3], b[tb][3], qf.z, qf.w);
                    if (grp == 0) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[tb][e] = t[e] * f[tb][e >> 1];
                    } else {
                        fma_pair(s[tb][0], s[tb][1], t[0], t[1], f[tb][0]);
                        fma_pair(s[tb][2], s[tb][3], t[2], t[3], f[tb][1]);
                    }
                }
            }
        }
        // ---- online softmax in the log2 domain: score s counts as s * sc
        bool raise = false;
        float mx[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if constexpr (kPartial) {
#pragma unroll
                for (int tb = 0; tb < 2; ++tb) {
                    if (tb * 16 + pg >= left) s[tb][j] = -INFINITY;
                    if (tb * 16 + 8 + pg >= left) s[tb][2 + j] = -INFINITY;
                }
            }
            mx[j] = fmaxf(fmaxf(s[0][j], s[0][2 + j]), fmaxf(s[1][j], s[1][2 + j]));
            raise = raise || fmaf(mx[j], sc[j], mu[j]) > kPOffset + kLazy;
        }
        if (__any_sync(0xffffffffu, raise)) {
            float al[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float x = mx[j] * sc[j];
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                const float was = kPOffset - mu[j], m = fmaxf(was, x);
                al[j] = m == -INFINITY ? 1.f : fast_exp2(was - m);
                mu[j] = kPOffset - m;
                l[j] *= al[j];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                acc[i][0] *= al[0];
                acc[i][1] *= al[1];
                acc[i][2] *= al[0];
                acc[i][3] *= al[1];
            }
        }
        uint32_t pb[2][2];  // P^T fragments of the two 16-token blocks
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            fma_pairs(s[tb][0], s[tb][1], s[tb][0], s[tb][1], sc[0], sc[1], mu[0], mu[1]);
            fma_pairs(s[tb][2], s[tb][3], s[tb][2], s[tb][3], sc[0], sc[1], mu[0], mu[1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[tb][e] = fast_exp2(s[tb][e]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) l[j] += (s[0][j] + s[0][2 + j]) + (s[1][j] + s[1][2 + j]);
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            pb[tb][0] = transpose_8x8(pack_f16x2(s[tb][0], s[tb][1]));
            pb[tb][1] = transpose_8x8(pack_f16x2(s[tb][2], s[tb][3]));
        }
        // ---- O^T += V^T P^T: a thread's A rows are columns 16 g .. 16 g + 15
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            uint2 x[4];
            uint32_t vs[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // MMA columns 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9
                const int t = tb * 16 + (i >> 1) * 8;
                x[i] = lds64(chunk + v_off[i & 1] + t * kCodeBytes);
                vs[i] = lds16(chunk + vs_off[i & 1] + t * kScaleBytes);
                // rows past the last token may hold anything, NaN scales too
                if (kPartial && t + row_token(2 * tq + (i & 1)) >= left) vs[i] = 0u;
            }
            const uint32_t sa = vs[0] | (vs[1] << 16), sb = vs[2] | (vs[3] << 16);
            constexpr uint32_t kLow = 0x0f0f0f0fu;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t x0 = half ? x[0].y : x[0].x, x1 = half ? x[1].y : x[1].x;
                const uint32_t x2 = half ? x[2].y : x[2].x, x3 = half ? x[3].y : x[3].x;
                // byte i: the even (odd) column 2 i of two neighbouring tokens
                uint32_t a0[4], a1[4], a2[4], a3[4];
                codes_to_f16((x0 & kLow) | ((x1 << 4) & ~kLow), a0);
                codes_to_f16(((x0 >> 4) & kLow) | (x1 & ~kLow), a1);
                codes_to_f16((x2 & kLow) | ((x3 << 4) & ~kLow), a2);
                codes_to_f16(((x2 >> 4) & kLow) | (x3 & ~kLow), a3);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t f0 = mul_f16x2(a0[i], sa), f1 = mul_f16x2(a1[i], sa);
                    const uint32_t f2 = mul_f16x2(a2[i], sb), f3 = mul_f16x2(a3[i], sb);
                    mma_f16(acc[half * 4 + i], f0, f1, f2, f3, pb[tb][0], pb[tb][1]);
                }
            }
        }
    }

    // The accumulator as f32 [8][128] into `dump` (float4 columns XOR-swizzled
    // by the row), the rows' maxima and sums.
    __device__ __forceinline__ void dump(float* dump, float* red_m, float* red_l, int lane) {
        const int g = lane >> 2, tq = lane & 3;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float t = l[j];
            t += __shfl_xor_sync(0xffffffffu, t, 4);
            t += __shfl_xor_sync(0xffffffffu, t, 8);
            t += __shfl_xor_sync(0xffffffffu, t, 16);
            const int row = 2 * tq + j;
            if (g == 0) {
                red_m[row] = kPOffset - mu[j];
                red_l[row] = t;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col4 = (g * 4 + i) ^ (row & 7);
                *reinterpret_cast<float4*>(dump + row * kHeadDim + col4 * 4) =
                    make_float4(acc[2 * i][j], acc[2 * i][2 + j], acc[2 * i + 1][j],
                                acc[2 * i + 1][2 + j]);
            }
        }
    }
};

// kCluster: launched as clusters of p.cluster_c CTAs, one unit each (an
// instantiation of its own, so its code does not weigh on the others).
template <class C, class WL, bool kCluster>
__global__ void __launch_bounds__(kThreads, C::kCtas)
    quant_decode_kernel(const __grid_constant__ QuantDecodeParams qp,
                        const __grid_constant__ WL work) {
    extern __shared__ __align__(128) uint8_t base[];
    const DecodeParams& p = qp.d;
    float* red_m = reinterpret_cast<float*>(base + C::kRedOff);
    float* red_l = red_m + kWarps * 8;
    volatile int* dump_at = reinterpret_cast<volatile int*>(base + C::kFlagOff);  // [warp]
    volatile int* range = dump_at + kWarps;  // first unit, end unit
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    uint64_t* q_bar = reinterpret_cast<uint64_t*>(base + C::kBarOff);
    if (threadIdx.x == 0) {
        mbar_init(q_bar, 1);
        fence_mbar_init();
    }
    if constexpr (kCluster) cluster_arrive();  // (rank 0 is there once all have)
    // as a programmatic dependent: nothing in global memory before this
    grid_dependency_wait();
    // This CTA's units, from the parameter buffer or the workspace. Their range
    // and first entries go through shared memory: every warp passes the same
    // number of barriers, whatever happens to the list meanwhile.
    const int4* list = p.units;
    Unit* shared_list = reinterpret_cast<Unit*>(base + C::kListOff);
    int a = 0, b = 0;
    bool listed = false;
    if constexpr (std::is_same<WL, WorkList>::value) {
        if (list == nullptr) {
            list = work.unit;
            a = work.cta_begin[blockIdx.x];
            b = work.cta_begin[blockIdx.x + 1];
            listed = true;
        }
    }
    int4 it0 = make_int4(0, 0, 0, 0);  // the first unit, beside the range
    if (!listed) {
        const int4 r = __ldg(p.cta_rec + 2 * blockIdx.x);
        it0 = __ldg(p.cta_rec + 2 * blockIdx.x + 1);
        a = r.x;
        b = r.y;
    }
    const bool mine = (p.ws_stamp == nullptr || *p.ws_stamp == p.stamp) && a >= 0 &&
                      b <= p.n_units && a <= b;
    if (!mine) a = b = 0;
    if (threadIdx.x == 0) {
        if (blockIdx.x == 0) {
            *p.last_epoch = p.epoch;
            if (p.clear_stamp != nullptr) *p.clear_stamp = 0ull;
        }
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        if (!mine) record_status(p.status, p.epoch, kDevicePlanMismatch);
        range[0] = a;
        range[1] = b;
    }
    // warp 0 decodes and checks the units in shared memory, the others' check
    // comes when they are reached
    Unit own;
    int4 own_it = make_int4(0, 0, 0, 0);
    const bool have = threadIdx.x < kListed && static_cast<int>(threadIdx.x) < b - a;
    if (have) {
        own_it = threadIdx.x == 0 && !listed ? it0 : list[a + threadIdx.x];
        own = decode_unit<true>(qp, own_it);
        shared_list[threadIdx.x] = own;
    }
    __syncthreads();
    const int u_begin = range[0], u_end = range[1];
    if (!kCluster && u_begin >= u_end) return;
    const List units{shared_list, list, u_begin};

    uint8_t* ring = base + warp * C::kStages * C::kSlotBytes;
    const uint32_t ring_addr = smem_addr(ring);
    const uint32_t dst =
        (lane >> 2) * kCodeBytes + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
    const uint32_t sdst = (lane < 16 ? C::kKsOff : C::kVsOff) + (lane & 15) * 16;
    // The query rows of a unit (contiguous) come as one bulk copy, a unit ahead;
    // one that is not a unit of this plan has none.
    const int G = p.group;
    int q_issued = 0;  // copies issued, as every thread counts them
    auto copy_query = [&](int i) {
        if (i >= u_end) return;
        const Unit u = units.get(qp, i);
        if (u.valid == 0) return;
        if (threadIdx.x == 0) {
            const uint32_t bytes = qp.heads * G * kHeadDim * 2;
            mbar_arrive_expect_tx(q_bar, bytes);
            bulk_load(smem_addr(base) + C::kRawOff,
                      p.q + (static_cast<size_t>(u.b) * p.num_qo_heads + u.h * G) * kHeadDim, bytes,
                      q_bar);
        }
        ++q_issued;
    };
    // Waits for the last of them and makes the fragments. Every thread waits.
    auto take_query = [&](int i) {
        if (i >= u_end || units.get(qp, i).valid == 0) return;
        const uint32_t parity = (q_issued - 1) & 1;
        if (!mbar_wait(q_bar, parity, nullptr, p.wait_ns)) {
            record_status(p.status, p.epoch, kDeviceWaitTimeout);
            mbar_wait(q_bar, parity, nullptr, kWaitTimeoutNs);  // the copy still lands first
        }
        for (int hd = 0; hd < qp.heads; ++hd)
            convert_query<1>(base + C::kRawOff + hd * G * (kHeadDim * 2), G, p.scale_log2,
                             base + C::kQOff + hd * C::kQHeadBytes,
                             reinterpret_cast<float*>(base + C::kScOff) + hd * C::kRows);
    };
    copy_query(u_begin);
    Stream<C> in;
    in.wl2 = qp.heads == 2 ? 1 : 2;
    in.w = warp & ((1 << in.wl2) - 1);
    in.head = warp >> in.wl2;
    in.u_end = u_end;
    in.unit = u_begin - 1;
    in.load_next_window(qp, units, lane);  // the first unit's
    in.c = in.n_chunks = 0;
    for (int i = 0; i < C::kStages; ++i)
        in.refill(qp, units, ring_addr + i * C::kSlotBytes, dst, sdst, lane);
    if (have && !tables_match(p, own, own_it)) record_status(p.status, p.epoch, kDevicePlanMismatch);
    take_query(u_begin);
    __syncthreads();
    copy_query(u_begin + 1);

    if constexpr (kCluster) cluster_wait();
    State<C> st;
    st.set_lane(lane);
    const uint32_t q_addr = smem_addr(base) + C::kQOff + in.head * C::kQHeadBytes;
    const float* sc_row = reinterpret_cast<const float*>(base + C::kScOff) + in.head * C::kRows;
    int slot = 0;  // of the next chunk
    for (int ui = u_begin; ui < u_end; ++ui) {
        const Unit u = units.get(qp, ui);
        if (ui - u_begin >= kListed && threadIdx.x == 0 && !tables_match(p, u, __ldg(list + ui)))
            record_status(p.status, p.epoch, kDevicePlanMismatch);
        const int n_chunks = (u.valid + kChunk - 1) / kChunk;
        int held = -1;  // the slot of the warp's last chunk, not refilled yet
        st.init(q_addr, sc_row, lane);
        for (int c = in.w; c < n_chunks; c += 1 << in.wl2) {
            cp_async_wait<C::kStages - 1>();
            __syncwarp();  // every lane's copies of the chunk have landed
            const uint32_t chunk = ring_addr + slot * C::kSlotBytes;
            const int left = u.valid - c * kChunk;
            if (left >= kChunk)
                st.template consume<false>(chunk, left, lane);
            else
                st.template consume<true>(chunk, left, lane);
            __syncwarp();
            if (c + (1 << in.wl2) < n_chunks)
                in.refill(qp, units, chunk, dst, sdst, lane);
            else
                held = slot;
            slot = slot + 1 == C::kStages ? 0 : slot + 1;
        }
        // ---- merge the warps' states, each through the slot its warp read last
        const int dump_off = (warp * C::kStages + held) * C::kSlotBytes;
        if (lane == 0) dump_at[warp] = held >= 0 ? dump_off : -1;
        if (held >= 0)
            st.dump(reinterpret_cast<float*>(base + dump_off), red_m + warp * 8, red_l + warp * 8,
                    lane);
        __syncthreads();
        const int rows = u.valid > 0 ? G : 0;
        // a warp takes whole rows: a lane four columns
        for (int i = warp; i < rows * qp.heads; i += kWarps) {
            const int hd = i >= rows ? 1 : 0, r = i - hd * rows;
            const int w0 = hd << in.wl2;  // the head's first warp
            float mw[kWarps], M = -INFINITY;
            int at[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const bool there = w < 1 << in.wl2;
                at[w] = there ? dump_at[w0 + w] : -1;
                mw[w] = at[w] >= 0 ? red_m[(w0 + w) * 8 + r] : -INFINITY;
                M = fmaxf(M, mw[w]);
            }
            const float mu = M == -INFINITY ? 0.f : M;
            float L = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (at[w] < 0) continue;
                const float f = fast_exp2(mw[w] - mu);
                const float4 v = *reinterpret_cast<const float4*>(
                    base + at[w] + (r * kHeadDim + ((lane ^ (r & 7)) * 4)) * 4);
                L = fmaf(red_l[(w0 + w) * 8 + r], f, L);
                o.x = fmaf(v.x, f, o.x);
                o.y = fmaf(v.y, f, o.y);
                o.z = fmaf(v.z, f, o.z);
                o.w = fmaf(v.w, f, o.w);
            }
            const float inv = L != 0.f ? __fdividef(1.f, L) : 0.f;
            o.x *= inv;
            o.y *= inv;
            o.z *= inv;
            o.w *= inv;
            const int row_in_unit = hd * G + r;
            float* lse = nullptr;
            float to_lse = 1.f;
            if (u.slot < 0) {
                const size_t row =
                    static_cast<size_t>(u.b) * p.num_qo_heads + u.h * G + row_in_unit;
                uint2 v;
                v.x = pack_bf16x2(o.x, o.y);
                v.y = pack_bf16x2(o.z, o.w);
                *reinterpret_cast<uint2*>(p.out + row * kHeadDim + lane * 4) = v;
                if (p.lse != nullptr) lse = p.lse + row;
                to_lse = kLn2;
            } else if constexpr (kCluster) {
                const int rank = static_cast<int>(cluster_ctarank());
                const uint32_t at_row = rank * C::kRows + r;
                st_cluster_v4(map_rank0(smem_addr(base) + C::kClusterOff +
                                        (at_row * kHeadDim + lane * 4) * 4), o);
                if (lane == 0)
                    st_cluster_f32(map_rank0(smem_addr(base) + C::kClusterSums + at_row * 4),
                                   L != 0.f ? M - kPOffset + __log2f(L) : -INFINITY);
            } else {
                // partial states are [slot][heads * G][128]
                const size_t row = static_cast<size_t>(u.slot) * G * qp.heads + row_in_unit;
                *reinterpret_cast<float4*>(p.part_o + row * kHeadDim + lane * 4) = o;
                lse = p.part_lse + row;
            }
            if (lane == 0 && lse != nullptr)
                *lse = L != 0.f ? (M - kPOffset + __log2f(L)) * to_lse : -INFINITY;
        }
        take_query(ui + 1);  // no warp reads this unit's any more
        __syncthreads();
        copy_query(ui + 2);
        if (held >= 0)
            in.refill(qp, units, ring_addr + held * C::kSlotBytes, dst, sdst, lane);
    }
    cp_async_wait<0>();
    if constexpr (kCluster) {
        // Every piece's state is in rank 0 now (a piece that is not a unit of
        // this plan weighs nothing), which merges them, a warp a row.
        const Unit u = u_begin < u_end ? units.get(qp, u_begin) : Unit{};
        if (u.valid == 0 && threadIdx.x < C::kRows)
            st_cluster_f32(map_rank0(smem_addr(base) + C::kClusterSums +
                                     (cluster_ctarank() * C::kRows + threadIdx.x) * 4),
                           -INFINITY);
        cluster_arrive();
        cluster_wait();
        if (cluster_ctarank() != 0 || u.valid == 0) return;
        const float* sums = reinterpret_cast<const float*>(base + C::kClusterSums);
        const float* vals = reinterpret_cast<const float*>(base + C::kClusterOff);
        for (int r = warp; r < G; r += kWarps) {
            float sv[kMaxClusterCtas], M = -INFINITY, W = 0.f;
#pragma unroll
            for (int i = 0; i < kMaxClusterCtas; ++i) {
                sv[i] = i < p.cluster_c ? sums[i * C::kRows + r] : -INFINITY;
                M = fmaxf(M, sv[i]);
            }
            const float mu = M == -INFINITY ? 0.f : M;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kMaxClusterCtas; ++i) {
                if (sv[i] == -INFINITY) continue;
                const float f = fast_exp2(sv[i] - mu);
                const float4 v = *reinterpret_cast<const float4*>(
                    vals + (i * C::kRows + r) * kHeadDim + lane * 4);
                W += f;
                o.x = fmaf(v.x, f, o.x);
                o.y = fmaf(v.y, f, o.y);
                o.z = fmaf(v.z, f, o.z);
                o.w = fmaf(v.w, f, o.w);
            }
            const float inv = W != 0.f ? __fdividef(1.f, W) : 0.f;
            const size_t row = static_cast<size_t>(u.b) * p.num_qo_heads + u.h * G + r;
            uint2 v;
            v.x = pack_bf16x2(o.x * inv, o.y * inv);
            v.y = pack_bf16x2(o.z * inv, o.w * inv);
            *reinterpret_cast<uint2*>(p.out + row * kHeadDim + lane * 4) = v;
            if (lane == 0 && p.lse != nullptr)
                p.lse[row] = W != 0.f ? (M + __log2f(W)) * kLn2 : -INFINITY;
        }
    }
}

template <class C, class WL, bool kCluster>
cudaError_t ensure_smem() {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
    if (bit != 0 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(quant_decode_kernel<C, WL, kCluster>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kCluster ? C::kSmemBytesCluster : C::kSmemBytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

template <class C, class WL, bool kCluster>
cudaError_t launch_ex(const QuantDecodeParams& p, const WL& w, int grid, cudaStream_t stream,
                      bool pdl) {
    const cudaError_t e = ensure_smem<C, WL, kCluster>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kCluster ? C::kSmemBytesCluster : C::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if constexpr (kCluster) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(p.d.cluster_c);
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
    return cudaLaunchKernelEx(&cfg, quant_decode_kernel<C, WL, kCluster>, p, w);
}

template <class C>
cudaError_t launch(const QuantDecodeParams& p, const WorkList* w, int grid, cudaStream_t stream,
                   bool pdl) {
    if (p.d.cluster_c > 1) {
        if (grid % p.d.cluster_c != 0 || p.d.cluster_c > kMaxClusterCtas || p.heads != 1)
            return cudaErrorInvalidValue;
        if (w != nullptr) return launch_ex<C, WorkList, true>(p, *w, grid, stream, pdl);
        return launch_ex<C, NoList, true>(p, NoList{0}, grid, stream, pdl);
    }
    if (w != nullptr) return launch_ex<C, WorkList, false>(p, *w, grid, stream, pdl);
    return launch_ex<C, NoList, false>(p, NoList{0}, grid, stream, pdl);
}

}  // namespace

// The page size changes neither the registers (capped by the launch bound) nor
// the shared memory.
VariantShape quant_shape(int variant) {
    if (variant != kVariantQuant8) return quant_wide_shape(variant);
    using C = QCfg<16>;
    return {kThreads, kWarps * kChunk, C::kStages, C::kSmemBytes};
}

cudaError_t quant_occupancy(int variant, int* n) {
    if (variant != kVariantQuant8) return quant_wide_occupancy(variant, n);
    using C = QCfg<16>;
    const cudaError_t e = ensure_smem<C, WorkList, false>();
    if (e != cudaSuccess) return e;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(
        n, quant_decode_kernel<C, WorkList, false>, kThreads, C::kSmemBytes);
}

cudaError_t quant_resident_clusters(int size, int* n) {
    using C = QCfg<16>;
    const cudaError_t e = ensure_smem<C, WorkList, true>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytesCluster;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(size);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(n, quant_decode_kernel<C, WorkList, true>, &cfg);
}

int quant_cluster_ctas_per_sm() { return 228 * 1024 / (QCfg<16>::kSmemBytesCluster + 1024); }

cudaError_t launch_decode_quant(int variant, const QuantDecodeParams& p, const WorkList* w,
                                int grid, cudaStream_t stream, bool pdl) {
    if (variant != kVariantQuant8)
        return launch_decode_quant_wide(variant, p, w, grid, stream, pdl);
    switch (p.d.page_size) {
        case 8: return launch<QCfg<8>>(p, w, grid, stream, pdl);
        case 16: return launch<QCfg<16>>(p, w, grid, stream, pdl);
        case 32: return launch<QCfg<32>>(p, w, grid, stream, pdl);
        case 64: return launch<QCfg<64>>(p, w, grid, stream, pdl);
    }
    return cudaErrorInvalidValue;
}

}  // namespace oxd
