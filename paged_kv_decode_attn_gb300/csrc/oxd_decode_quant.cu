// Decode attention over a 4-bit paged cache for sm_103a (oxd_quant_decode_run).
//
// For every query row q of a group and the tokens t of its request
//   x_t = sm_scale * sum_c ks[t,c] (q_c . e2m1(kc[t,c])),  c the four groups of 32
//   out = sum_t softmax(x)_t vs[t,.] e2m1(vc[t,.]),  lse = ln sum_t exp(x_t)
// 144 bytes a token and KV head, 3.6 times fewer than bf16: at the rate HBM
// delivers them (about 42 codes a clock and SM) the codes' conversion and the
// products have to be lean, so
//   * each of a CTA's four warps streams its own 32-token chunks of the CTA's
//     work units through a private ring of shared-memory slots (TMA copies that
//     the warp itself refills; no producer warp, no barrier between warps until
//     a unit ends);
//   * the tokens are the M dimension of mma.sync m16n8k16 (S^T = K Q^T,
//     O^T = V^T P^T), so the unpacked codes are the A fragment as they come out
//     of shared memory, a group of up to 8 heads is one N tile, and neither
//     operand goes back through shared memory;
//   * codes become f16 pairs by cvt.f16x2.e2m1x2, exact. K's scales multiply
//     the F32 sums of each 32-column group (4 FMAs for 2 MMAs), V's scales the
//     f16 codes; P goes from the S^T accumulator to the P^T operand by
//     movmatrix;
//   * the running maximum is raised only when a score passes it by 2^4, so most
//     chunks need one warp vote and no reduction or rescaling. P is held in f16
//     as exp2(x - m + 10): at most 2^14, and full precision down to 2^-24 of
//     the largest weight.
// A unit's four warp states are merged through the slots the warps last read;
// split streams leave F32 partial states for the merge kernel, as in the bf16
// decode. Waits are bounded: a warp whose wait runs out records it, skips the
// rest of its work but not the unit barriers, and waits for its copies in
// flight before it leaves.
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "oxd_e2m1.cuh"
#include "oxd_internal.h"
#include "oxd_ptx.cuh"

namespace oxd {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kLazy = 4.f;     // log2: how far a score may pass the running maximum
constexpr float kPOffset = 10.f; // log2 of the weight a score at the running maximum gets

// kNT: 8-head tiles a warp holds.
template <int kNT_, int kStages_, int kCtas_>
struct QCfg {
    static constexpr int kNT = kNT_;
    static constexpr int kRows = 8 * kNT;
    static constexpr int kStages = kStages_;
    static constexpr int kCtas = kCtas_;  // resident CTAs a SM (registers)
    // slot: K codes | V codes | K scales | V scales of 32 tokens. 512-byte
    // aligned, the period of the 64-byte swizzle.
    static constexpr int kVOff = kQuantChunk * kCodeBytes;
    static constexpr int kKsOff = 2 * kVOff;
    static constexpr int kVsOff = kKsOff + kQuantChunk * kScaleBytes;
    static constexpr int kSlotBytes = kVsOff + kQuantChunk * kScaleBytes;
    static_assert(kSlotBytes % 512 == 0, "slots keep the swizzle phase");
    static_assert(8 * kHeadDim * 4 <= kSlotBytes, "a dumped 8-row state fits a slot");
    static constexpr int kRingBytes = kWarps * kStages * kSlotBytes;
    static constexpr int kBarOff = kRingBytes;
    static constexpr int kRedOff = kBarOff + kWarps * kStages * 8;
    static constexpr int kFlagOff = kRedOff + 2 * kWarps * 8 * 4;  // abort, dump slot of each warp
    static constexpr int kSmemBytes = 512 + kFlagOff + 32;
};
using CfgQ8 = QCfg<1, 3, 4>;
using CfgQ16 = QCfg<2, 4, 3>;

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}

// D = A * B + D, m16n8k16, f16 inputs, f32 accumulate.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    __half2 v = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<uint32_t*>(&v);
}

// Token of MMA row r (0..7) of an 8-token block: 2 <-> 3 and 6 <-> 7 trade
// places, so the four V rows that a quarter of a warp reads at once lie in
// different banks.
__device__ __forceinline__ int row_token(int r) { return r ^ ((r >> 1) & 1); }

// A work unit, checked against the plan.
struct Unit {
    int first;    // offset of its first page in `indices`
    int n_pages;
    int b, h, row0, slot;
    int valid;    // tokens
    int n_chunks;
    bool ok;
};

__device__ __forceinline__ Unit decode_unit(const DecodeParams& p, const int4 it) {
    Unit u;
    u.first = it.x;
    u.n_pages = it.y & ((1 << kUnitPagesBits) - 1);
    const int last_len = (it.y >> kUnitPagesBits) & 0x7f;  // 0: not the request's last page
    u.b = it.z & ((1 << kUnitBBits) - 1);
    u.row0 = ((it.z >> kUnitBBits) & 1) * 16;
    u.h = static_cast<int>(static_cast<uint32_t>(it.z) >> (kUnitBBits + 1));
    u.slot = it.w;
    u.ok = u.n_pages >= 1 && it.x >= 0 && static_cast<int64_t>(it.x) + u.n_pages <= p.nnz &&
           u.b < p.batch && u.h < p.num_kv_heads && u.row0 < p.group && it.w >= -1 &&
           it.w < p.n_slots && last_len <= p.page_size;
    u.valid = last_len ? (u.n_pages - 1) * p.page_size + last_len : u.n_pages * p.page_size;
    u.n_chunks = u.ok ? (u.valid + kQuantChunk - 1) / kQuantChunk : 0;
    return u;
}

// One warp's stream of chunks: the refilling side, up to kStages chunks ahead
// of the consuming one. Chunk k of the warp in a unit is the unit's chunk
// warp + 4 k. The page indices of a run of chunks sit in the lanes (`win`,
// the next run in `ahead`), and the next unit's entry and first indices are
// read while the current unit's chunks are still being issued.
template <class C>
struct Stream {
    const QuantDecodeParams* qp;
    const int4* units;
    int u_end;
    int warp, lane;
    uint32_t ring, bars;   // shared addresses of the warp's slots and barriers
    int rows, ppc, run;    // tokens a box, pages a chunk, chunks a window
    int unit;              // unit being issued
    Unit u;
    int k;                 // next chunk of this warp in it
    int win, ahead, win_k;
    int4 nx_it;
    int nx_win;
    bool nx_have;          // nx_win holds unit + 1's first indices
    int issued;

    __device__ __forceinline__ int load_window(const Unit& x, int k0) const {
        const int ps = qp->d.page_size;
        const int c = warp + kWarps * (k0 + lane / ppc);
        const int pg = (c * kQuantChunk) / ps + lane % ppc;
        int v = 0;
        if (x.ok && lane / ppc < run && c < x.n_chunks && pg < x.n_pages)
            v = __ldg(qp->d.indices + x.first + pg);
        return v;
    }
    // An index outside the pool is recorded and replaced by page 0.
    __device__ __forceinline__ int check(int v) const {
        const bool bad = v < 0 || static_cast<int64_t>(v) >= qp->d.num_pages;
        if (__any_sync(0xffffffffu, bad) && lane == 0)
            record_status(qp->d.status, qp->d.epoch, kDeviceBadPage);
        return bad ? 0 : v;
    }
    __device__ __forceinline__ void load_next_item() {
        if (unit + 1 < u_end) nx_it = __ldg(units + unit + 1);
        nx_have = false;
    }
    __device__ __forceinline__ void load_next_window() {
        nx_win = unit + 1 < u_end ? load_window(decode_unit(qp->d, nx_it), 0) : 0;
        nx_have = true;
    }
    __device__ __forceinline__ void begin(int u_begin) {
        unit = u_begin;
        issued = 0;
        k = 0;
        u.ok = false;
        u.n_chunks = 0;
        if (unit < u_end) {
            u = decode_unit(qp->d, __ldg(units + unit));
            win = check(load_window(u, 0));
            ahead = load_window(u, run);
            win_k = 0;
            load_next_item();
        }
    }
    // Issues the next chunk's copies into its slot, if there is one.
    __device__ __forceinline__ void refill() {
        while (unit < u_end && warp + kWarps * k >= u.n_chunks) {
            if (!nx_have) load_next_window();
            ++unit;
            if (unit < u_end) {
                u = decode_unit(qp->d, nx_it);
                win = check(nx_win);
                ahead = load_window(u, run);
                win_k = 0;
                k = 0;
                load_next_item();
            }
        }
        if (unit >= u_end) return;
        if (k - win_k >= run) {
            win = check(ahead);
            win_k += run;
            ahead = load_window(u, win_k + run);
        }
        const DecodeParams& p = qp->d;
        const int ps = p.page_size;
        const int c = warp + kWarps * k;
        const int pg0 = (c * kQuantChunk) / ps;
        const int npg = min(ppc, u.n_pages - pg0);
        const int t0 = ps > kQuantChunk ? (c & 1) * kQuantChunk : 0;
        const int s = issued % C::kStages;
        const uint32_t slot = ring + s * C::kSlotBytes;
        uint64_t* bar = bar_ptr(s);
        if (lane == 0)
            mbar_arrive_expect_tx(bar, npg * rows * 2 * (kCodeBytes + kScaleBytes));
        __syncwarp();
        // lane 4 j + o: copy o (K codes, V codes, K scales, V scales) of page j
        const int j = lane >> 2, o = lane & 3;
        const int page = __shfl_sync(0xffffffffu, win, ((k - win_k) * ppc + j) & 31);
        if (j < npg) {
            if (o < 2) {
                tma_load_4d(slot + (o ? C::kVOff : 0) + j * rows * kCodeBytes, o ? map_v : map_k, bar, 0,
                            p.layout == 0 ? u.h : t0, p.layout == 0 ? t0 : u.h, page);
            } else {
                const uint16_t* src = (o == 2 ? qp->k_scales : qp->v_scales) +
                                      scale_index(page, t0, u.h, p.num_kv_heads, ps);
                bulk_load(slot + (o == 2 ? C::kKsOff : C::kVsOff) + j * rows * kScaleBytes, src,
                          rows * kScaleBytes, bar);
            }
        }
        ++issued;
        ++k;
        if (!nx_have) load_next_window();
    }
    const CUtensorMap* map_k;
    const CUtensorMap* map_v;
    uint64_t* bar_base;
    __device__ __forceinline__ uint64_t* bar_ptr(int s) const { return bar_base + s; }
};

template <class C>
struct State {
    uint32_t q[C::kNT][8][2];  // B fragments of the query rows, one pair per 16 columns
    float sc[C::kNT][2];       // logit scale (log2) of heads 2 tq, 2 tq + 1
    float m[C::kNT][2], l[C::kNT][2];
    float acc[C::kNT][8][4];

    // Columns 32 c + 8 tq .. + 8 of head g feed the two k steps of group c, in
    // the order the codes of a token leave its word. q is scaled by a power of
    // two so that the head's largest size lies in [1, 2) (f16's range).
    __device__ __forceinline__ void init(const uint16_t* q_rows, int nrows, float scale_log2,
                                         int lane) {
        const int g = lane >> 2, tq = lane & 3;
#pragma unroll
        for (int n = 0; n < C::kNT; ++n) {
            uint32_t w[16];
            const bool have = n * 8 + g < nrows;
            const uint4* src =
                reinterpret_cast<const uint4*>(q_rows + static_cast<size_t>(n * 8 + g) * kHeadDim);
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint4 x = have ? __ldg(src + c * 4 + tq) : make_uint4(0, 0, 0, 0);
                w[4 * c] = x.x;
                w[4 * c + 1] = x.y;
                w[4 * c + 2] = x.z;
                w[4 * c + 3] = x.w;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
                top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // exponent field of the largest size, kept where 2^+-exponent is a
            // normal float
            const uint32_t e = min(max(top >> 7, 1u), 253u);
            const float f = __uint_as_float((254u - e) << 23);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                q[n][i >> 1][i & 1] = pack_f16x2(__uint_as_float(w[i] << 16) * f,
                                                 __uint_as_float(w[i] & 0xffff0000u) * f);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t eh = __shfl_sync(0xffffffffu, e, (2 * tq + j) * 4);
                sc[n][j] = scale_log2 * __uint_as_float(eh << 23);
                m[n][j] = -INFINITY;
                l[n][j] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc[n][i][0] = acc[n][i][1] = acc[n][i][2] = acc[n][i][3] = 0.f;
        }
    }

    // One chunk: tokens [u0, u0 + 32) of the unit, in `slot`.
    __device__ __forceinline__ void consume(uint32_t slot, int u0, int valid, int lane) {
        const int g = lane >> 2, tq = lane & 3;
        const int pg = row_token(g);
        // ---- S^T = K Q^T
        float s[2][C::kNT][4];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            const int tok = tb * 16 + ((lane >> 3) & 1) * 8 + row_token(lane & 7);
            const uint32_t row = slot + tok * kCodeBytes;
            const uint32_t sw = (tok >> 1) & 3;
            const uint2 k0 = lds64(slot + C::kKsOff + (tb * 16 + pg) * kScaleBytes);
            const uint2 k1 = lds64(slot + C::kKsOff + (tb * 16 + 8 + pg) * kScaleBytes);
            const float2 s01 = f16x2_floats(k0.x), s23 = f16x2_floats(k0.y);
            const float2 t01 = f16x2_floats(k1.x), t23 = f16x2_floats(k1.y);
            const float ks0[4] = {s01.x, s01.y, s23.x, s23.y};
            const float ks1[4] = {t01.x, t01.y, t23.x, t23.y};
#pragma unroll
            for (int c = 0; c < 4; c += 2) {
                uint32_t w[4];
                ldsm_x4(row + (((c + (lane >> 4)) ^ sw) << 4), w);
#pragma unroll
                for (int cc = 0; cc < 2; ++cc) {
                    uint32_t a[4], b[4];
                    codes_to_f16(w[2 * cc], a);
                    codes_to_f16(w[2 * cc + 1], b);
                    const int grp = c + cc;
#pragma unroll
                    for (int n = 0; n < C::kNT; ++n) {
                        float t[4] = {0.f, 0.f, 0.f, 0.f};
                        mma_f16(t, a[0], b[0], a[1], b[1], q[n][2 * grp][0], q[n][2 * grp][1]);
                        mma_f16(t, a[2], b[2], a[3], b[3], q[n][2 * grp + 1][0],
                                q[n][2 * grp + 1][1]);
                        if (grp == 0) {
                            s[tb][n][0] = t[0] * ks0[0];
                            s[tb][n][1] = t[1] * ks0[0];
                            s[tb][n][2] = t[2] * ks1[0];
                            s[tb][n][3] = t[3] * ks1[0];
                        } else {
                            s[tb][n][0] = fmaf(t[0], ks0[grp], s[tb][n][0]);
                            s[tb][n][1] = fmaf(t[1], ks0[grp], s[tb][n][1]);
                            s[tb][n][2] = fmaf(t[2], ks1[grp], s[tb][n][2]);
                            s[tb][n][3] = fmaf(t[3], ks1[grp], s[tb][n][3]);
                        }
                    }
                }
            }
        }
        // ---- online softmax in the log2 domain
        const bool partial = u0 + kQuantChunk > valid;
        bool raise = false;
        float mx[C::kNT][2];
#pragma unroll
        for (int n = 0; n < C::kNT; ++n) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int tb = 0; tb < 2; ++tb) {
                    s[tb][n][j] *= sc[n][j];
                    s[tb][n][2 + j] *= sc[n][j];
                    if (partial) {
                        const int t = u0 + tb * 16 + pg;
                        if (t >= valid) s[tb][n][j] = -INFINITY;
                        if (t + 8 >= valid) s[tb][n][2 + j] = -INFINITY;
                    }
                }
                mx[n][j] = fmaxf(fmaxf(s[0][n][j], s[0][n][2 + j]),
                                 fmaxf(s[1][n][j], s[1][n][2 + j]));
                raise = raise || mx[n][j] > m[n][j] + kLazy;
            }
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int n = 0; n < C::kNT; ++n) {
                float al[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = mx[n][j];
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                    const float mn = fmaxf(m[n][j], x);
                    al[j] = mn == -INFINITY ? 1.f : fast_exp2(m[n][j] - mn);
                    m[n][j] = mn;
                    l[n][j] *= al[j];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    acc[n][i][0] *= al[0];
                    acc[n][i][1] *= al[1];
                    acc[n][i][2] *= al[0];
                    acc[n][i][3] *= al[1];
                }
            }
        }
        uint32_t pb[2][C::kNT][2];  // P^T fragments of the two 16-token blocks
#pragma unroll
        for (int n = 0; n < C::kNT; ++n) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float mu = m[n][j] == -INFINITY ? 0.f : m[n][j] - kPOffset;
#pragma unroll
                for (int tb = 0; tb < 2; ++tb) {
                    s[tb][n][j] = fast_exp2(s[tb][n][j] - mu);
                    s[tb][n][2 + j] = fast_exp2(s[tb][n][2 + j] - mu);
                }
                l[n][j] += (s[0][n][j] + s[0][n][2 + j]) + (s[1][n][j] + s[1][n][2 + j]);
            }
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
                pb[tb][n][0] = transpose_8x8(pack_f16x2(s[tb][n][0], s[tb][n][1]));
                pb[tb][n][1] = transpose_8x8(pack_f16x2(s[tb][n][2], s[tb][n][3]));
            }
        }
        // ---- O^T += V^T P^T: a thread's A rows are columns 16 g .. 16 g + 15
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            uint2 x[4];
            uint32_t vs[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // MMA columns 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9
                const int tok = tb * 16 + (i >> 1) * 8 + ((2 * tq + (i & 1)) ^ (tq & 1));
                x[i] = lds64(slot + C::kVOff + tok * kCodeBytes +
                             ((((g >> 1) ^ (tok >> 1)) & 3) << 4) + (g & 1) * 8);
                vs[i] = lds16(slot + C::kVsOff + tok * kScaleBytes + (g >> 1) * 2);
                // rows past the last token may hold anything, NaN scales too
                if (partial && u0 + tok >= valid) vs[i] = 0u;
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
#pragma unroll
                    for (int n = 0; n < C::kNT; ++n)
                        mma_f16(acc[n][half * 4 + i], f0, f1, f2, f3, pb[tb][n][0], pb[tb][n][1]);
                }
            }
        }
    }

    // Rows 8 n .. 8 n + 7 of the accumulator as f32 [8][128] into `dump`
    // (float4 columns XOR-swizzled by the row), their maxima and sums.
    __device__ __forceinline__ void dump(int n, float* dump, float* red_m, float* red_l,
                                         int lane) {
        const int g = lane >> 2, tq = lane & 3;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float t = l[n][j];
            t += __shfl_xor_sync(0xffffffffu, t, 4);
            t += __shfl_xor_sync(0xffffffffu, t, 8);
            t += __shfl_xor_sync(0xffffffffu, t, 16);
            const int row = 2 * tq + j;
            if (g == 0) {
                red_m[row] = m[n][j];
                red_l[row] = t;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col4 = (g * 4 + i) ^ (row & 7);
                *reinterpret_cast<float4*>(dump + row * kHeadDim + col4 * 4) =
                    make_float4(acc[n][2 * i][j], acc[n][2 * i][2 + j], acc[n][2 * i + 1][j],
                                acc[n][2 * i + 1][2 + j]);
            }
        }
    }
};

template <class C, class WL>
__global__ void __launch_bounds__(kThreads, C::kCtas)
    quant_decode_kernel(const __grid_constant__ CUtensorMap tmap_k,
                        const __grid_constant__ CUtensorMap tmap_v,
                        const __grid_constant__ QuantDecodeParams qp,
                        const __grid_constant__ WL work) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 511) &
                                               ~static_cast<uintptr_t>(511));
    const DecodeParams& p = qp.d;
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + C::kBarOff);
    float* red_m = reinterpret_cast<float*>(base + C::kRedOff);
    float* red_l = red_m + kWarps * 8;
    volatile int* flags = reinterpret_cast<volatile int*>(base + C::kFlagOff);  // [0] abort
    volatile int* dump_slot = flags + 1;  // [warp]: the slot its state is dumped in, or -1
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kWarps * C::kStages; ++i) mbar_init(bars + i, 1);
        flags[0] = 0;
        fence_mbar_init();
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_v);
    }
    // as a programmatic dependent: nothing in global memory before this
    grid_dependency_wait();
    // This CTA's units, from the parameter buffer or the workspace; one thread
    // reads the range, so every warp passes the same number of barriers.
    const int4* units = p.units;
    volatile int* range = flags + 1;  // (first, end), before the dump slots are used
    if (threadIdx.x == 0) {
        if (blockIdx.x == 0) {
            *p.last_epoch = p.epoch;
            if (p.clear_stamp != nullptr) *p.clear_stamp = 0ull;
        }
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        int a = 0, b = 0;
        bool listed = false;
        if constexpr (std::is_same<WL, WorkList>::value) {
            if (units == nullptr) {
                a = work.cta_begin[blockIdx.x];
                b = work.cta_begin[blockIdx.x + 1];
                listed = true;
            }
        }
        if (!listed) {
            const int4 r = __ldg(p.cta_rec + 2 * blockIdx.x);
            a = r.x;
            b = r.y;
        }
        if ((p.ws_stamp != nullptr && *p.ws_stamp != p.stamp) || a < 0 || b > p.n_units || a > b) {
            record_status(p.status, p.epoch, kDevicePlanMismatch);
            a = b = 0;
        }
        range[0] = a;
        range[1] = b;
    }
    if constexpr (std::is_same<WL, WorkList>::value) {
        if (units == nullptr) units = work.unit;
    }
    __syncthreads();
    const int u_begin = range[0], u_end = range[1];
    __syncthreads();

    Stream<C> in;
    in.qp = &qp;
    in.units = units;
    in.u_end = u_end;
    in.warp = warp;
    in.lane = lane;
    in.ring = smem_addr(base) + warp * C::kStages * C::kSlotBytes;
    in.bar_base = bars + warp * C::kStages;
    in.map_k = &tmap_k;
    in.map_v = &tmap_v;
    in.rows = min(p.page_size, kQuantChunk);
    in.ppc = kQuantChunk / in.rows;
    in.run = 32 / in.ppc;
    in.begin(u_begin);
    for (int i = 0; i < C::kStages; ++i) in.refill();

    State<C> st;
    bool dead = false;   // a wait of this warp ran out
    int taken = 0;       // chunks consumed
    const int G = p.group;
    int4 it = u_begin < u_end ? __ldg(units + u_begin) : make_int4(0, 0, 0, 0);
    for (int ui = u_begin; ui < u_end; ++ui) {
        const int4 it_now = it;
        const Unit u = decode_unit(p, it_now);
        if (ui + 1 < u_end) it = __ldg(units + ui + 1);
        const int nrows = min(G - u.row0, C::kRows);
        const size_t row_base =
            static_cast<size_t>(u.b) * p.num_qo_heads + u.h * G + u.row0;
        if (threadIdx.x == 0) {
            if (!u.ok) {
                record_status(p.status, p.epoch, kDevicePlanMismatch);
            } else {
                const int last_len = (it_now.y >> kUnitPagesBits) & 0x7f;
                if ((it_now.y < 0 && p.indptr[u.b] != it_now.x) ||
                    (last_len && (p.indptr[u.b + 1] != it_now.x + u.n_pages ||
                                  p.last_page_len[u.b] != last_len)))
                    record_status(p.status, p.epoch, kDevicePlanMismatch);
            }
        }
        int held = -1;  // the slot of the warp's last chunk, not refilled yet
        if (warp < u.n_chunks) st.init(p.q + row_base * kHeadDim, nrows, p.scale_log2, lane);
        for (int c = warp; c < u.n_chunks && !dead; c += kWarps) {
            const int s = taken % C::kStages;
            const bool got = mbar_wait(in.bar_ptr(s), (taken / C::kStages) & 1, flags, p.wait_ns);
            if (!__all_sync(0xffffffffu, got)) {
                dead = true;
                if (lane == 0) {
                    flags[0] = 1;
                    record_status(p.status, p.epoch, kDeviceWaitTimeout);
                }
                break;
            }
            ++taken;
            st.consume(in.ring + s * C::kSlotBytes, c * kQuantChunk, u.valid, lane);
            __syncwarp();
            if (c + kWarps < u.n_chunks)
                in.refill();
            else
                held = s;
        }
        // ---- merge the warps' states, eight rows at a time
#pragma unroll
        for (int n = 0; n < C::kNT; ++n) {
            if (lane == 0) dump_slot[warp] = held;
            if (held >= 0)
                st.dump(n,
                        reinterpret_cast<float*>(base + (warp * C::kStages + held) * C::kSlotBytes),
                        red_m + warp * 8, red_l + warp * 8, lane);
            __syncthreads();
            const int rows = u.ok ? min(8, nrows - n * 8) : 0;
            for (int i = threadIdx.x; i < rows * (kHeadDim / 4); i += kThreads) {
                const int r = i / (kHeadDim / 4), c4 = i % (kHeadDim / 4);
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    if (dump_slot[w] >= 0) M = fmaxf(M, red_m[w * 8 + r]);
                const float mu = M == -INFINITY ? 0.f : M;
                float L = 0.f;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const int sl = dump_slot[w];
                    if (sl < 0) continue;
                    const float f = fast_exp2(red_m[w * 8 + r] - mu);
                    const float4 a = *reinterpret_cast<const float4*>(
                        base + (w * C::kStages + sl) * C::kSlotBytes +
                        (r * kHeadDim + ((c4 ^ (r & 7)) * 4)) * 4);
                    L += red_l[w * 8 + r] * f;
                    o.x += a.x * f;
                    o.y += a.y * f;
                    o.z += a.z * f;
                    o.w += a.w * f;
                }
                const float inv = L != 0.f ? 1.f / L : 0.f;
                o.x *= inv;
                o.y *= inv;
                o.z *= inv;
                o.w *= inv;
                const float lse2 = L != 0.f ? M - kPOffset + log2f(L) : -INFINITY;
                if (u.slot < 0) {
                    const size_t row = row_base + n * 8 + r;
                    uint2 v;
                    v.x = pack_bf16x2(o.x, o.y);
                    v.y = pack_bf16x2(o.z, o.w);
                    *reinterpret_cast<uint2*>(p.out + row * kHeadDim + c4 * 4) = v;
                    if (c4 == 0 && p.lse != nullptr) p.lse[row] = lse2 * kLn2;
                } else {
                    const size_t row = static_cast<size_t>(u.slot) * G + u.row0 + n * 8 + r;
                    *reinterpret_cast<float4*>(p.part_o + row * kHeadDim + c4 * 4) = o;
                    if (c4 == 0) p.part_lse[row] = lse2;
                }
            }
            __syncthreads();
        }
        if (held >= 0) {
            // the dump was written and read by plain accesses; the next copy
            // into the slot comes from the async proxy
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            in.refill();
        }
    }
    // Copies in flight (after a wait ran out, or issued from a list that changed
    // meanwhile) land before the CTA leaves.
    for (; taken < in.issued; ++taken)
        mbar_wait(in.bar_ptr(taken % C::kStages), (taken / C::kStages) & 1, nullptr, kWaitTimeoutNs);
}

template <class C, class WL>
cudaError_t ensure_smem() {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
    if (bit != 0 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(quant_decode_kernel<C, WL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmemBytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

template <class C, class WL>
cudaError_t launch_ex(const CUtensorMap& tk, const CUtensorMap& tv, const QuantDecodeParams& p,
                      const WL& w, int grid, cudaStream_t stream, bool pdl) {
    const cudaError_t e = ensure_smem<C, WL>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, quant_decode_kernel<C, WL>, tk, tv, p, w);
}

template <class C>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const QuantDecodeParams& p,
                   const WorkList* w, int grid, cudaStream_t stream, bool pdl) {
    if (w != nullptr) return launch_ex<C>(tk, tv, p, *w, grid, stream, pdl);
    return launch_ex<C>(tk, tv, p, NoList{0}, grid, stream, pdl);
}

template <class C>
cudaError_t occupancy(int* n) {
    const cudaError_t e = ensure_smem<C, WorkList>();
    if (e != cudaSuccess) return e;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, quant_decode_kernel<C, WorkList>,
                                                         kThreads, C::kSmemBytes);
}

}  // namespace

VariantShape quant_shape(int variant) {
    if (variant == kVariantQuant8)
        return {kThreads, kWarps * kQuantChunk, CfgQ8::kStages, CfgQ8::kSmemBytes};
    return {kThreads, kWarps * kQuantChunk, CfgQ16::kStages, CfgQ16::kSmemBytes};
}

cudaError_t quant_occupancy(int variant, int* n) {
    return variant == kVariantQuant8 ? occupancy<CfgQ8>(n) : occupancy<CfgQ16>(n);
}

cudaError_t launch_decode_quant(int variant, const CUtensorMap& tk, const CUtensorMap& tv,
                                const QuantDecodeParams& p, const WorkList* w, int grid,
                                cudaStream_t stream, bool pdl) {
    if (variant == kVariantQuant8) return launch<CfgQ8>(tk, tv, p, w, grid, stream, pdl);
    return launch<CfgQ16>(tk, tv, p, w, grid, stream, pdl);
}

}  // namespace oxd
