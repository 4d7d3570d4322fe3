// One warp's softmax state over chunks of 32 tokens of a 4-bit cache, for groups of
// up to 8 query heads: the tokens are the M dimension of mma.sync m16n8k16. Shared by
// the decode (oxd_decode_quant.cu) and the window decode (oxd_window_quant.cu).
#pragma once

#include "oxd_decode_quant.cuh"

namespace oxd {
namespace {

constexpr int kChunk = 32;  // tokens a warp takes at a time

// Token of MMA row r (0..7) of an 8-token block: 2 <-> 3 and 6 <-> 7 trade
// places, so the four V rows that a quarter of a warp reads at once lie in
// different banks.
__device__ __forceinline__ int row_token(int r) { return r ^ ((r >> 1) & 1); }

// C gives the offsets of a chunk's parts in its slot: kVOff, kKsOff, kVsOff (K's codes
// come first).
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

}  // namespace
}  // namespace oxd
