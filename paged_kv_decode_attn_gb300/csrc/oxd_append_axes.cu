// Rotary embedding with position axes + paged KV append for sm_103a, into
// bf16 pages (oxd_rope_axes_append) or 4-bit pages (oxd_quant_rope_append).
//
//   angle of pair i = rope_positions[axis_i][t] * theta^(-2i/128)
//   y_i = x_i cos - x_{i+64} sin,  y_{i+64} = x_{i+64} cos + x_i sin
//
// A call reads q, k and v once and writes q_out and the page rows once, so
// bytes bound it (long calls) or the chain position -> page -> refcount (a
// decode step). A block of eight warps takes four tokens (one in short calls,
// which spreads them over the SMs; a 16384-token prompt of 32 and 8 heads into
// 4-bit pages takes 111, 77, 65 and 68 us with one, two, four and eight tokens a
// block). Its threads form the tokens' 64 cosines and sines each, one pair a
// thread, which all of a token's heads share (formed per row in double, they were
// the whole cost); then each warp takes rows of one token, four at a time, eight
// lanes a row: lane s of a row holds columns 8s .. 8s + 7 and 64 + 8s ..
// (two 16-byte loads), so a rotation pairs values of one lane, a 4-bit group
// of 32 is four lanes, and a row's 8 cosines stay in registers.
//
// Which code a K value of a 4-bit row gets is a comparison, so there the
// rotated value is formed to about 2^-32 of the pair (cosines, sines and
// products as sums of two floats) before it is rounded to bf16: the codes are
// those of the exactly rotated row but for about one value in 10^9, where
// float arithmetic would flip one in 10^6 and some groups' scales. Everything
// else rotates in float.
#include <cuda_bf16.h>

#include "oxd_e2m1.cuh"
#include "oxd_internal.h"
#include "oxd_ptx.cuh"

namespace oxd {
namespace {

constexpr int kWarps = 8;
constexpr int kRowsPerTask = 4;  // rows (heads) a warp takes at a time
constexpr int kBatch = 2;        // tasks of query rows in flight a warp
constexpr int kPairs = kHeadDim / 2;

// a + b = s + e exactly.
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
    s = __fadd_rn(a, b);
    const float t = __fadd_rn(s, -a);
    e = __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -t)), __fadd_rn(b, -t));
}

// a * b = p + e exactly.
__device__ __forceinline__ void two_prod(float a, float b, float& p, float& e) {
    p = __fmul_rn(a, b);
    e = fmaf(a, b, -p);
}

// cos and sin of pos * g turns, each as a sum of two floats good to about
// 2^-32. g.x + g.y + g.z is the frequency in turns; pos < 2^24. The product is
// kept exactly, whole quarter turns are taken off, and what is left, at most
// an eighth of a turn, goes through the Taylor series with its leading terms
// in two floats (the others are below 2^-11 of the result, so their float
// roundings stay below 2^-32).
__device__ __forceinline__ float4 cos_sin(int pos, float4 g) {
    const float P = static_cast<float>(pos);
    float h1, e1, h2, e2, s, a, b;
    two_prod(P, g.x, h1, e1);
    two_prod(P, g.y, h2, e2);
    two_sum(h1 - rintf(h1), e1, s, a);
    two_sum(s, h2, s, b);
    float lo = (a + b) + (e2 + P * g.z);
    two_sum(s, lo, s, lo);
    const float quarter = rintf(4.f * s);
    s = fmaf(-0.25f, quarter, s);  // exact
    two_sum(s, lo, s, lo);
    // z = 2 pi s
    constexpr float kTwoPiHi = 6.2831854820251465f, kTwoPiLo = -1.7484556000744883e-7f;
    float zh, zl;
    two_prod(s, kTwoPiHi, zh, zl);
    zl = fmaf(s, kTwoPiLo, fmaf(lo, kTwoPiHi, zl));
    // u = z^2, q = u^2
    float uh, ul, q, qe;
    two_prod(zh, zh, uh, ul);
    ul = fmaf(2.f * zh, zl, ul);
    two_prod(uh, uh, q, qe);
    qe = fmaf(2.f * uh, ul, qe);
    // sin z = z (1 + t), t = -u/6 + u^2/120 - u^3/5040 + ...
    constexpr float k6Hi = -1.f / 6.f, k6Lo = 4.967053731e-9f;       // -1/6 = Hi + Lo
    constexpr float k120Hi = 1.f / 120.f, k120Lo = -4.346172015e-10f;     // 1/120
    float m, me, n, ne, t, te, w, we;
    two_prod(uh, k6Hi, m, me);
    me = fmaf(uh, k6Lo, fmaf(ul, k6Hi, me));
    two_prod(q, k120Hi, n, ne);
    ne = fmaf(q, k120Lo, fmaf(qe, k120Hi, ne));
    float v = fmaf(uh, -2.5052108e-8f, 2.7557319e-6f);  // -1/11!, 1/9!
    v = q * uh * fmaf(uh, v, -1.9841270e-4f);             // -1/7!
    two_sum(m, n, t, te);
    te += me + (ne + v);
    two_prod(zh, t, w, we);
    we = fmaf(zh, te, fmaf(zl, t, we));
    float sn, snl;
    two_sum(zh, w, sn, snl);
    snl += zl + we;
    // cos z = 1 - u/2 + u^2/24 - u^3/720 + ...
    constexpr float k24Hi = 1.f / 24.f, k24Lo = -1.241763433e-9f;    // 1/24
    float y, ye;
    two_prod(q, k24Hi, y, ye);
    ye = fmaf(q, k24Lo, fmaf(qe, k24Hi, ye));
    float r = fmaf(uh, 2.0876757e-9f, -2.7557319e-7f);  // 1/12!, -1/10!
    r = fmaf(uh, r, 2.4801587e-5f);                       // 1/8!
    r = q * uh * fmaf(uh, r, -1.3888889e-3f);             // -1/6!
    float cs, csl, x, xe;
    two_sum(1.f, -0.5f * uh, cs, csl);
    two_sum(cs, y, x, xe);
    csl += xe + (ye + r) - 0.5f * ul;
    two_sum(x, csl, cs, csl);
    two_sum(sn, snl, sn, snl);
    const int k = static_cast<int>(quarter) & 3;  // sin, cos of z + k quarter turns
    float4 o = (k & 1) ? make_float4(-sn, cs, -snl, csl) : make_float4(cs, sn, csl, snl);
    if (k & 2) o = make_float4(-o.x, -o.y, -o.z, -o.w);
    return o;  // cos, sin, their low parts
}

// A bf16 number from hi + lo (hi the nearest float): hi rounds the right way
// by itself unless it lies exactly between two bf16 numbers.
__device__ __forceinline__ float nudge_tie(float hi, float lo) {
    uint32_t b = __float_as_uint(hi);
    if ((b & 0xffffu) == 0x8000u && lo != 0.f) b += ((lo > 0.f) == (hi > 0.f)) ? 1u : ~0u;
    return __uint_as_float(b);
}

// a c - b s (c, s with low parts cl, sl), rounded to bf16 once. kLarge: for sizes
// from 2^126 on, whose sum may pass the largest float, and infinities, whose low
// parts would be NaN.
template <bool kLarge>
__device__ __forceinline__ float exact_turn(float a, float c, float cl, float b, float s,
                                            float sl) {
    float p, pe, q, qe, d, de;
    if (kLarge) {
        a *= 0.25f;
        b *= 0.25f;
    }
    two_prod(a, c, p, pe);
    two_prod(-b, s, q, qe);
    two_sum(p, q, d, de);
    if (kLarge && !(fabsf(d) <= 3.40282347e38f)) return d;
    const float rest = fmaf(a, cl, fmaf(-b, sl, (pe + qe) + de));
    const float hi = __fadd_rn(d, rest);
    const float y = nudge_tie(hi, __fadd_rn(rest, -__fadd_rn(hi, -d)));
    return kLarge ? 4.f * y : y;
}

// The lane's 16 columns of a row: eight below 64 and their partners.
struct Slice {
    uint4 lo, hi;
};

__device__ __forceinline__ Slice load_slice(const uint16_t* row, int s) {
    return {*reinterpret_cast<const uint4*>(row + 8 * s),
            *reinterpret_cast<const uint4*>(row + 64 + 8 * s)};
}
__device__ __forceinline__ void store_slice(uint16_t* row, int s, const Slice& x) {
    *reinterpret_cast<uint4*>(row + 8 * s) = x.lo;
    *reinterpret_cast<uint4*>(row + 64 + 8 * s) = x.hi;
}
// cs: the token's cosines and sines in shared memory, the lane's pair j at 8 j;
// low: their low parts.
__device__ __forceinline__ Slice rotate(const Slice& x, const float2* cs) {
    const uint32_t* a = &x.lo.x;
    const uint32_t* b = &x.hi.x;
    Slice y;
    uint32_t* ya = &y.lo.x;
    uint32_t* yb = &y.hi.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a0 = bf16_low(a[i]), a1 = bf16_high(a[i]);
        const float b0 = bf16_low(b[i]), b1 = bf16_high(b[i]);
        const float2 t0 = cs[8 * (2 * i)], t1 = cs[8 * (2 * i + 1)];
        ya[i] = pack_bf16x2(a0 * t0.x - b0 * t0.y, a1 * t1.x - b1 * t1.y);
        yb[i] = pack_bf16x2(b0 * t0.x + a0 * t0.y, b1 * t1.x + a1 * t1.y);
    }
    return y;
}

// The larger sizes of two pairs, with any signs.
__device__ __forceinline__ uint32_t max_sizes_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Rotates w[i] and w[4 + i], pairs of columns and their partners, exactly.
template <bool kLarge>
__device__ __forceinline__ void turn_slice(uint32_t (&w)[8], const float2* cs, const float2* low) {
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        const float a0 = bf16_low(w[i]), a1 = bf16_high(w[i]);
        const float b0 = bf16_low(w[4 + i]), b1 = bf16_high(w[4 + i]);
        const float2 t0 = cs[8 * (2 * i)], t1 = cs[8 * (2 * i + 1)];
        const float2 l0 = low[8 * (2 * i)], l1 = low[8 * (2 * i + 1)];
        w[i] = pack_bf16x2(exact_turn<kLarge>(a0, t0.x, l0.x, b0, t0.y, l0.y),
                           exact_turn<kLarge>(a1, t1.x, l1.x, b1, t1.y, l1.y));
        w[4 + i] = pack_bf16x2(exact_turn<kLarge>(b0, t0.x, l0.x, -a0, t0.y, l0.y),
                               exact_turn<kLarge>(b1, t1.x, l1.x, -a1, t1.y, l1.y));
    }
}

// As rotate, with the bf16 numbers nearest to the exact rotation. The float
// result y is within 2^-21 (|a| + |b|) of it (cosine and sine rounded once, two
// products, a sum): where both ends of that range round alike, that is it. A
// lane with a value where they do not (about one in 200, infinities among them)
// forms its slice anew with the low parts, one pair of columns at a time.
__device__ __forceinline__ Slice rotate_exact(const Slice& x, const float2* cs,
                                              const float2* low) {
    const uint32_t* a = &x.lo.x;
    const uint32_t* b = &x.hi.x;
    Slice y;
    uint32_t* ya = &y.lo.x;
    uint32_t* yb = &y.hi.x;
    constexpr float kErr = 4.76837158e-7f;  // 2^-21
    uint32_t differ = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a0 = bf16_low(a[i]), a1 = bf16_high(a[i]);
        const float b0 = bf16_low(b[i]), b1 = bf16_high(b[i]);
        const float2 t0 = cs[8 * (2 * i)], t1 = cs[8 * (2 * i + 1)];
        const float n0 = fabsf(a0) + fabsf(b0), n1 = fabsf(a1) + fabsf(b1);
        const float u0 = a0 * t0.x - b0 * t0.y, u1 = a1 * t1.x - b1 * t1.y;
        const float v0 = b0 * t0.x + a0 * t0.y, v1 = b1 * t1.x + a1 * t1.y;
        ya[i] = pack_bf16x2(fmaf(n0, kErr, u0), fmaf(n1, kErr, u1));
        yb[i] = pack_bf16x2(fmaf(n0, kErr, v0), fmaf(n1, kErr, v1));
        differ |= ya[i] ^ pack_bf16x2(fmaf(n0, -kErr, u0), fmaf(n1, -kErr, u1));
        differ |= yb[i] ^ pack_bf16x2(fmaf(n0, -kErr, v0), fmaf(n1, -kErr, v1));
    }
    if (differ != 0) {
        uint32_t w[8], top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = a[i];
            w[4 + i] = b[i];
            top = max_sizes_bf16x2(top, max_sizes_bf16x2(a[i], b[i]));
        }
        if (__vcmpgeu2(top & 0x7fff7fffu, 0x7e807e80u) == 0)  // 2^126
            turn_slice<false>(w, cs, low);
        else
            turn_slice<true>(w, cs, low);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ya[i] = w[i];
            yb[i] = w[4 + i];
        }
    }
    return y;
}

// Holds a row in 4 bits. Lanes 0..3 (4..7) of a row have group 0 (1) in their
// low and group 2 (3) in their high columns. Every lane of the warp calls it;
// `live` lanes store.
__device__ __forceinline__ void hold_slice(uint8_t* codes, uint16_t* scales, const Slice& x, int s,
                                           bool live) {
    uint32_t sc[2], code[2];
    hold_eight(x.lo, code[0], sc[0]);
    hold_eight(x.hi, code[1], sc[1]);
    const uint32_t far0 = __shfl_xor_sync(0xffffffffu, sc[0], 4);
    const uint32_t far1 = __shfl_xor_sync(0xffffffffu, sc[1], 4);
    if (live) {
        *reinterpret_cast<uint32_t*>(codes + 4 * s) = code[0];
        *reinterpret_cast<uint32_t*>(codes + 32 + 4 * s) = code[1];
        if (s == 0)
            *reinterpret_cast<uint2*>(scales) = make_uint2(sc[0] | (far0 << 16), sc[1] | (far1 << 16));
    }
}

// kTokens: tokens a block takes; its warps are divided among them.
template <bool k4, int kTokens>
__global__ void __launch_bounds__(kWarps * 32, 4)
    axes_append_kernel(const __grid_constant__ AxesAppendParams p) {
    constexpr int kTokenWarps = kWarps / kTokens;
    __shared__ float2 cs_all[kTokens][kPairs], low_all[k4 ? kTokens : 1][kPairs];
    __shared__ float4 turns[kTokens > 1 ? kPairs : 1];
    __shared__ int bad_rope[kTokens];
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.last_epoch = p.epoch;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = lane & 7, sub = lane >> 3;  // columns of the row, row of the task
    const int local = warp / kTokenWarps, wi = warp % kTokenWarps;
    const long long t_all = static_cast<long long>(blockIdx.x) * kTokens + local;
    const bool have = t_all < p.T;
    const int t = have ? static_cast<int>(t_all) : 0;
    const int kv_tasks = (p.Hkv + kRowsPerTask - 1) / kRowsPerTask;

    // The first rows and the page walk are under way while the angles are
    // formed. KV tasks go to the token's first warps.
    const bool kv_warp = have && wi < kv_tasks;
    Slice k0, v0;
    if (kv_warp && wi * kRowsPerTask + sub < p.Hkv) {
        const size_t row = (static_cast<size_t>(t) * p.Hkv + wi * kRowsPerTask + sub) * kHeadDim;
        k0 = load_slice(p.k + row, s);
        v0 = load_slice(p.v + row, s);
    }
    int b = -1, pos = -1;
    if (kv_warp) {
        b = p.token_request[t];
        pos = p.positions[t];
    }
    // Lanes that read different parameters are served one by one: once a block.
    if (kTokens > 1 && threadIdx.x < kPairs) turns[threadIdx.x] = p.turns[threadIdx.x];
    if (threadIdx.x < kTokens) bad_rope[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < kTokens * kPairs; i += kWarps * 32) {
        const long long ti = static_cast<long long>(blockIdx.x) * kTokens + i / kPairs;
        if (ti < p.T) {
            const float4 g = kTokens > 1 ? turns[i % kPairs] : p.turns[i % kPairs];
            const int rp = p.rope_positions[static_cast<size_t>(__float_as_int(g.w)) * p.T + ti];
            if (rp < 0 || rp >= (1 << 24)) bad_rope[i / kPairs] = 1;
            // pair 8 s + j at 8 j + s: the eight lanes of a row read a line
            const int at = (i % 8) * 8 + i % kPairs / 8;
            const float4 f = cos_sin(rp & ((1 << 24) - 1), g);
            cs_all[i / kPairs][at] = make_float2(f.x, f.y);
            if constexpr (k4) low_all[i / kPairs][at] = make_float2(f.z, f.w);
        }
    }
    int code = 0;
    int64_t page = -1;
    if (kv_warp) {
        int lo = 0, hi = 0;
        if (b >= 0 && b < p.B) {
            lo = p.indptr[b];
            hi = p.indptr[b + 1];
        }
        if (b < 0 || b >= p.B || lo < 0 || hi < lo || hi > p.num_indices || pos < 0 ||
            pos >= (1 << 24) ||
            static_cast<int64_t>(pos) >= static_cast<int64_t>(hi - lo) * p.page_size) {
            code = kDeviceBadPosition;
        } else {
            page = p.indices[lo + pos / p.page_size];
            if (page < 0 || page >= p.num_pages)
                code = kDeviceBadPage;
            else if (p.refcount[page] != 1)
                code = kDeviceSharedPage;
        }
    }
    __syncthreads();
    if (!have) return;
    const float2* cs = cs_all[local] + s;

    if (kv_warp) {
        if (code == 0 && bad_rope[local]) code = kDeviceBadPosition;
        if (code != 0 && wi == 0 && lane == 0) record_status(p.status, p.epoch, code);
        // the token's first row in the pools, and what a head's rows and scales
        // are apart
        const int slot = code == 0 ? pos & (p.page_size - 1) : 0;
        const size_t row0 = row_index(p.layout, code == 0 ? page : 0, slot, 0, p.Hkv, p.page_size);
        const int stride = p.layout == 0 ? 1 : p.page_size;
        const uint16_t* k_in = p.k + static_cast<size_t>(t) * p.Hkv * kHeadDim;
        const uint16_t* v_in = p.v + static_cast<size_t>(t) * p.Hkv * kHeadDim;
        for (int task = wi; task < kv_tasks && code == 0; task += kTokenWarps) {
            const int h = task * kRowsPerTask + sub;
            const bool live = h < p.Hkv;
            if (task != wi && live) {
                k0 = load_slice(k_in + h * kHeadDim, s);
                v0 = load_slice(v_in + h * kHeadDim, s);
            }
            if (!live) k0 = v0 = Slice{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
            const int hd = live ? h : 0;
            const size_t row = row0 + static_cast<size_t>(hd) * stride;
            if constexpr (k4) {
                const size_t sc = scale_index(page, slot, hd, p.Hkv, p.page_size);
                hold_slice(static_cast<uint8_t*>(p.k_pages) + row * kCodeBytes, p.k_scales + sc,
                           rotate_exact(k0, cs, low_all[local] + s), s, live);
                hold_slice(static_cast<uint8_t*>(p.v_pages) + row * kCodeBytes, p.v_scales + sc, v0,
                           s, live);
            } else if (live) {
                store_slice(static_cast<uint16_t*>(p.k_pages) + row * kHeadDim, s, rotate(k0, cs));
                store_slice(static_cast<uint16_t*>(p.v_pages) + row * kHeadDim, s, v0);
            }
        }
    }
    // Query rows, a batch of tasks' loads ahead of its stores (q_out may be q).
    // The warps are taken from the last on, behind the KV warps.
    const uint16_t* q_in = p.q + static_cast<size_t>(t) * p.Hq * kHeadDim;
    uint16_t* q_to = p.q_out + static_cast<size_t>(t) * p.Hq * kHeadDim;
    for (int h0 = (kTokenWarps - 1 - wi) * kRowsPerTask + sub; h0 - sub < p.Hq;
         h0 += kTokenWarps * kRowsPerTask * kBatch) {
        Slice x[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int h = h0 + j * kTokenWarps * kRowsPerTask;
            if (h < p.Hq) x[j] = load_slice(q_in + h * kHeadDim, s);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int h = h0 + j * kTokenWarps * kRowsPerTask;
            if (h < p.Hq) store_slice(q_to + h * kHeadDim, s, rotate(x[j], cs));
        }
    }
}

template <bool k4, int kTokens>
cudaError_t launch(const AxesAppendParams& p, cudaStream_t stream) {
    const long long blocks = (static_cast<long long>(p.T) + kTokens - 1) / kTokens;
    axes_append_kernel<k4, kTokens>
        <<<static_cast<unsigned>(blocks), kWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_axes_append(const AxesAppendParams& p, cudaStream_t stream) {
    if (p.T < 1) return cudaErrorInvalidConfiguration;
    // Four tokens a block form their angles with every thread; a call of few
    // tokens spreads each over a block of its own while these are all resident at
    // once, four on each of the GB300's 152 SMs (608 tokens of 32 and 8 heads into
    // 4-bit pages 7.4 us, in fours 7.9; 700 tokens 10.7 and 8.7; bf16 pages 6.4 and
    // 7.1, 8.3 and 7.5).
    constexpr int kResidentBlocks = 152 * 4;
    const bool k4 = p.k_scales != nullptr;
    if (p.T <= kResidentBlocks) return k4 ? launch<true, 1>(p, stream) : launch<false, 1>(p, stream);
    return k4 ? launch<true, 4>(p, stream) : launch<false, 4>(p, stream);
}

}  // namespace oxd
