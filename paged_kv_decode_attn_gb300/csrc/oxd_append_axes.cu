// Rotary embedding with position axes + paged KV append for sm_103a, into
// bf16 pages (oxd_rope_axes_append) or 4-bit pages (oxd_quant_rope_append).
//
// One warp per row: the K and V rows of a (token, KV head), or a query row.
// Lane l owns columns 2l, 2l + 1 and 64 + 2l, 65 + 2l, the two rotary pairs
// 2l and 2l + 1. Angles and rotation in double; the K row of a 4-bit cache is
// the bf16 number nearest to the rotated value.
#include <cuda_bf16.h>

#include "oxd_e2m1.cuh"
#include "oxd_internal.h"
#include "oxd_ptx.cuh"

namespace oxd {
namespace {

constexpr int kWarps = 8;

struct Row {
    uint32_t lo, hi;  // columns (2l, 2l + 1) and (64 + 2l, 65 + 2l), bf16 pairs
};

__device__ __forceinline__ Row load_row(const uint16_t* src, int lane) {
    return {*reinterpret_cast<const uint32_t*>(src + 2 * lane),
            *reinterpret_cast<const uint32_t*>(src + 64 + 2 * lane)};
}

__device__ __forceinline__ Row rotate(Row x, const double (&c)[2], const double (&s)[2]) {
    const float a0 = __uint_as_float(x.lo << 16), a1 = __uint_as_float(x.lo & 0xffff0000u);
    const float b0 = __uint_as_float(x.hi << 16), b1 = __uint_as_float(x.hi & 0xffff0000u);
    __nv_bfloat162 lo, hi;
    lo.x = __double2bfloat16(a0 * c[0] - b0 * s[0]);
    lo.y = __double2bfloat16(a1 * c[1] - b1 * s[1]);
    hi.x = __double2bfloat16(b0 * c[0] + a0 * s[0]);
    hi.y = __double2bfloat16(b1 * c[1] + a1 * s[1]);
    return {*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi)};
}

__device__ __forceinline__ void store_row(uint16_t* dst, Row x, int lane) {
    *reinterpret_cast<uint32_t*>(dst + 2 * lane) = x.lo;
    *reinterpret_cast<uint32_t*>(dst + 64 + 2 * lane) = x.hi;
}

// Holds a row in 4 bits: columns below 64 are groups 0 (lanes 0..15) and 1
// (lanes 16..31), the others groups 2 and 3.
__device__ __forceinline__ void hold_row(uint8_t* codes, uint16_t* scales, Row x, int lane) {
    const uint32_t w[2] = {x.lo, x.hi};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float x0 = __uint_as_float(w[j] << 16), x1 = __uint_as_float(w[j] & 0xffff0000u);
        float amax = fmaxf(fabsf(x0), fabsf(x1));
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const uint16_t s = group_scale(amax);
        codes[32 * j + lane] = static_cast<uint8_t>(code_pair(x0, x1, scale_inverse(s)));
        if ((lane & 15) == 0) scales[2 * j + lane / 16] = s;
    }
}

template <bool k4>
__global__ void __launch_bounds__(kWarps * 32) axes_append_kernel(const AxesAppendParams p) {
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.last_epoch = p.epoch;
    const int lane = threadIdx.x & 31;
    const long long gw = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int heads = p.Hkv + p.Hq;
    if (gw >= static_cast<long long>(p.T) * heads) return;
    const int t = static_cast<int>(gw / heads), h = static_cast<int>(gw % heads);
    double c[2], s[2];
    bool ok_rope = true;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int pos = p.rope_positions[static_cast<size_t>(p.pair_axis[2 * lane + j]) * p.T + t];
        ok_rope = ok_rope && pos >= 0 && pos < (1 << 24);
        const double turns = (pos & ((1 << 24) - 1)) * p.turns[2 * lane + j];
        sincospi(2.0 * (turns - rint(turns)), &s[j], &c[j]);
    }
    ok_rope = __all_sync(0xffffffffu, ok_rope);
    if (h >= p.Hkv) {
        const size_t row = (static_cast<size_t>(t) * p.Hq + h - p.Hkv) * kHeadDim;
        store_row(p.q_out + row, rotate(load_row(p.q + row, lane), c, s), lane);
        return;
    }
    const int b = p.token_request[t], pos = p.positions[t];
    int code = 0, lo = 0, hi = 0;
    int64_t page = -1;
    if (b >= 0 && b < p.B) {
        lo = p.indptr[b];
        hi = p.indptr[b + 1];
    }
    if (b < 0 || b >= p.B || lo < 0 || hi < lo || hi > p.num_indices || pos < 0 ||
        pos >= (1 << 24) || !ok_rope ||
        static_cast<int64_t>(pos) >= static_cast<int64_t>(hi - lo) * p.page_size) {
        code = kDeviceBadPosition;
    } else {
        page = p.indices[lo + pos / p.page_size];
        if (page < 0 || page >= p.num_pages)
            code = kDeviceBadPage;
        else if (p.refcount[page] != 1)
            code = kDeviceSharedPage;
    }
    if (code != 0) {
        if (h == 0 && lane == 0) record_status(p.status, p.epoch, code);
        return;
    }
    const size_t src = (static_cast<size_t>(t) * p.Hkv + h) * kHeadDim;
    const Row k = rotate(load_row(p.k + src, lane), c, s), v = load_row(p.v + src, lane);
    const int slot = pos % p.page_size;
    const size_t dst = row_index(p.layout, page, slot, h, p.Hkv, p.page_size);
    if constexpr (k4) {
        const size_t sc = scale_index(page, slot, h, p.Hkv, p.page_size);
        hold_row(static_cast<uint8_t*>(p.k_pages) + dst * kCodeBytes, p.k_scales + sc, k, lane);
        hold_row(static_cast<uint8_t*>(p.v_pages) + dst * kCodeBytes, p.v_scales + sc, v, lane);
    } else {
        store_row(static_cast<uint16_t*>(p.k_pages) + dst * kHeadDim, k, lane);
        store_row(static_cast<uint16_t*>(p.v_pages) + dst * kHeadDim, v, lane);
    }
}

}  // namespace

cudaError_t launch_axes_append(const AxesAppendParams& p, cudaStream_t stream) {
    const long long warps = static_cast<long long>(p.T) * (p.Hkv + p.Hq);
    const long long blocks = (warps + kWarps - 1) / kWarps;
    if (p.T < 1 || blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (p.k_scales != nullptr)
        axes_append_kernel<true><<<static_cast<unsigned>(blocks), kWarps * 32, 0, stream>>>(p);
    else
        axes_append_kernel<false><<<static_cast<unsigned>(blocks), kWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace oxd
