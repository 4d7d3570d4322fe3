// Page copies between paged caches for sm_103a, K and V together: bit for bit
// between equal formats, held in 4 bits from bf16 rows, or written back as
// bf16 from 4-bit rows (oxd_copy_pages).
//
// One warp per (pair, tensor, token, head) row.
#include <cuda_bf16.h>

#include "oxd_e2m1.cuh"
#include "oxd_internal.h"
#include "oxd_ptx.cuh"

namespace oxd {
namespace {

constexpr int kWarps = 8;

template <bool kSrc4, bool kDst4>
__global__ void __launch_bounds__(kWarps * 32) copy_pages_kernel(const CopyPagesParams p) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.last_epoch = p.epoch;
    const int lane = threadIdx.x & 31;
    const long long rows = static_cast<long long>(p.n) * 2 * p.page_size * p.H;
    for (long long r = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); r < rows;
         r += static_cast<long long>(gridDim.x) * kWarps) {
        long long x = r;
        const int h = static_cast<int>(x % p.H);
        x /= p.H;
        const int t = static_cast<int>(x % p.page_size);
        x /= p.page_size;
        const int tensor = static_cast<int>(x & 1);
        const int i = static_cast<int>(x >> 1);
        const int src = p.src_pages[i], dst = p.dst_pages[i];
        if (src == -1) continue;
        int code = 0;
        if (src < 0 || src >= p.src.num_pages || dst < 0 || dst >= p.dst.num_pages)
            code = kDeviceBadPage;
        else if (p.refcount != nullptr && p.refcount[dst] != 1)
            code = kDeviceSharedPage;
        if (code != 0) {
            if (lane == 0 && t == 0 && h == 0) record_status(p.status, p.epoch, code);
            continue;
        }
        const size_t from = row_index(p.src.layout, src, t, h, p.H, p.page_size);
        const size_t to = row_index(p.dst.layout, dst, t, h, p.H, p.page_size);
        const size_t from_s = scale_index(src, t, h, p.H, p.page_size);
        const size_t to_s = scale_index(dst, t, h, p.H, p.page_size);
        if constexpr (kSrc4 && kDst4) {
            reinterpret_cast<uint16_t*>(p.dst.data[tensor] + to * kCodeBytes)[lane] =
                reinterpret_cast<const uint16_t*>(p.src.data[tensor] + from * kCodeBytes)[lane];
            if (lane < kRowScales)
                p.dst.scales[tensor][to_s + lane] = p.src.scales[tensor][from_s + lane];
        } else {
            // lane: columns [4 lane, 4 lane + 4), group lane / 8
            uint2 v;
            if constexpr (kSrc4) {
                const uint32_t w = reinterpret_cast<const uint16_t*>(p.src.data[tensor] +
                                                                     from * kCodeBytes)[lane];
                const float s = __half2float(
                    __ushort_as_half(p.src.scales[tensor][from_s + lane / 8]));
                uint32_t c[4];
                codes_to_f16(w, c);
                const float2 a = f16x2_floats(c[0]), b = f16x2_floats(c[1]);
                v.x = pack_bf16x2(a.x * s, a.y * s);
                v.y = pack_bf16x2(b.x * s, b.y * s);
            } else {
                v = reinterpret_cast<const uint2*>(p.src.data[tensor] + from * kHeadDim * 2)[lane];
            }
            if constexpr (kDst4) {
                const float x0 = __uint_as_float(v.x << 16), x1 = __uint_as_float(v.x & 0xffff0000u);
                const float x2 = __uint_as_float(v.y << 16), x3 = __uint_as_float(v.y & 0xffff0000u);
                float amax = fmaxf(fmaxf(fabsf(x0), fabsf(x1)), fmaxf(fabsf(x2), fabsf(x3)));
#pragma unroll
                for (int o = 1; o < 8; o <<= 1)
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                const uint16_t s = group_scale(amax);
                const float inv = scale_inverse(s);
                reinterpret_cast<uint16_t*>(p.dst.data[tensor] + to * kCodeBytes)[lane] =
                    static_cast<uint16_t>(code_pair(x0, x1, inv) | (code_pair(x2, x3, inv) << 8));
                if ((lane & 7) == 0) p.dst.scales[tensor][to_s + lane / 8] = s;
            } else {
                reinterpret_cast<uint2*>(p.dst.data[tensor] + to * kHeadDim * 2)[lane] = v;
            }
        }
    }
}

}  // namespace

cudaError_t launch_copy_pages(const CopyPagesParams& p, cudaStream_t stream) {
    const long long rows = static_cast<long long>(p.n) * 2 * p.page_size * p.H;
    const long long blocks = (rows + kWarps - 1) / kWarps;
    const unsigned grid = static_cast<unsigned>(blocks < 1 ? 1 : blocks > 152 * 8 ? 152 * 8 : blocks);
    const bool s4 = p.src.scales[0] != nullptr, d4 = p.dst.scales[0] != nullptr;
    if (s4 && d4)
        copy_pages_kernel<true, true><<<grid, kWarps * 32, 0, stream>>>(p);
    else if (s4)
        copy_pages_kernel<true, false><<<grid, kWarps * 32, 0, stream>>>(p);
    else if (d4)
        copy_pages_kernel<false, true><<<grid, kWarps * 32, 0, stream>>>(p);
    else
        copy_pages_kernel<false, false><<<grid, kWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace oxd
