// Decode attention over a 4-bit paged cache for sm_103a (oxd_quant_decode_run).
//
// The planner's work units (runs of pages of one request for one KV head) as
// for the bf16 decode; four warps a CTA, each taking every fourth query row
// of the group over the unit's tokens with the F32 online softmax on CUDA
// cores.
#include <cuda_bf16.h>

#include <type_traits>

#include "oxd_e2m1.cuh"
#include "oxd_internal.h"
#include "oxd_ptx.cuh"

namespace oxd {
namespace {

constexpr int kWarps = 4;

template <class WL>
__global__ void __launch_bounds__(kWarps * 32)
    quant_decode_kernel(const __grid_constant__ QuantDecodeParams qp,
                        const __grid_constant__ WL work) {
    const DecodeParams& p = qp.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    if (threadIdx.x == 0) {
        if (blockIdx.x == 0) {
            *p.last_epoch = p.epoch;
            if (p.clear_stamp != nullptr) *p.clear_stamp = 0ull;
        }
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    const int4* units = p.units;
    int u0, u1;
    bool listed = false;
    if constexpr (std::is_same<WL, WorkList>::value) {
        if (units == nullptr) {
            units = work.unit;
            u0 = work.cta_begin[blockIdx.x];
            u1 = work.cta_begin[blockIdx.x + 1];
            listed = true;
        }
    }
    if (!listed) {
        const int4 r = p.cta_rec[2 * blockIdx.x];
        u0 = r.x;
        u1 = r.y;
    }
    if ((p.ws_stamp != nullptr && *p.ws_stamp != p.stamp) || u0 < 0 || u1 > p.n_units) {
        if (threadIdx.x == 0) record_status(p.status, p.epoch, kDevicePlanMismatch);
        return;
    }
    const int ps = p.page_size, G = p.group;
    for (int u = u0; u < u1; ++u) {
        const int4 it = units[u];
        const int n_pages = it.y & ((1 << kUnitPagesBits) - 1);
        const int last_len = (it.y >> kUnitPagesBits) & 0x7f;
        const int b = it.z & ((1 << kUnitBBits) - 1);
        const int row0 = ((it.z >> kUnitBBits) & 1) * 16;
        const int h = static_cast<int>(static_cast<uint32_t>(it.z) >> (kUnitBBits + 1));
        const bool unit_ok = n_pages >= 1 && it.x >= 0 &&
                             static_cast<int64_t>(it.x) + n_pages <= p.nnz && b < p.batch &&
                             h < p.num_kv_heads && row0 < G && it.w >= -1 && it.w < p.n_slots &&
                             last_len <= ps;
        if (!unit_ok) {
            if (threadIdx.x == 0) record_status(p.status, p.epoch, kDevicePlanMismatch);
            continue;
        }
        if (threadIdx.x == 0 &&
            ((it.y < 0 && p.indptr[b] != it.x) ||
             (last_len && (p.indptr[b + 1] != it.x + n_pages || p.last_page_len[b] != last_len))))
            record_status(p.status, p.epoch, kDevicePlanMismatch);
        const int valid = last_len ? (n_pages - 1) * ps + last_len : n_pages * ps;
        for (int g = row0 + warp; g < min(G, row0 + 16); g += kWarps) {
            const size_t row = static_cast<size_t>(b) * p.num_qo_heads + h * G + g;
            const uint2 qv = reinterpret_cast<const uint2*>(p.q + row * kHeadDim)[lane];
            const float q0 = __uint_as_float(qv.x << 16), q1 = __uint_as_float(qv.x & 0xffff0000u);
            const float q2 = __uint_as_float(qv.y << 16), q3 = __uint_as_float(qv.y & 0xffff0000u);
            float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
            for (int tok = 0; tok < valid; ++tok) {
                int page = p.indices[it.x + tok / ps];
                if (page < 0 || page >= p.num_pages) {
                    if (lane == 0) record_status(p.status, p.epoch, kDeviceBadPage);
                    page = 0;
                }
                const int t = tok % ps;
                const size_t r = row_index(p.layout, page, t, h, p.num_kv_heads, ps);
                const size_t sc = scale_index(page, t, h, p.num_kv_heads, ps) + lane / 8;
                uint32_t c[4];
                codes_to_f16(reinterpret_cast<const uint16_t*>(qp.k_codes + r * kCodeBytes)[lane], c);
                const float ks = __half2float(__ushort_as_half(qp.k_scales[sc]));
                const float2 k01 = f16x2_floats(c[0]), k23 = f16x2_floats(c[1]);
                float x = ks * (q0 * k01.x + q1 * k01.y + q2 * k23.x + q3 * k23.y);
#pragma unroll
                for (int s = 1; s < 32; s <<= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
                x *= p.scale_log2;
                const float mn = fmaxf(m, x), mu = mn == -INFINITY ? 0.f : mn;
                const float al = fast_exp2(m - mu), w = fast_exp2(x - mu);
                m = mn;
                l = l * al + w;
                codes_to_f16(reinterpret_cast<const uint16_t*>(qp.v_codes + r * kCodeBytes)[lane], c);
                const float vs = w * __half2float(__ushort_as_half(qp.v_scales[sc]));
                const float2 v01 = f16x2_floats(c[0]), v23 = f16x2_floats(c[1]);
                o[0] = o[0] * al + vs * v01.x;
                o[1] = o[1] * al + vs * v01.y;
                o[2] = o[2] * al + vs * v23.x;
                o[3] = o[3] * al + vs * v23.y;
            }
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const float lse2 = l > 0.f ? m + log2f(l) : -INFINITY;
            if (it.w < 0) {
                uint2 packed;
                packed.x = pack_bf16x2(o[0] * inv, o[1] * inv);
                packed.y = pack_bf16x2(o[2] * inv, o[3] * inv);
                reinterpret_cast<uint2*>(p.out + row * kHeadDim)[lane] = packed;
                if (lane == 0 && p.lse != nullptr) p.lse[row] = lse2 * kLn2;
            } else {
                const size_t part = static_cast<size_t>(it.w) * G + g;
                reinterpret_cast<float4*>(p.part_o + part * kHeadDim)[lane] =
                    make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
                if (lane == 0) p.part_lse[part] = lse2;
            }
        }
    }
}

template <class WL>
cudaError_t launch_ex(const QuantDecodeParams& p, const WL& w, int grid, cudaStream_t stream,
                      bool pdl) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, quant_decode_kernel<WL>, p, w);
}

}  // namespace

VariantShape quant_shape(int) { return {kWarps * 32, 128, 1, 1024}; }

cudaError_t quant_occupancy(int, int* n) {
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, quant_decode_kernel<WorkList>,
                                                         kWarps * 32, 0);
}

cudaError_t launch_decode_quant(int, const CUtensorMap&, const CUtensorMap&,
                                const QuantDecodeParams& p, const WorkList* w, int grid,
                                cudaStream_t stream, bool pdl) {
    if (w != nullptr) return launch_ex(p, *w, grid, stream, pdl);
    return launch_ex(p, NoList{0}, grid, stream, pdl);
}

}  // namespace oxd
