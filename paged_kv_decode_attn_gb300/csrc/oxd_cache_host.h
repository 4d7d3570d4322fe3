// Checks that the C entries of calls without a plan share (oxd_quant_host.cpp,
// oxd_window_host.cpp): the device of a call's arrays, and the arrays of a cache.
// Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <initializer_list>

#include "../../include/oxd.h"
#include "oxd_host_util.h"
#include "oxd_internal.h"

namespace oxd {
namespace {  // (per file: a library's statics are its own)

inline bool page_size_ok(int ps) { return ps == 8 || ps == 16 || ps == 32 || ps == 64; }
inline bool layout_ok(int l) { return l == OXD_LAYOUT_NHD || l == OXD_LAYOUT_HND; }

typedef CUresult (*PointerAttributeFn)(void*, CUpointer_attribute, CUdeviceptr);

inline PointerAttributeFn pointer_attribute() {
    static const PointerAttributeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuPointerGetAttribute", &p, 12000,
                                                         cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return reinterpret_cast<PointerAttributeFn>(ok ? p : nullptr);
    }();
    return fn;
}

// A call with device memory of another device than the calling thread's current
// one among its arrays (NULL ones aside) is refused before a kernel on the wrong
// device touches it; managed memory, and memory the driver does not know, is
// taken. One attribute of the driver's is 32 ns an array, the runtime's 55.
// With one device there is nothing to ask.
inline bool on_current_device(std::initializer_list<const void*> arrays) {
    static const int devices = [] {
        int n = 0;
        if (cudaGetDeviceCount(&n) == cudaSuccess) return n;
        cudaGetLastError();
        return 0;  // no device to be wrong about: the launch reports it
    }();
    int cur = -1;
    if (devices < 2 || cudaGetDevice(&cur) != cudaSuccess) return true;
    const PointerAttributeFn attribute = pointer_attribute();
    for (const void* p : arrays) {
        int dev = -1;
        if (p == nullptr ||
            (attribute != nullptr &&
             attribute(&dev, CU_POINTER_ATTRIBUTE_DEVICE_ORDINAL,
                       reinterpret_cast<CUdeviceptr>(p)) == CUDA_SUCCESS &&
             dev == cur))
            continue;
        cudaPointerAttributes a;
        if (cudaPointerGetAttributes(&a, p) != cudaSuccess)
            cudaGetLastError();
        else if (a.type == cudaMemoryTypeDevice && a.device != cur)
            return false;
    }
    return true;
}

// The arrays of one cache: K, V and, in 4 bits, their scales.
struct Pools {
    Span s[4];
    int n;
};

inline Pools pool_spans(const oxd_kv_pools& p, bool e2m1, int64_t pages, int ps, int H) {
    const size_t rows = static_cast<size_t>(pages) * ps * H;
    if (!e2m1) return {{span(p.k, rows * kHeadDim * 2), span(p.v, rows * kHeadDim * 2)}, 2};
    return {{span(p.k, rows * kCodeBytes), span(p.v, rows * kCodeBytes),
             span(p.k_scales, rows * kScaleBytes), span(p.v_scales, rows * kScaleBytes)},
            4};
}

inline bool pools_aligned(const oxd_kv_pools& p) {
    return aligned(p.k, 16) && aligned(p.v, 16) && aligned(p.k_scales, 16) &&
           aligned(p.v_scales, 16);
}

}  // namespace
}  // namespace oxd
