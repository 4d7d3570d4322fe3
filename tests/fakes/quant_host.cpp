// A stand-in for the device under the C entries of the appends and the page copies, for tests of
// their host side: "allocations" on devices the test names, and launches that only keep their
// parameters.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstring>

#include "oxd_internal.h"

namespace {

constexpr int kMost = 64;
struct Allocation {
    uintptr_t lo, hi;
    int device, type;
} allocations[kMost];
int n_allocations = 0, current = 0, launches = 0;
float turns[oxd::kHeadDim / 2][4];

const Allocation* find(const void* p) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    for (int i = 0; i < n_allocations; ++i)
        if (a >= allocations[i].lo && a < allocations[i].hi) return &allocations[i];
    return nullptr;
}

CUresult pointer_attribute(void* data, CUpointer_attribute what, CUdeviceptr p) {
    const Allocation* a = find(reinterpret_cast<const void*>(p));
    if (a == nullptr || what != CU_POINTER_ATTRIBUTE_DEVICE_ORDINAL)
        return CUDA_ERROR_INVALID_VALUE;
    *static_cast<int*>(data) = a->device;
    return CUDA_SUCCESS;
}

}  // namespace

extern "C" {

void fake_reset(int device) {
    current = device;
    n_allocations = launches = 0;
}
void fake_allocate(uintptr_t at, size_t bytes, int device, int type) {
    if (n_allocations < kMost) allocations[n_allocations++] = {at, at + bytes, device, type};
}
int fake_launches(void) { return launches; }
const float* fake_turns(void) { return &turns[0][0]; }

cudaError_t cudaGetDevice(int* device) {
    *device = current;
    return cudaSuccess;
}
cudaError_t cudaGetDeviceCount(int* n) {
    *n = 2;
    return cudaSuccess;
}
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes* out, const void* p) {
    std::memset(out, 0, sizeof(*out));
    const Allocation* a = find(p);
    out->type = a == nullptr ? cudaMemoryTypeUnregistered : static_cast<cudaMemoryType>(a->type);
    out->device = a == nullptr ? -2 : a->device;
    return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char* name, void** f, unsigned int,
                                             unsigned long long,
                                             cudaDriverEntryPointQueryResult* result) {
    const bool known = std::strcmp(name, "cuPointerGetAttribute") == 0;
    *f = known ? reinterpret_cast<void*>(&pointer_attribute) : nullptr;
    *result = known ? cudaDriverEntryPointSuccess : cudaDriverEntryPointSymbolNotFound;
    return cudaSuccess;
}
}

namespace oxd {
uint32_t next_run_epoch() { return 1; }
cudaError_t launch_axes_append(const AxesAppendParams& p, cudaStream_t) {
    std::memcpy(turns, p.turns, sizeof(turns));
    ++launches;
    return cudaSuccess;
}
cudaError_t launch_copy_pages(const CopyPagesParams&, cudaStream_t) {
    ++launches;
    return cudaSuccess;
}
}  // namespace oxd
