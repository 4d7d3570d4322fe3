// Page copies between paged caches for sm_103a, K and V together: bit for bit
// between equal formats, held in 4 bits from bf16 rows, or written back as
// bf16 from 4-bit rows (oxd_copy_pages).
//
// Bytes bound it: every row is read once and written once. The work is cut
// into slices of one (pair, tensor): 32 rows of 128 columns that eight warps
// take four at a time, eight lanes a row (16 columns of a lane: 8s .. 8s + 7
// and 64 + 8s ..), so every access is 16 bytes of bf16 or 4 bytes of codes and
// a 4-bit group of 32 columns is four lanes. Rows are counted in the
// destination's order, so its writes are contiguous; with equal layouts the
// reads are too. Equal formats and layouts need no rows: a page is one run of
// bytes, copied 16 bytes a lane.
#include <cuda_bf16.h>

#include "oxd_e2m1.cuh"
#include "oxd_internal.h"
#include "oxd_ptx.cuh"

namespace oxd {
namespace {

constexpr int kThreads = 256;

// The pages of pair i, or false with the error (or the skipped pair) dealt with.
__device__ __forceinline__ bool pair_pages(const CopyPagesParams& p, int i, bool first, int* src,
                                           int* dst) {
    const int s = p.src_pages[i], d = p.dst_pages[i];
    *src = s;
    *dst = d;
    if (s == -1) return false;
    int code = 0;
    if (s < 0 || s >= p.src.num_pages || d < 0 || d >= p.dst.num_pages)
        code = kDeviceBadPage;
    else if (p.refcount != nullptr && p.refcount[d] != 1)
        code = kDeviceSharedPage;
    if (code != 0 && first && threadIdx.x == 0) record_status(p.status, p.epoch, code);
    return code == 0;
}

// Equal formats and layouts: kPieces 16-byte pieces a thread.
template <bool k4>
__global__ void __launch_bounds__(kThreads) copy_pages_kernel(const __grid_constant__ CopyPagesParams p) {
    constexpr int kPieces = 4;
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.last_epoch = p.epoch;
    const int page_rows = p.page_size * p.H;
    const int row_pieces = (k4 ? kCodeBytes : kHeadDim * 2) / 16;
    const int data = page_rows * row_pieces;                     // pieces of a page's rows
    const int all = data + (k4 ? page_rows * kScaleBytes / 16 : 0);  // and of its scales
    const int slice = blockIdx.x >> 1, tensor = blockIdx.x & 1;
    for (int i = blockIdx.y; i < p.n; i += gridDim.y) {
        int src, dst;
        if (!pair_pages(p, i, blockIdx.x == 0, &src, &dst)) continue;
        const uint4* from = reinterpret_cast<const uint4*>(p.src.data[tensor]) +
                            static_cast<size_t>(src) * data;
        uint4* to = reinterpret_cast<uint4*>(p.dst.data[tensor]) + static_cast<size_t>(dst) * data;
        uint4 v[kPieces];
        const int c0 = slice * kThreads * kPieces + threadIdx.x;
        const uint4* from_s = nullptr;
        uint4* to_s = nullptr;
        if constexpr (k4) {
            from_s = reinterpret_cast<const uint4*>(p.src.scales[tensor]) +
                     static_cast<size_t>(src) * (all - data) - data;
            to_s = reinterpret_cast<uint4*>(p.dst.scales[tensor]) +
                   static_cast<size_t>(dst) * (all - data) - data;
        }
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const int c = c0 + j * kThreads;
            if (c < all) v[j] = k4 && c >= data ? from_s[c] : from[c];
        }
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const int c = c0 + j * kThreads;
            if (c < all) {
                if (k4 && c >= data)
                    to_s[c] = v[j];
                else
                    to[c] = v[j];
            }
        }
    }
}

// A page's rows of one tensor: where they and their scales begin.
struct PageRows {
    uint8_t* data;
    uint16_t* scales;
};

template <bool k4>
__device__ __forceinline__ PageRows page_rows_of(const PagePools& c, int tensor, int page,
                                                 int rows) {
    const size_t first = static_cast<size_t>(page) * rows;
    return {c.data[tensor] + first * (k4 ? kCodeBytes : kHeadDim * 2),
            k4 ? c.scales[tensor] + first * kRowScales : nullptr};
}

// What a lane holds of a row: as bf16 pairs, or as codes and the scales of its
// two groups. row: in the pool's order; sc: in the order of scales (heads before
// tokens).
template <bool k4>
struct Piece;
template <>
struct Piece<false> {
    uint4 lo, hi;
    __device__ __forceinline__ void load(const PageRows& c, uint32_t row, uint32_t, int s) {
        const uint4* r = reinterpret_cast<const uint4*>(c.data) + row * 16 + s;
        lo = r[0];
        hi = r[8];
    }
    __device__ __forceinline__ void store(const PageRows& c, uint32_t row, uint32_t, int s,
                                          bool live) const {
        uint4* r = reinterpret_cast<uint4*>(c.data) + row * 16 + s;
        if (live) {
            r[0] = lo;
            r[8] = hi;
        }
    }
};
template <>
struct Piece<true> {
    uint32_t lo, hi;      // codes of columns 8s .. 8s + 7 and 64 + 8s ..
    uint32_t s_lo, s_hi;  // f16 scales of the groups they lie in
    __device__ __forceinline__ void load(const PageRows& c, uint32_t row, uint32_t sc, int s) {
        const uint32_t* r = reinterpret_cast<const uint32_t*>(c.data) + row * 16 + s;
        lo = r[0];
        hi = r[8];
        s_lo = c.scales[sc * kRowScales + s / 4];
        s_hi = c.scales[sc * kRowScales + 2 + s / 4];
    }
    // Every lane of the warp calls it; `live` lanes store.
    __device__ __forceinline__ void store(const PageRows& c, uint32_t row, uint32_t sc, int s,
                                          bool live) const {
        const uint32_t a = __shfl_xor_sync(0xffffffffu, s_lo, 4);
        const uint32_t b = __shfl_xor_sync(0xffffffffu, s_hi, 4);
        if (live) {
            uint32_t* r = reinterpret_cast<uint32_t*>(c.data) + row * 16 + s;
            r[0] = lo;
            r[8] = hi;
            if (s == 0)
                *reinterpret_cast<uint2*>(c.scales + sc * kRowScales) =
                    make_uint2(s_lo | (a << 16), s_hi | (b << 16));
        }
    }
};

__device__ __forceinline__ uint4 unhold(uint32_t code, uint32_t scale) {
    const float s = __half2float(__ushort_as_half(static_cast<uint16_t>(scale)));
    uint32_t h[4], o[4];
    codes_to_f16(code, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = f16x2_floats(h[i]);
        o[i] = pack_bf16x2(f.x * s, f.y * s);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ void convert(const Piece<false>& a, Piece<false>& b) { b = a; }
__device__ __forceinline__ void convert(const Piece<true>& a, Piece<true>& b) { b = a; }
__device__ __forceinline__ void convert(const Piece<false>& a, Piece<true>& b) {
    hold_eight(a.lo, b.lo, b.s_lo);
    hold_eight(a.hi, b.hi, b.s_hi);
}
__device__ __forceinline__ void convert(const Piece<true>& a, Piece<false>& b) {
    b.lo = unhold(a.lo, a.s_lo);
    b.hi = unhold(a.hi, a.s_hi);
}

// Other formats or layouts: kRows rows a thread's eight lanes take. A block's
// life is a chain of loads (pair, refcount, rows), so the more blocks an SM holds
// the better: eight at 32 registers, though a few spill, pack and unpack 4096
// pages in 123 us, six at 40 registers in 130, as the compiler would have it
// (48) in 133. One row a thread 146, four 137.
constexpr int kRows = 2;
constexpr int kSliceRows = kThreads / 8 * kRows;

template <bool kSrc4, bool kDst4>
__global__ void __launch_bounds__(kThreads, 8)
    convert_pages_kernel(const __grid_constant__ CopyPagesParams p) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.last_epoch = p.epoch;
    const int s = threadIdx.x & 7;
    const int page_rows = p.page_size * p.H;
    const int slice = blockIdx.x >> 1, tensor = blockIdx.x & 1;
    // Rows are counted in the destination's order, (token, head) or (head,
    // token); `inner` counts the second.
    const uint32_t inner = p.dst.layout == 0 ? p.H : p.page_size;
    const uint32_t outer = p.dst.layout == 0 ? p.page_size : p.H;
    for (int i = blockIdx.y; i < p.n; i += gridDim.y) {
        int src, dst;
        if (!pair_pages(p, i, blockIdx.x == 0, &src, &dst)) continue;
        const PageRows from = page_rows_of<kSrc4>(p.src, tensor, src, page_rows);
        const PageRows to = page_rows_of<kDst4>(p.dst, tensor, dst, page_rows);
        Piece<kSrc4> a[kRows];
        uint32_t row[kRows], sc[kRows];
        bool live[kRows];
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const int r = slice * kSliceRows + j * (kThreads / 8) + (threadIdx.x >> 3);
            live[j] = r < page_rows;
            row[j] = live[j] ? r : 0;
            uint32_t hi = row[j];
            if (inner > 1) hi = p.inner_magic ? __umulhi(row[j], p.inner_magic) : row[j] / inner;
            const uint32_t other = (row[j] - hi * inner) * outer + hi;  // in the other order
            sc[j] = p.dst.layout == 0 ? other : row[j];
            a[j].load(from, p.src.layout == p.dst.layout ? row[j] : other, sc[j], s);
        }
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            Piece<kDst4> b;
            convert(a[j], b);
            b.store(to, row[j], sc[j], s, live[j]);
        }
    }
}

// A row of blocks for every pair (the pairs in turn past kMaxPairRows): K and V in
// turn, slice by slice.
template <class F>
cudaError_t launch(F kernel, const CopyPagesParams& p, long long slices, cudaStream_t stream) {
    const int pairs = p.n < 1 ? 1 : p.n > kMaxPairRows ? kMaxPairRows : p.n;
    const dim3 grid(2 * static_cast<unsigned>(slices), pairs);
    kernel<<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_copy_pages(const CopyPagesParams& p, cudaStream_t stream) {
    const bool s4 = p.src.scales[0] != nullptr, d4 = p.dst.scales[0] != nullptr;
    const long long rows = static_cast<long long>(p.page_size) * p.H;
    if (s4 == d4 && p.src.layout == p.dst.layout) {
        const long long pieces = rows * (s4 ? kCodeBytes + kScaleBytes : kHeadDim * 2) / 16;
        const long long slices = (pieces + kThreads * 4 - 1) / (kThreads * 4);
        return s4 ? launch(copy_pages_kernel<true>, p, slices, stream)
                  : launch(copy_pages_kernel<false>, p, slices, stream);
    }
    const long long slices = (rows + kSliceRows - 1) / kSliceRows;
    if (s4 && d4) return launch(convert_pages_kernel<true, true>, p, slices, stream);
    if (s4) return launch(convert_pages_kernel<true, false>, p, slices, stream);
    if (d4) return launch(convert_pages_kernel<false, true>, p, slices, stream);
    return launch(convert_pages_kernel<false, false>, p, slices, stream);
}

}  // namespace oxd
