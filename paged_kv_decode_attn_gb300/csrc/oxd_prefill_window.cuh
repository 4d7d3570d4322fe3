// A tile's sight under a window, as the prefill kernels use it.
#pragma once

#include "oxd_prefill.h"
#include "oxd_ptx.cuh"

namespace oxd {
namespace {

// Tokens are counted from the piece's first, without the skipped pages.
struct TileWindow {
    int front, skip;  // pages of the piece from `front` on lie `skip` further in the table
    int p0;           // position of the tile's first query
    int sinks;
    int lo;           // tokens in [sinks, lo) are seen by no row of the tile

    __device__ __forceinline__ void init(const PrefillParams& p, const PrefillUnit& u) {
        const WindowPages w = window_pages(p.window, p.sinks, u.p0, p.page_size);
        front = w.front - u.kv_begin / p.page_size;
        skip = w.skip;
        p0 = u.p0 - skip * p.page_size - u.kv_begin;
        sinks = p.sinks - u.kv_begin;
        lo = p0 - p.window + 1;
    }
    // Entry of the block table, from the request's first, of page j of the piece.
    __device__ __forceinline__ int64_t entry(const PrefillUnit& u, int ps, int j) const {
        return static_cast<int64_t>(u.kv_begin / ps) + j + (j >= front ? skip : 0);
    }
    // Whether the piece's pages lie inside the index array.
    __device__ __forceinline__ bool inside(const PrefillUnit& u, int ps, int64_t nnz) const {
        return u.page_base >= 0 && u.page_base + entry(u, ps, u.n_pages - 1) < nnz;
    }
    // Rows [hidden0, hidden1) of a stage of `n` tokens that starts at `base` are tokens
    // that no row sees.
    __device__ __forceinline__ int hidden0(int base, int n) const {
        return min(max(sinks - base, 0), n);
    }
    __device__ __forceinline__ int hidden1(int base, int n) const { return min(lo - base, n); }
    __device__ __forceinline__ bool hides(int base, int n) const {
        return hidden1(base, n) > hidden0(base, n);
    }
};

}  // namespace
}  // namespace oxd
