// A tile's sight under a window, as both prefill kernels use it (their kWindow
// instances; the others compile none of it).
#pragma once

#include "oxd_prefill.h"
#include "oxd_ptx.cuh"

namespace oxd {
namespace {

template <int kStage>
struct TileWindow {
    int gap_at, skip;  // local stages from gap_at on lie `skip` stages further
    int lo, sinks;     // tokens in [sinks, lo) are seen by no row of the tile
    int kv_begin, window;

    __device__ __forceinline__ void init(const PrefillParams& p, const PrefillUnit& u) {
        const WindowStages w = window_stages(p.window, p.sinks, u.p0, kStage);
        const int first = u.kv_begin / kStage;
        skip = w.skip;
        gap_at = first < w.front ? w.front - first : 0x7fffffff;
        lo = u.p0 >= p.window ? u.p0 - p.window + 1 : 0;
        sinks = p.sinks;
        kv_begin = u.kv_begin;
        window = p.window;
    }
    // Stages of the request between the piece's first and its stage s.
    __device__ __forceinline__ int stage(int s) const { return s + (s >= gap_at ? skip : 0); }
    // First token of stage s.
    __device__ __forceinline__ int base(int s) const { return kv_begin + stage(s) * kStage; }
    // Whether the piece's pages lie inside the index array.
    __device__ __forceinline__ bool inside(const PrefillUnit& u, int n_st, int pps,
                                           int64_t nnz) const {
        return static_cast<int64_t>(u.idx_begin) + u.n_pages +
                   (n_st > gap_at ? static_cast<int64_t>(skip) * pps : 0) <= nnz;
    }
    // Whether some row may see a token of the page that starts at token t.
    __device__ __forceinline__ bool page_seen(int t, int ps) const {
        return t < sinks || t + ps > lo;
    }
    // Rows [r0, r1) of a stage that starts at `b` are tokens that no row sees.
    __device__ __forceinline__ int hidden0(int b) const { return max(sinks - b, 0); }
    __device__ __forceinline__ int hidden1(int b) const { return min(lo - b, kStage); }
    __device__ __forceinline__ bool hides(int s) const {
        const int b = base(s);
        return hidden1(b) > hidden0(b);
    }
    // Whether every row up to position p_last sees the start of the stage at `b` (its
    // end is the causal mask's).
    __device__ __forceinline__ bool whole(int b, int p_last) const {
        return b > p_last - window || b + kStage <= sinks;
    }
};

// The page that lane 2j + c copies in a stage: page j of it. A page that no row sees
// is not looked up, and copied from behind the pool: zeros.
template <int kStage>
__device__ __forceinline__ int window_page(const TileWindow<kStage>& w, const PrefillParams& p,
                                           const PrefillUnit& u, int s, int n_st, int lane) {
    const int ps = p.page_size, pps = kStage / ps, j = lane >> 1;
    if (s >= n_st || s * pps + j >= u.n_pages || j >= pps) return 0;
    if (!w.page_seen(w.base(s) + j * ps, ps)) return static_cast<int>(p.num_pages);
    const int page = __ldg(p.indices + u.idx_begin + static_cast<int64_t>(w.stage(s)) * pps + j);
    return page < 0 || static_cast<int64_t>(page) >= p.num_pages ? -1 : page;
}

}  // namespace
}  // namespace oxd
