// C entries of the window decodes and of the table builder: operand checks and one
// launch each. (The prefill with a window is planned in oxd_prefill_host.cpp.)
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstddef>

#include "../../include/oxd.h"
#include "oxd_cache_host.h"
#include "oxd_host_util.h"
#include "oxd_internal.h"

using namespace oxd;

namespace {

int log2_of(int page_size) { return page_size == 8 ? 3 : page_size == 16 ? 4 : page_size == 32 ? 5 : 6; }

oxd_status window_decode(const oxd_window_decode_desc* desc, const void* q,
                         const oxd_kv_pools& pools, bool e2m1, const int32_t* indptr,
                         const int32_t* indices, const int32_t* last_page_len, float sm_scale,
                         void* out, float* lse, void* workspace, size_t workspace_bytes,
                         void* stream) {
    if (desc == nullptr || q == nullptr || pools.k == nullptr || pools.v == nullptr ||
        (e2m1 && (pools.k_scales == nullptr || pools.v_scales == nullptr)) || indptr == nullptr ||
        indices == nullptr || last_page_len == nullptr || out == nullptr || workspace == nullptr)
        return OXD_ERR_INVALID_ARGUMENT;
    const oxd_window_decode_desc& d = *desc;
    if (d.batch < 1 || d.num_qo_heads < 1 || d.num_kv_heads < 1 || d.num_pages < 1 ||
        d.num_indices < 1 || d.window < 1 || d.sinks < 0 || d.max_splits < 0 ||
        d.num_qo_heads % d.num_kv_heads != 0 || !layout_ok(d.layout) || !std::isfinite(sm_scale) ||
        d.reserved[0] != 0 || d.reserved[1] != 0)
        return OXD_ERR_INVALID_ARGUMENT;
    const int G = d.num_qo_heads / d.num_kv_heads;
    if (d.head_dim != kHeadDim || !page_size_ok(d.page_size) || G > kMaxGroup)
        return OXD_ERR_UNSUPPORTED;
    const int64_t streams = static_cast<int64_t>(d.batch) * d.num_kv_heads;
    if (static_cast<int64_t>(d.window) + d.sinks > kMaxWindowTokens ||
        d.num_pages >= (int64_t{1} << 31) ||
        d.num_pages > (int64_t{1} << 32) / d.page_size / d.num_kv_heads ||
        streams * kMaxWindowSplits * 4 > INT32_MAX)
        return OXD_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(out, 16) || !pools_aligned(pools) || !aligned(indptr, 4) ||
        !aligned(indices, 4) || !aligned(last_page_len, 4) || !aligned(lse, 4) ||
        !aligned(workspace, 256))
        return OXD_ERR_ALIGNMENT;
    if (workspace_bytes < sizeof(WsHeader)) return OXD_ERR_WORKSPACE_TOO_SMALL;

    const size_t rows = static_cast<size_t>(d.batch) * d.num_qo_heads;
    const Pools ps = pool_spans(pools, e2m1, d.num_pages, d.page_size, d.num_kv_heads);
    const Span in[] = {span(q, rows * kHeadDim * 2),
                       span(indptr, (static_cast<size_t>(d.batch) + 1) * 4),
                       span(indices, static_cast<size_t>(d.num_indices) * 4),
                       span(last_page_len, static_cast<size_t>(d.batch) * 4)};
    const Span outs[] = {span(out, rows * kHeadDim * 2), lse ? span(lse, rows * 4) : Span{0, 0},
                         span(workspace, sizeof(WsHeader))};
    for (int i = 0; i < 3; ++i) {
        for (const Span& x : in)
            if (overlap(outs[i], x)) return OXD_ERR_ALIAS;
        for (int j = 0; j < ps.n; ++j)
            if (overlap(outs[i], ps.s[j])) return OXD_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return OXD_ERR_ALIAS;
    }
    if (!on_current_device({q, pools.k, pools.v, e2m1 ? pools.k_scales : nullptr,
                            e2m1 ? pools.v_scales : nullptr, indptr, indices, last_page_len, out,
                            lse, workspace}))
        return OXD_ERR_INVALID_ARGUMENT;

    WindowParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint8_t*>(pools.k);
    p.v = static_cast<const uint8_t*>(pools.v);
    p.k_scales = e2m1 ? static_cast<const uint16_t*>(pools.k_scales) : nullptr;
    p.v_scales = e2m1 ? static_cast<const uint16_t*>(pools.v_scales) : nullptr;
    p.indptr = indptr;
    p.indices = indices;
    p.last_page_len = last_page_len;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.status = reinterpret_cast<unsigned long long*>(ws + offsetof(WsHeader, status));
    p.last_epoch = reinterpret_cast<uint32_t*>(ws + offsetof(WsHeader, last_epoch));
    p.epoch = next_run_epoch();
    p.batch = d.batch;
    p.num_qo_heads = d.num_qo_heads;
    p.num_kv_heads = d.num_kv_heads;
    p.group = G;
    p.page_shift = log2_of(d.page_size);
    p.layout = d.layout;
    p.num_indices = d.num_indices;
    p.window = d.window;
    p.sinks = d.sinks;
    p.num_pages = d.num_pages;
    p.scale_log2 = sm_scale * 1.4426950408889634f;  // log2(e)
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = e2m1 ? launch_window_quant(p, d.max_splits, s, d.pdl != 0)
                               : launch_window_decode(p, d.max_splits, s, d.pdl != 0);
    return e == cudaSuccess ? OXD_OK : OXD_ERR_CUDA;
}

}  // namespace

extern "C" oxd_status oxd_window_decode(const oxd_window_decode_desc* desc, const void* q,
                                        const void* k_pages, const void* v_pages,
                                        const int32_t* indptr, const int32_t* indices,
                                        const int32_t* last_page_len, float sm_scale, void* out,
                                        float* lse, void* workspace, size_t workspace_bytes,
                                        void* stream) {
    const oxd_kv_pools pools = {const_cast<void*>(k_pages), const_cast<void*>(v_pages), nullptr,
                                nullptr};
    return window_decode(desc, q, pools, false, indptr, indices, last_page_len, sm_scale, out, lse,
                         workspace, workspace_bytes, stream);
}

extern "C" oxd_status oxd_quant_window_decode(const oxd_window_decode_desc* desc, const void* q,
                                              const oxd_kv_pools* cache, const int32_t* indptr,
                                              const int32_t* indices, const int32_t* last_page_len,
                                              float sm_scale, void* out, float* lse,
                                              void* workspace, size_t workspace_bytes,
                                              void* stream) {
    if (cache == nullptr) return OXD_ERR_INVALID_ARGUMENT;
    return window_decode(desc, q, *cache, true, indptr, indices, last_page_len, sm_scale, out, lse,
                         workspace, workspace_bytes, stream);
}

extern "C" oxd_status oxd_build_tables(const oxd_build_tables_desc* desc, const int32_t* lengths,
                                       const int32_t* new_tokens, int32_t* page_rows,
                                       const int32_t* held, int32_t* held_out,
                                       const int32_t* free_pages, const int32_t* taken,
                                       int32_t* taken_out, int32_t* page_refcount, int32_t* indptr,
                                       int32_t* indices, int32_t* last_page_len,
                                       int32_t* qo_indptr, int32_t* token_request,
                                       int32_t* positions, int64_t* slots, void* workspace,
                                       size_t workspace_bytes, void* stream) {
    if (desc == nullptr || lengths == nullptr || page_rows == nullptr || held == nullptr ||
        held_out == nullptr || indptr == nullptr || indices == nullptr ||
        last_page_len == nullptr || workspace == nullptr)
        return OXD_ERR_INVALID_ARGUMENT;
    const oxd_build_tables_desc& d = *desc;
    if (d.batch < 1 || d.row_pages < 1 || d.num_indices < 1 || d.num_tokens < 0 ||
        d.num_free < 0 || d.num_pages < 1 || d.window < 0 || d.sinks < 0 || d.reserved != 0)
        return OXD_ERR_INVALID_ARGUMENT;
    // the free list comes whole, the token maps come with their starts
    if (d.num_free > 0 && (free_pages == nullptr || taken == nullptr || taken_out == nullptr))
        return OXD_ERR_INVALID_ARGUMENT;
    if (d.num_tokens > 0 && (new_tokens == nullptr || qo_indptr == nullptr ||
                             token_request == nullptr || positions == nullptr))
        return OXD_ERR_INVALID_ARGUMENT;
    if (!page_size_ok(d.page_size)) return OXD_ERR_UNSUPPORTED;
    constexpr int64_t kMost = 1 << 30;
    const int64_t row_tokens = static_cast<int64_t>(d.row_pages) * d.page_size;
    if (d.num_pages >= (int64_t{1} << 31) || row_tokens > kMost || d.batch > kMost / row_tokens ||
        d.num_free > kMost || d.num_indices > kMost || d.num_tokens > kMost || d.window > kMost ||
        d.sinks > kMost)
        return OXD_ERR_UNSUPPORTED;
    const bool maps = d.num_tokens > 0, free = d.num_free > 0;
    if (!aligned(lengths, 4) || !aligned(new_tokens, 4) || !aligned(page_rows, 4) ||
        !aligned(held, 4) || !aligned(held_out, 4) || !aligned(free_pages, 4) ||
        !aligned(taken, 4) || !aligned(taken_out, 4) || !aligned(page_refcount, 4) ||
        !aligned(indptr, 4) || !aligned(indices, 4) || !aligned(last_page_len, 4) ||
        !aligned(qo_indptr, 4) || !aligned(token_request, 4) || !aligned(positions, 4) ||
        !aligned(slots, 8) || !aligned(workspace, 256))
        return OXD_ERR_ALIGNMENT;
    if (workspace_bytes < sizeof(WsHeader)) return OXD_ERR_WORKSPACE_TOO_SMALL;

    const size_t B4 = static_cast<size_t>(d.batch) * 4, T = static_cast<size_t>(d.num_tokens);
    const Span none = {0, 0};
    auto opt = [&](const void* p, size_t bytes) { return p != nullptr ? span(p, bytes) : none; };
    const Span in[] = {span(lengths, B4), opt(new_tokens, B4),
                       free ? span(free_pages, static_cast<size_t>(d.num_free) * 4) : none,
                       span(held, B4), free ? span(taken, 4) : none};
    const Span outs[] = {span(page_rows, static_cast<size_t>(d.row_pages) * B4),
                         span(held_out, B4),
                         free ? span(taken_out, 4) : none,
                         opt(page_refcount, static_cast<size_t>(d.num_pages) * 4),
                         span(indptr, B4 + 4),
                         span(indices, static_cast<size_t>(d.num_indices) * 4),
                         span(last_page_len, B4),
                         maps ? span(qo_indptr, B4 + 4) : none,
                         maps ? span(token_request, T * 4) : none,
                         maps ? span(positions, T * 4) : none,
                         maps ? opt(slots, T * 8) : none,
                         span(workspace, sizeof(WsHeader))};
    constexpr int kIn = sizeof(in) / sizeof(in[0]), kOut = sizeof(outs) / sizeof(outs[0]);
    for (int i = 0; i < kOut; ++i) {
        for (int j = 0; j < kIn; ++j)
            // held and taken may be updated in place
            if (overlap(outs[i], in[j]) && !(i == 1 && j == 3 && held_out == held) &&
                !(i == 2 && j == 4 && taken_out == taken))
                return OXD_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return OXD_ERR_ALIAS;
    }
    if (!on_current_device({lengths, new_tokens, page_rows, held, held_out, free_pages, taken,
                            taken_out, page_refcount, indptr, indices, last_page_len, qo_indptr,
                            token_request, positions, slots, workspace}))
        return OXD_ERR_INVALID_ARGUMENT;

    TablesParams p{};
    p.lengths = lengths;
    p.new_tokens = new_tokens;
    p.rows = page_rows;
    p.held = held;
    p.held_out = held_out;
    p.free_pages = free_pages;
    p.taken = taken;
    p.taken_out = taken_out;
    p.refcount = page_refcount;
    p.indptr = indptr;
    p.indices = indices;
    p.last_page_len = last_page_len;
    p.qo_indptr = maps ? qo_indptr : nullptr;
    p.token_request = maps ? token_request : nullptr;
    p.positions = maps ? positions : nullptr;
    p.slots = maps ? slots : nullptr;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.status = reinterpret_cast<unsigned long long*>(ws + offsetof(WsHeader, status));
    p.last_epoch = reinterpret_cast<uint32_t*>(ws + offsetof(WsHeader, last_epoch));
    p.epoch = next_run_epoch();
    p.batch = d.batch;
    p.page_shift = log2_of(d.page_size);
    p.row_pages = d.row_pages;
    p.num_indices = d.num_indices;
    p.num_tokens = d.num_tokens;
    p.num_free = d.num_free;
    p.window = d.window;
    p.sinks = d.sinks;
    p.num_pages = d.num_pages;
    return launch_build_tables(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? OXD_OK
                                                                                    : OXD_ERR_CUDA;
}
