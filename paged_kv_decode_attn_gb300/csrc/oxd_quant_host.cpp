// C entries of the multi-axis append, the 4-bit append and the page copies:
// operand checks and one launch each.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstring>
#include <initializer_list>

#include "../../include/oxd.h"
#include "oxd_host_util.h"
#include "oxd_internal.h"

using namespace oxd;

namespace {

bool page_size_ok(int ps) { return ps == 8 || ps == 16 || ps == 32 || ps == 64; }
bool layout_ok(int l) { return l == OXD_LAYOUT_NHD || l == OXD_LAYOUT_HND; }

typedef CUresult (*PointerAttributeFn)(void*, CUpointer_attribute, CUdeviceptr);

PointerAttributeFn pointer_attribute() {
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
bool on_current_device(std::initializer_list<const void*> arrays) {
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

Pools pool_spans(const oxd_kv_pools& p, bool e2m1, int64_t pages, int ps, int H) {
    const size_t rows = static_cast<size_t>(pages) * ps * H;
    if (!e2m1) return {{span(p.k, rows * kHeadDim * 2), span(p.v, rows * kHeadDim * 2)}, 2};
    return {{span(p.k, rows * kCodeBytes), span(p.v, rows * kCodeBytes),
             span(p.k_scales, rows * kScaleBytes), span(p.v_scales, rows * kScaleBytes)},
            4};
}

bool pools_aligned(const oxd_kv_pools& p) {
    return aligned(p.k, 16) && aligned(p.v, 16) && aligned(p.k_scales, 16) &&
           aligned(p.v_scales, 16);
}

// A number as the sum of two doubles, good to about 2^-104.
struct Double2 {
    double hi, lo;
};
Double2 operator*(Double2 a, Double2 b) {
    const double p = a.hi * b.hi;
    const double e = std::fma(a.hi, b.hi, -p) + std::fma(a.hi, b.lo, a.lo * b.hi);
    const double hi = p + e;
    return {hi, e - (hi - p)};
}

// The frequencies theta^(-2i/128) / (2 pi), in turns a position, each as the sum
// of three floats: a far position (below 2^24) times a double's rounding, 2^-53,
// would be 2^-29 of a turn's angle, past what the kernel's rotation is good to.
// r = theta^(-1/64) comes from pow by one Newton step on r^64 theta = 1.
void frequencies(double theta, float4* turns) {
    const double r0 = std::pow(theta, -1.0 / 64);
    Double2 w = {r0, 0.0};
    for (int i = 0; i < 6; ++i) w = w * w;
    w = w * Double2{theta, 0.0};
    const Double2 r = {r0, r0 * (((1.0 - w.hi) - w.lo) / 64)};
    Double2 g = {0.15915494309189535, -9.839338337591243e-18};  // 1 / (2 pi)
    for (int i = 0; i < kHeadDim / 2; ++i, g = g * r) {
        turns[i].x = static_cast<float>(g.hi);
        const double rest = g.hi - turns[i].x;
        turns[i].y = static_cast<float>(rest);
        turns[i].z = static_cast<float>((rest - turns[i].y) + g.lo);
    }
}

oxd_status axes_append(const oxd_axes_append_desc* desc, const void* q, const void* k,
                       const void* v, const int32_t* token_request, const int32_t* positions,
                       const int32_t* rope_positions, const int32_t* indptr,
                       const int32_t* indices, const int32_t* page_refcount, void* q_out,
                       const oxd_kv_pools& pools, bool e2m1, void* workspace,
                       size_t workspace_bytes, void* stream) {
    if (desc == nullptr || q == nullptr || k == nullptr || v == nullptr ||
        token_request == nullptr || positions == nullptr || indptr == nullptr ||
        indices == nullptr || page_refcount == nullptr || q_out == nullptr ||
        pools.k == nullptr || pools.v == nullptr ||
        (e2m1 && (pools.k_scales == nullptr || pools.v_scales == nullptr)) || workspace == nullptr)
        return OXD_ERR_INVALID_ARGUMENT;
    const oxd_axes_append_desc& d = *desc;
    if (d.num_tokens < 1 || d.batch < 1 || d.num_qo_heads < 1 || d.num_kv_heads < 1 ||
        d.num_pages < 1 || d.num_indices < 1 || d.reserved != 0 || !layout_ok(d.layout) ||
        d.num_axes < 1 || d.num_axes > 4 || !(std::isfinite(d.rope_theta) && d.rope_theta > 1.0))
        return OXD_ERR_INVALID_ARGUMENT;
    for (int i = 0; i < kHeadDim / 2; ++i)
        if (d.pair_axis[i] >= d.num_axes) return OXD_ERR_INVALID_ARGUMENT;
    if (d.head_dim != kHeadDim || !page_size_ok(d.page_size)) return OXD_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(d.num_tokens) *
            (static_cast<int64_t>(d.num_qo_heads) + d.num_kv_heads) > (int64_t{1} << 33) ||
        d.num_pages >= (int64_t{1} << 31) || d.num_qo_heads > (1 << 20) ||
        d.num_kv_heads > (1 << 20))
        return OXD_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) ||
        !pools_aligned(pools) || !aligned(token_request, 4) || !aligned(positions, 4) ||
        !aligned(rope_positions, 4) || !aligned(indptr, 4) || !aligned(indices, 4) ||
        !aligned(page_refcount, 4) || !aligned(workspace, 256))
        return OXD_ERR_ALIGNMENT;
    if (workspace_bytes < sizeof(WsHeader)) return OXD_ERR_WORKSPACE_TOO_SMALL;

    const size_t T = static_cast<size_t>(d.num_tokens);
    const size_t qbytes = T * d.num_qo_heads * kHeadDim * 2;
    const size_t kvbytes = T * d.num_kv_heads * kHeadDim * 2;
    const Span in[] = {span(k, kvbytes), span(v, kvbytes), span(token_request, T * 4),
                       span(positions, T * 4),
                       rope_positions ? span(rope_positions, T * 4 * d.num_axes) : Span{0, 0},
                       span(indptr, (static_cast<size_t>(d.batch) + 1) * 4),
                       span(indices, static_cast<size_t>(d.num_indices) * 4),
                       span(page_refcount, static_cast<size_t>(d.num_pages) * 4)};
    const Span qin = span(q, qbytes);
    const Pools ps = pool_spans(pools, e2m1, d.num_pages, d.page_size, d.num_kv_heads);
    Span outs[6] = {span(q_out, qbytes), span(workspace, sizeof(WsHeader))};
    const int n_outs = 2 + ps.n;
    for (int i = 0; i < ps.n; ++i) outs[2 + i] = ps.s[i];
    for (int i = 0; i < n_outs; ++i) {
        for (const Span& x : in)
            if (overlap(outs[i], x)) return OXD_ERR_ALIAS;
        // q_out may be q exactly (each row is read before it is written, by
        // the same warp)
        if (overlap(outs[i], qin) && !(i == 0 && q_out == q)) return OXD_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return OXD_ERR_ALIAS;
    }
    if (!on_current_device({q, k, v, token_request, positions, rope_positions, indptr, indices,
                            page_refcount, q_out, pools.k, pools.v, e2m1 ? pools.k_scales : nullptr,
                            e2m1 ? pools.v_scales : nullptr, workspace}))
        return OXD_ERR_INVALID_ARGUMENT;

    AxesAppendParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.token_request = token_request;
    p.positions = positions;
    p.rope_positions = rope_positions != nullptr ? rope_positions : positions;
    p.indptr = indptr;
    p.indices = indices;
    p.refcount = page_refcount;
    p.q_out = static_cast<uint16_t*>(q_out);
    p.k_pages = pools.k;
    p.v_pages = pools.v;
    p.k_scales = e2m1 ? static_cast<uint16_t*>(pools.k_scales) : nullptr;
    p.v_scales = e2m1 ? static_cast<uint16_t*>(pools.v_scales) : nullptr;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.status = reinterpret_cast<unsigned long long*>(ws + offsetof(WsHeader, status));
    p.last_epoch = reinterpret_cast<uint32_t*>(ws + offsetof(WsHeader, last_epoch));
    p.epoch = next_run_epoch();
    p.T = d.num_tokens;
    p.B = d.batch;
    p.Hq = d.num_qo_heads;
    p.Hkv = d.num_kv_heads;
    p.page_size = d.page_size;
    p.layout = d.layout;
    p.num_indices = d.num_indices;
    p.num_pages = d.num_pages;
    frequencies(d.rope_theta, p.turns);
    for (int i = 0; i < kHeadDim / 2; ++i) {
        const int32_t axis = rope_positions != nullptr ? d.pair_axis[i] : 0;
        std::memcpy(&p.turns[i].w, &axis, sizeof(axis));
    }
    if (launch_axes_append(p, static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return OXD_ERR_CUDA;
    return OXD_OK;
}

}  // namespace

extern "C" oxd_status oxd_rope_axes_append(
    const oxd_axes_append_desc* desc, const void* q, const void* k, const void* v,
    const int32_t* token_request, const int32_t* positions, const int32_t* rope_positions,
    const int32_t* indptr, const int32_t* indices, const int32_t* page_refcount, void* q_out,
    void* k_pages, void* v_pages, void* workspace, size_t workspace_bytes, void* stream) {
    const oxd_kv_pools pools = {k_pages, v_pages, nullptr, nullptr};
    return axes_append(desc, q, k, v, token_request, positions, rope_positions, indptr, indices,
                       page_refcount, q_out, pools, false, workspace, workspace_bytes, stream);
}

extern "C" oxd_status oxd_quant_rope_append(
    const oxd_axes_append_desc* desc, const void* q, const void* k, const void* v,
    const int32_t* token_request, const int32_t* positions, const int32_t* rope_positions,
    const int32_t* indptr, const int32_t* indices, const int32_t* page_refcount, void* q_out,
    const oxd_kv_pools* cache, void* workspace, size_t workspace_bytes, void* stream) {
    if (cache == nullptr) return OXD_ERR_INVALID_ARGUMENT;
    return axes_append(desc, q, k, v, token_request, positions, rope_positions, indptr, indices,
                       page_refcount, q_out, *cache, true, workspace, workspace_bytes, stream);
}

extern "C" oxd_status oxd_copy_pages(const oxd_copy_pages_desc* desc, const oxd_kv_pools* src,
                                     const oxd_kv_pools* dst, const int32_t* src_pages,
                                     const int32_t* dst_pages, const int32_t* dst_refcount,
                                     void* workspace, size_t workspace_bytes, void* stream) {
    if (desc == nullptr || src == nullptr || dst == nullptr || workspace == nullptr)
        return OXD_ERR_INVALID_ARGUMENT;
    const oxd_copy_pages_desc& d = *desc;
    auto format_ok = [](int f) { return f == OXD_FORMAT_BF16 || f == OXD_FORMAT_E2M1; };
    if (d.num_pairs < 0 || d.num_kv_heads < 1 || d.src_num_pages < 1 || d.dst_num_pages < 1 ||
        !format_ok(d.src_format) || !format_ok(d.dst_format) || !layout_ok(d.src_layout) ||
        !layout_ok(d.dst_layout) || d.reserved[0] != 0 || d.reserved[1] != 0)
        return OXD_ERR_INVALID_ARGUMENT;
    if (d.num_pairs > 0 && (src_pages == nullptr || dst_pages == nullptr))
        return OXD_ERR_INVALID_ARGUMENT;
    const bool s4 = d.src_format == OXD_FORMAT_E2M1, d4 = d.dst_format == OXD_FORMAT_E2M1;
    for (const oxd_kv_pools* c : {src, dst}) {
        const bool four = c == src ? s4 : d4;
        if (c->k == nullptr || c->v == nullptr || (c->k_scales != nullptr) != four ||
            (c->v_scales != nullptr) != four)
            return OXD_ERR_INVALID_ARGUMENT;
    }
    if (d.head_dim != kHeadDim || !page_size_ok(d.page_size)) return OXD_ERR_UNSUPPORTED;
    // (a page's 16-byte pieces are counted in 32 bits, and so are the pairs, in
    // steps of up to kMaxPairRows)
    if (d.src_num_pages >= (int64_t{1} << 31) || d.dst_num_pages >= (int64_t{1} << 31) ||
        d.num_kv_heads > (1 << 20) || d.num_pairs > INT32_MAX - kMaxPairRows)
        return OXD_ERR_UNSUPPORTED;
    if (!pools_aligned(*src) || !pools_aligned(*dst) || !aligned(src_pages, 4) ||
        !aligned(dst_pages, 4) || !aligned(dst_refcount, 4) || !aligned(workspace, 256))
        return OXD_ERR_ALIGNMENT;
    if (workspace_bytes < sizeof(WsHeader)) return OXD_ERR_WORKSPACE_TOO_SMALL;

    const size_t n = static_cast<size_t>(d.num_pairs);
    const Pools from = pool_spans(*src, s4, d.src_num_pages, d.page_size, d.num_kv_heads);
    const Pools to = pool_spans(*dst, d4, d.dst_num_pages, d.page_size, d.num_kv_heads);
    const Span in[] = {span(src_pages, n * 4), span(dst_pages, n * 4),
                       dst_refcount ? span(dst_refcount, static_cast<size_t>(d.dst_num_pages) * 4)
                                    : Span{0, 0}};
    const Span ws_span = span(workspace, sizeof(WsHeader));
    const bool same = src->k == dst->k && src->v == dst->v && src->k_scales == dst->k_scales &&
                      src->v_scales == dst->v_scales && s4 == d4 &&
                      d.src_layout == d.dst_layout && d.src_num_pages == d.dst_num_pages;
    for (const Span& x : in)
        if (overlap(ws_span, x)) return OXD_ERR_ALIAS;
    for (int i = 0; i < from.n; ++i)
        if (overlap(ws_span, from.s[i])) return OXD_ERR_ALIAS;
    for (int i = 0; i < to.n; ++i) {
        if (overlap(ws_span, to.s[i])) return OXD_ERR_ALIAS;
        for (const Span& x : in)
            if (overlap(to.s[i], x)) return OXD_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(to.s[i], to.s[j])) return OXD_ERR_ALIAS;
        for (int j = 0; j < from.n && !same; ++j)
            if (overlap(to.s[i], from.s[j])) return OXD_ERR_ALIAS;
    }
    if (!on_current_device({src->k, src->v, src->k_scales, src->v_scales, dst->k, dst->v,
                            dst->k_scales, dst->v_scales, src_pages, dst_pages, dst_refcount,
                            workspace}))
        return OXD_ERR_INVALID_ARGUMENT;

    CopyPagesParams p{};
    auto pools = [](const oxd_kv_pools& c, int64_t pages, int layout) {
        return PagePools{{static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.v)},
                         {static_cast<uint16_t*>(c.k_scales), static_cast<uint16_t*>(c.v_scales)},
                         pages,
                         layout};
    };
    p.src = pools(*src, d.src_num_pages, d.src_layout);
    p.dst = pools(*dst, d.dst_num_pages, d.dst_layout);
    p.src_pages = src_pages;
    p.dst_pages = dst_pages;
    p.refcount = dst_refcount;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.status = reinterpret_cast<unsigned long long*>(ws + offsetof(WsHeader, status));
    p.last_epoch = reinterpret_cast<uint32_t*>(ws + offsetof(WsHeader, last_epoch));
    p.epoch = next_run_epoch();
    p.n = d.num_pairs;
    p.H = d.num_kv_heads;
    p.page_size = d.page_size;
    // n / inner = the high word of n * magic for n < page_size * H, where that
    // many times inner stays below 2^32
    const uint64_t inner = d.dst_layout == OXD_LAYOUT_NHD ? d.num_kv_heads : d.page_size;
    if (inner > 1 && static_cast<uint64_t>(d.num_kv_heads) * d.page_size * inner < (uint64_t{1} << 32))
        p.inner_magic = static_cast<uint32_t>((uint64_t{1} << 32) / inner + 1);
    if (launch_copy_pages(p, static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return OXD_ERR_CUDA;
    return OXD_OK;
}
