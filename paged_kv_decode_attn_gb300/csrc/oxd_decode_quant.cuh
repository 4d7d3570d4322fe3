// What the two decode kernels over a 4-bit paged cache share
// (oxd_decode_quant.cu, oxd_decode_quant_wide.cu): PTX wrappers, work units and
// the query fragments.
#pragma once

#include "oxd_e2m1.cuh"
#include "oxd_internal.h"
#include "oxd_ptx.cuh"

namespace oxd {
namespace {

constexpr float kLazy = 4.f;     // log2: how far a score may pass the running maximum
constexpr float kPOffset = 10.f; // log2 of the weight a score at the running maximum gets

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t (&v)[4]) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3])
                 : "memory");
}

__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(static_cast<uint16_t>(a)) : "memory");
}

// D = A * B + D, m16n8k16, f16 inputs, f32 accumulate.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A * B.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    __half2 v = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<uint32_t*>(&v);
}

// A work unit, checked against the plan: no tokens if it is not one of it.
struct Unit {
    int first;     // offset of its first page in `indices`
    int n_pages;
    int valid;     // tokens
    int b, h;      // request, (first) KV head
    int slot;      // -1: the unit is its whole stream
    int row0;      // its first row in the slot, which has stream_heads * G
    int reserved;
};
static_assert(sizeof(Unit) == 32, "two 16-byte loads");

// kAllHeads: whether a unit covers all heads of its stream (else one of them,
// the second where the half bit says so).
template <bool kAllHeads>
__device__ __forceinline__ Unit decode_unit(const QuantDecodeParams& qp, const int4 it) {
    const DecodeParams& p = qp.d;
    Unit u;
    u.first = it.x;
    u.n_pages = it.y & ((1 << kUnitPagesBits) - 1);
    const int last_len = (it.y >> kUnitPagesBits) & 0x7f;  // 0: not the request's last page
    u.b = it.z & ((1 << kUnitBBits) - 1);
    const int second = (it.z >> kUnitBBits) & 1;
    u.h = static_cast<int>(static_cast<uint32_t>(it.z) >> (kUnitBBits + 1)) * qp.heads + second;
    u.slot = it.w;
    u.row0 = second * p.group;
    u.reserved = 0;
    const bool ok = u.n_pages >= 1 && it.x >= 0 &&
                    static_cast<int64_t>(it.x) + u.n_pages <= p.nnz && u.b < p.batch &&
                    second < (kAllHeads ? 1 : qp.heads) &&
                    u.h + (kAllHeads ? qp.heads : 1) <= p.num_kv_heads && it.w >= -1 &&
                    it.w < p.n_slots && last_len <= p.page_size;
    u.valid = !ok        ? 0
              : last_len ? (u.n_pages - 1) * p.page_size + last_len
                         : u.n_pages * p.page_size;
    return u;
}

// Whether the device's block tables say what the unit's plan was made from.
__device__ __forceinline__ bool tables_match(const DecodeParams& p, const Unit& u, const int4 it) {
    const int last_len = (it.y >> kUnitPagesBits) & 0x7f;
    return u.valid > 0 && (it.y >= 0 || p.indptr[u.b] == u.first) &&
           (last_len == 0 || (p.indptr[u.b + 1] == u.first + u.n_pages &&
                              p.last_page_len[u.b] == last_len));
}

// A CTA's units: the first kListed decoded in shared memory, others from the list.
constexpr int kListed = 32;
template <bool kAllHeads>
struct UnitList {
    const Unit* shared;
    const int4* list;
    int first;
    __device__ __forceinline__ Unit get(const QuantDecodeParams& qp, int i) const {
        if (i - first < kListed) return shared[i - first];
        return decode_unit<kAllHeads>(qp, __ldg(list + i));
    }
};

// (a, b) = (x, y) * (s, s) + (a, b)
__device__ __forceinline__ void fma_pair(float& a, float& b, float x, float y, float s) {
    asm("{\n\t.reg .b64 u, v, w;\n\t"
        "mov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %4};\n\tmov.b64 w, {%0, %1};\n\t"
        "fma.rn.f32x2 w, u, v, w;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(x), "f"(y), "f"(s));
}

// (x, y) * (s, t) + (c, d)
__device__ __forceinline__ void fma_pairs(float& a, float& b, float x, float y, float s, float t,
                                          float c, float d) {
    asm("{\n\t.reg .b64 u, v, w;\n\t"
        "mov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\tmov.b64 w, {%6, %7};\n\t"
        "fma.rn.f32x2 w, u, v, w;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(a), "=f"(b)
        : "f"(x), "f"(y), "f"(s), "f"(t), "f"(c), "f"(d));
}

// Makes f16 fragments of query rows that lie at `raw`, [rows][128] bf16:
// eight rows a pass, 16 threads of 128 a row, a thread 8 columns (one lane's
// fragment of a group). A row is scaled by a power of two so that its largest
// size lies in [1, 2) (f16's range); a negative logit scale's sign goes into q,
// and a scale of zero becomes the smallest normal number (logits below 2^-100),
// so a masked score of -inf stays one. Fragments [group c][tile][lane] of 16
// bytes at `out`, logit scales (log2) at `sc`; rows past the last are zeros.
template <int kTiles>
__device__ __forceinline__ void convert_query(const uint8_t* raw, int rows, float scale_log2,
                                              uint8_t* out, float* sc) {
    const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
    for (int n = 0; n < kTiles; ++n) {
        const int r = n * 8 + row;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r < rows) x = *reinterpret_cast<const uint4*>(raw + r * (kHeadDim * 2) + col * 16);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) top = __vmaxu2(top, w[j] & 0x7fff7fffu);
        top = max(top & 0xffffu, top >> 16);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        // exponent field of the largest size, kept where 2^+-exponent is a
        // normal float
        const uint32_t e = min(max(top >> 7, 1u), 253u);
        const float f = copysignf(__uint_as_float((254u - e) << 23), scale_log2);
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            h[j] = pack_f16x2(__uint_as_float(w[j] << 16) * f,
                              __uint_as_float(w[j] & 0xffff0000u) * f);
        *reinterpret_cast<uint4*>(out + ((col >> 2) * kTiles + n) * 512 +
                                  (row * 4 + (col & 3)) * 16) = make_uint4(h[0], h[1], h[2], h[3]);
        if (col == 0)
            sc[r] = fmaxf(fabsf(scale_log2) * __uint_as_float(e << 23), 1.17549435e-38f);
    }
}

}  // namespace
}  // namespace oxd
