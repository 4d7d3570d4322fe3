// Paged causal prefill with a sliding window for sm_103a, tiles of 256 rows
// (oxd_window_prefill_plan; oxd_prefill_narrow.cu takes the short ones).
//
// A query at position p of its request sees the tokens j <= p with j > p - window or
// j < sinks. Tiles, halves and stages are those of the prefill without a window
// (oxd_prefill.cu): up to 256 rows (query token, head of one KV head) in two halves of
// 128 MMA rows, S_h = Q_h K^T and O_h += P_h V on tcgen05 with S, P and O in tensor
// memory, K and V by TMA in stages of 128 tokens that serve both halves. What differs:
//   * a tile streams the pages with the sinks and the pages from its first query's
//     window on, as one sequence of tokens (a stage takes any eight pages of 16 tokens,
//     so the few sinks cost a page, not a stage: 8 prompts of 2048, window 1024, 408 us
//     with stages skipped, 300 so and persistent);
//   * with a window a tile is short (1024 tokens: nine stages), so that what a tile
//     costs besides its stages counts: the kernel is persistent, one CTA a SM walking
//     its list of pieces. K and V run ahead into the next piece, the next piece's query
//     rows are copied while the last stage's softmax runs, its first score
//     MMAs follow the last PV, and a half's epilogue overlaps the other half's products;
//   * every stage takes one pass over its scores against the row's reference (the
//     first: the maximum of the last 16 columns seen, each row its own; a lagging
//     reference is as good, see below),
//     16 columns at a time, at the window's edges masked by a bit a column; a warp's
//     rows are few tokens, so most blocks of 16 columns there are seen by none of them
//     and cost nothing. A pass whose sum shows a term above 2^64 is done again in two
//     (maximum, then weights).
// Rows of V that no query of the call sees (between the sinks and the window, behind the
// last token) are zeroed before the product, by the V warp as they land. Every wait is
// bounded (OXD_DEVICE_WAIT_TIMEOUT); on abort the MMAs and copies in flight are drained.
//
// 8 prompts of 2048 (GQA4 x 8 heads) at window 1024 take 248 to 254 us, 1060 TFLOP/s, at
// 4096 725 us, 1330. What the first loses against the rate of a matrix product, of a tile's 18.1
// us: 3.5 for its ends; a stage's chain, softmax (0.73 us), PV and the next scores (0.85),
// 1.6 us where its products alone are 1.3; and 11 % of the tokens in its stages, which
// a row does not see (tensor pipe 48 %, issue slots 35 %).
#include <cuda_bf16.h>

#include <atomic>

#include "oxd_internal.h"
#include "oxd_prefill.h"
#include "oxd_prefill_window.cuh"
#include "oxd_ptx.cuh"
#include "oxd_tcgen05.cuh"

namespace oxd {
namespace {

constexpr int kStages = 2;  // of the K ring and of the V ring
constexpr int kMmaWarp = 8;
constexpr int kKWarp = 9;
constexpr int kVWarp = 10;
constexpr int kThreads = 11 * 32;
constexpr int kTokens = kPrefillStageTokens;
constexpr int kHalfBytes = kTokens * 128;        // one 64-column half of K or V: 16 KB
constexpr int kSlotBytes = 2 * kHalfBytes;       // K or V of one stage
constexpr int kQHalf = 128 * 128;                // 64 columns of a half's 128 query rows
constexpr int kKOff = 4 * kQHalf;                // (Q of half h at 2 h kQHalf)
constexpr int kVOff = kKOff + kStages * kSlotBytes;
constexpr int kCtlOff = kVOff + kStages * kSlotBytes;  // 192 KB of operands
// Tensor memory, 512 columns: O_h at [128 h, +128), S_h (then P_h, bf16 pairs in the
// first 64 columns) at [256 + 128 h, +128).
constexpr uint32_t kTmemCols = 512;
static_assert(kTokens == 128, "score MMAs of N = 128, PV of K = 128");
static_assert(kPrefillRows == 2 * 128, "a tile is two 128-row halves");

// A unit as the warps need it; tokens counted from the piece's first (TileWindow).
struct Piece {
    int n_st;          // stages; 0: not a unit of this plan, skipped
    int nst[2];        // stages that each half streams
    int pages;         // pages of the piece
    int first;         // index of its first page in `indices`
    int front, skip;   // pages from `front` on lie `skip` entries further
    int p0, sinks;     // position of the first query, the sinks
    int hide0, hide1;  // tokens that no query of the call sees, [hide0, hide1) and those
    int end;           // from `end` on, behind the request's last
    int q_begin, n_tok, hkv;
    int state, n_pieces, piece;
    int pad[2];
};
static_assert(sizeof(Piece) == 80, "five 16-byte loads");

struct Ctl {
    uint64_t kfull[kStages], kempty[kStages], vfull[kStages], vempty[kStages];
    uint64_t q_ready[2];  // a half's query rows are in shared memory (G divides 128: their
                          // copies' bytes; else one arrival a warp)
    uint64_t s_ready[2];  // the n-th scores of the half: phase n
    uint64_t p_ready[2];  // their P written (one arrival a warp)
    uint64_t o_done[2];   // the half's last PV of a piece
    uint64_t vland;       // V of the k-th stage with rows to zero has landed: phase k (its vfull
                          // comes when they are zeroed)
    uint64_t mma_done;
    int kissued[kStages], vissued[kStages], qissued[2], landing, zeroed;
    uint32_t tmem;
    int flags[3];  // [0] abort, [1] pieces of this CTA, [2] its first unit
};
constexpr int kListOff = kCtlOff + (static_cast<int>(sizeof(Ctl)) + 15) / 16 * 16;
// a softmax warp's outputs on their way out: 32 rows of 128 bytes
constexpr int kOutOff = kListOff + kWindowUnits * static_cast<int>(sizeof(Piece));
constexpr int kOutBytes = 32 * 128;
constexpr int kSmemBytes = kOutOff + 8 * kOutBytes;
static_assert(kSmemBytes <= 227 * 1024, "one CTA a SM");

// The stages with rows of V that no query sees (zeroed before the product): [first, last]
// and those from `end` on.
struct HiddenStages {
    int first, last, end;
    __device__ __forceinline__ explicit HiddenStages(const Piece& c) {
        const bool any = c.hide1 > max(c.hide0, 0);
        first = any ? max(c.hide0, 0) / kTokens : 1;
        last = any ? (c.hide1 - 1) / kTokens : 0;
        end = max(c.end, 0) / kTokens;
    }
    __device__ __forceinline__ bool among(int g) const {
        return (g >= first && g <= last) || g >= end;
    }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The lowest n bits (all of 64, none for a negative n).
__device__ __forceinline__ unsigned long long below(int n) {
    return n >= 64 ? ~0ull : (1ull << max(n, 0)) - 1ull;
}

// Unit `u` as a piece; n_st 0 (recorded) if it is not one that this plan can have.
__device__ __forceinline__ Piece make_piece(const PrefillParams& p, const PrefillUnit& u) {
    const int ps = p.page_size, G = p.group;
    Piece c{};
    TileWindow w;
    bool ok = u.n_pages >= 1 && u.kv_valid >= 1 && u.kv_valid < (1 << 30) && u.kv_begin >= 0 &&
              u.kv_begin % kTokens == 0 &&
              static_cast<int64_t>(u.kv_valid) <= static_cast<int64_t>(u.n_pages) * ps &&
              u.b >= 0 && u.b < p.batch && u.hkv >= 0 && u.hkv < p.num_kv_heads && u.n_tok >= 1 &&
              u.n_tok <= p.tile_tokens && u.n_tok * G <= kPrefillRows && u.q_begin >= 0 &&
              u.q_begin <= p.n_q_tokens - u.n_tok && u.p0 >= 0 && u.p0 < u.kv_len &&
              u.kv_len < (1 << 30) && u.q_len >= 1 && u.q_len <= u.kv_len &&
              u.n_pieces >= 1 && u.piece >= 0 && u.piece < u.n_pieces;
    if (ok) {
        w.init(p, u);
        ok = w.inside(u, ps, p.nnz);
    }
    if (ok && u.n_pieces > 1)
        ok = u.state >= 0 && (static_cast<int64_t>(u.state) +
                              static_cast<int64_t>(u.n_tok - 1) * u.n_pieces + u.piece + 1) *
                                     G <=
                                 p.n_states;
    if (!ok) {
        record_status(p.status, p.epoch, kDevicePlanMismatch);
        return c;
    }
    c.n_st = (u.kv_valid + kTokens - 1) / kTokens;
    c.pages = u.n_pages;
    c.first = u.page_base + u.kv_begin / ps;
    c.front = w.front;
    c.skip = w.skip;
    c.p0 = w.p0;
    c.sinks = w.sinks;
    // The call's first query sees from token lo on; what lies before it and is no sink no
    // query sees. (With skipped pages in between: the rest of the sinks' pages, and of the
    // first page behind them if that is the first query's.)
    const int begin = u.kv_begin;
    const int lo = u.kv_len - u.q_len - p.window + 1;
    c.hide0 = w.sinks;
    c.hide1 = max(min((w.front + begin / ps) * ps, lo), lo - w.skip * ps) - begin;
    c.end = u.kv_len - w.skip * ps - begin;
    c.q_begin = u.q_begin;
    c.n_tok = u.n_tok;
    c.hkv = u.hkv;
    c.state = u.state;
    c.n_pieces = u.n_pieces;
    c.piece = u.piece;
    // a half streams the stages up to the position of its last query
    const int rows = u.n_tok * G;
    for (int h = 0; h < 2; ++h) {
        const int end = w.p0 + (min(rows, 128 * (h + 1)) - 1) / G + 1;  // tokens seen
        c.nst[h] = rows > 128 * h && end > 0 ? min(c.n_st, (end + kTokens - 1) / kTokens) : 0;
    }
    c.n_st = max(c.nst[0], c.nst[1]);
    return c;
}

__global__ void __launch_bounds__(kThreads, 1)
    prefill_window_kernel(const __grid_constant__ CUtensorMap tmap_k,
                          const __grid_constant__ CUtensorMap tmap_v,
                          const __grid_constant__ CUtensorMap tmap_q,
                          const __grid_constant__ PrefillParams p) {
    extern __shared__ __align__(1024) uint8_t sm[];
    Ctl& ctl = *reinterpret_cast<Ctl*>(sm + kCtlOff);
    const Piece* list = reinterpret_cast<const Piece*>(sm + kListOff);
    volatile int* flags = ctl.flags;
    const uint32_t s_base = smem_addr(sm);
    auto ring_k = [&](int n) { return s_base + kKOff + (n % kStages) * kSlotBytes; };
    auto ring_v = [&](int n) { return s_base + kVOff + (n % kStages) * kSlotBytes; };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ps = p.page_size, G = p.group;
    // launched as a programmatic dependent: nothing in global memory before this
    grid_dependency_wait();

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&ctl.kfull[s], 1);
            mbar_init(&ctl.kempty[s], 1);
            mbar_init(&ctl.vfull[s], 1);
            mbar_init(&ctl.vempty[s], 1);
            ctl.kissued[s] = ctl.vissued[s] = 0;
        }
        ctl.landing = ctl.zeroed = 0;
        for (int h = 0; h < 2; ++h) {
            mbar_init(&ctl.q_ready[h], 128 % G == 0 ? 1 : 4);
            mbar_init(&ctl.s_ready[h], 1);
            mbar_init(&ctl.p_ready[h], 4);
            mbar_init(&ctl.o_done[h], 1);
            ctl.qissued[h] = 0;
        }
        mbar_init(&ctl.vland, 1);
        mbar_init(&ctl.mma_done, 1);
        flags[0] = 0;
        fence_mbar_init();
        if (blockIdx.x == 0) {
            *p.last_epoch = p.epoch;
            if (p.clear_stamp != nullptr) *p.clear_stamp = 0ull;
        }
        // The merge kernel, when the plan has one, may be scheduled now; it waits for
        // this grid to complete before it reads anything.
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile(
            "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                smem_addr(&ctl.tmem)),
            "r"(kTmemCols)
            : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == kKWarp && lane == 0) {
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_v);
        prefetch_tmap(&tmap_q);
    }
    {
        // the CTA's pieces, a thread a unit, checked before anything uses them (and the
        // operand buffers' alignment, which the swizzled copies need)
        const bool mine = (p.ws_stamp == nullptr || *p.ws_stamp == p.stamp) && (s_base & 1023u) == 0;
        const int a = p.cta_begin[blockIdx.x], e = p.cta_begin[blockIdx.x + 1];
        const bool ok = mine && a >= 0 && e >= a && e <= p.n_units && e - a <= kWindowUnits;
        const int n = ok ? e - a : 0;
        for (int i = threadIdx.x; i < n; i += kThreads)
            *reinterpret_cast<Piece*>(sm + kListOff + i * sizeof(Piece)) =
                make_piece(p, p.units[a + i]);
        if (threadIdx.x == 0) {
            if (!ok) record_status(p.status, p.epoch, kDevicePlanMismatch);
            flags[1] = n;
            flags[2] = a;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int n_pieces = flags[1];
    const uint32_t tmem = ctl.tmem;
    auto t_o = [&](int h) { return tmem + 128u * static_cast<uint32_t>(h); };
    auto t_s = [&](int h) { return tmem + 256u + 128u * static_cast<uint32_t>(h); };
    auto s_q = [&](int h) { return s_base + 2u * kQHalf * static_cast<uint32_t>(h); };

    if (warp == kKWarp || warp == kVWarp) {
        // ================================================ producer warps
        // Lane 2j + c copies 64-column half c of page j of a stage; the page's index is
        // read a stage ahead, over the ends of pieces too.
        const bool is_k = warp == kKWarp;
        const int pps = kTokens / ps;  // pages a stage (at most 16)
        uint64_t* full = is_k ? ctl.kfull : ctl.vfull;
        uint64_t* empty = is_k ? ctl.kempty : ctl.vempty;
        int* issued = is_k ? ctl.kissued : ctl.vissued;
        const CUtensorMap* map = is_k ? &tmap_k : &tmap_v;
        const int j = lane >> 1;
        auto page_of = [&](int pi, int s) {
            for (; pi < n_pieces && s >= list[pi].n_st; ++pi) s = 0;
            if (pi >= n_pieces) return 0;
            const Piece& c = list[pi];
            const int pg = s * pps + j;
            if (j >= pps || pg >= c.pages) return 0;
            return __ldg(p.indices + c.first + pg + (pg >= c.front ? c.skip : 0));
        };
        int next = page_of(0, 0), n = 0;  // n: stages so far
        bool ok = true;
        // The V warp zeroes the rows of a stage that no query sees once they have landed,
        // before it waits for the next slot (whole 128-byte rows, so the swizzle does not
        // matter).
        int z_piece = -1, z_stage = 0, z_n = 0, z_count = 0;
        auto zero_pending = [&]() {
            if (z_piece < 0) return true;
            const Piece& c = list[z_piece];
            const int slot = z_n % kStages, base = z_stage * kTokens;
            z_piece = -1;
            if (!__all_sync(0xffffffffu, mbar_wait(&ctl.vland, z_count & 1, flags, p.wait_ns)))
                return false;
            uint8_t* v0 = sm + kVOff + slot * kSlotBytes;
            auto zero_rows = [&](int r0, int r1) {  // (none where r1 is not above r0 >= 0)
                for (int i = lane; i < (max(r1, r0) - r0) * 16; i += 32) {
                    const int row = r0 + (i >> 4), cc = i & 15;
                    *reinterpret_cast<uint4*>(v0 + (cc >> 3) * kHalfBytes + row * 128 +
                                              (cc & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
            };
            zero_rows(min(max(c.end - base, 0), kTokens), kTokens);
            zero_rows(min(max(c.hide0 - base, 0), kTokens), min(c.hide1 - base, kTokens));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&full[slot]);
                issued[slot] += 1;
                ctl.zeroed += 1;
            }
            ++z_count;
            return true;
        };
        for (int pi = 0; pi < n_pieces && ok; ++pi) {
            const Piece& c = list[pi];
            const HiddenStages hid(c);
            const int ca = p.layout == 0 ? c.hkv : 0;  // (d, A, B, page): NHD (d, head, token,
            const int cb = p.layout == 0 ? 0 : c.hkv;  // page), HND (d, token, head, page)
            for (int s = 0; s < c.n_st; ++s, ++n) {
                const int slot = n % kStages;
                const int npg = min(pps, c.pages - s * pps);
                // an index outside the pool is recorded and reads page 0
                const bool bad = next < 0 || static_cast<int64_t>(next) >= p.num_pages;
                if (__any_sync(0xffffffffu, bad) && lane == 0)
                    record_status(p.status, p.epoch, kDeviceBadPage);
                const int page = bad ? 0 : next;
                next = page_of(pi, s + 1);
                if (!is_k && !zero_pending()) {
                    ok = false;
                    break;
                }
                int okw = 1;
                if (lane == 0 && n >= kStages)
                    okw = mbar_wait(&empty[slot], ((n / kStages) + 1) & 1, flags, p.wait_ns) ? 1 : 0;
                if (!__shfl_sync(0xffffffffu, okw, 0)) {
                    ok = false;
                    break;
                }
                const bool zero = !is_k && hid.among(s);
                uint64_t* bar = zero ? &ctl.vland : &full[slot];
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, npg * ps * kHeadDim * 2);
                    if (zero)
                        ctl.landing += 1;
                    else
                        issued[slot] += 1;
                }
                __syncwarp();
                if (lane < 2 * npg)
                    tma_load_4d((is_k ? ring_k(n) : ring_v(n)) + j * ps * 128 +
                                    ((lane & 1) ? kHalfBytes : 0),
                                map, bar, (lane & 1) * 64, ca, cb, page);
                if (zero) {
                    z_piece = pi;
                    z_stage = s;
                    z_n = n;
                }
            }
        }
        if (ok && !is_k) ok = zero_pending();
        if (is_k) {
            // the device tables must be the ones the plan was made from (read here, off the
            // way to the first products)
            for (int i = lane; i < n_pieces; i += 32) {
                const PrefillUnit u = p.units[flags[2] + i];
                if (list[i].n_st == 0 || u.b < 0 || u.b >= p.batch) continue;
                const int64_t L =
                    static_cast<int64_t>(p.indptr[u.b + 1] - p.indptr[u.b] - 1) * ps +
                    p.last_page_len[u.b];
                if (p.qo_indptr[u.b] != u.qo_b || p.indptr[u.b] != u.page_base || L != u.kv_len)
                    record_status(p.status, p.epoch, kDevicePlanMismatch);
            }
            __syncwarp();
        }
        if (!ok && lane == 0) {
            flags[0] = 1;
            record_status(p.status, p.epoch, kDeviceWaitTimeout);
        }
    } else if (warp == kMmaWarp) {
        // ================================================ MMA warp
        // Within a piece, for g = 1 ..: PV_0(g - 1), QK_0(g), PV_1(g - 1), QK_1(g) (QK_h
        // after PV_h, whose P lies in the scores' place; MMAs run in issue order); behind
        // a piece's last PVs come the next one's first scores. A K (V) slot is released
        // once the last half that reads it has issued its product.
        if (n_pieces > 0) {
            constexpr uint32_t kIdQK = umma_idesc(128, kTokens, 0);
            constexpr uint32_t kIdPV = umma_idesc(128, kHeadDim, 1);
            const uint64_t qd0[2] = {umma_sdesc(s_q(0), 16, 1024), umma_sdesc(s_q(1), 16, 1024)};
            bool ok = true;
            auto wait = [&](uint64_t* bar, int phase) {
                ok = __all_sync(0xffffffffu,
                                ok && mbar_wait_tc(bar, phase & 1, flags, p.wait_ns));
                return ok;
            };
            int n_p[2] = {0, 0}, n_q[2] = {0, 0};
            // the half's scores of stage g of a piece whose first stage is the CTA's n0-th
            auto qk = [&](int h, int nst0, int nst1, int g, int n0) {
                const int n = n0 + g;
                if (g == 0 && !wait(&ctl.q_ready[h], n_q[h]++)) return;
                if ((h == 0 || g >= nst0) && !wait(&ctl.kfull[n % kStages], n / kStages)) return;
                tc_fence_after();
                // K = 128 in steps of 16: 32 bytes of a 128-byte swizzled row; columns
                // 64..127 in the other half
                const uint64_t kd0 = umma_sdesc(ring_k(n), 16, 1024);
#pragma unroll
                for (int ks = 0; ks < kHeadDim / 16; ++ks) {
                    const int a = ks >> 2, kk = ks & 3;
                    umma_ss_warp(t_s(h), qd0[h] + static_cast<uint64_t>((a * kQHalf + kk * 32) >> 4),
                                 kd0 + static_cast<uint64_t>((a * kHalfBytes + kk * 32) >> 4),
                                 kIdQK, ks > 0 ? 1u : 0u);
                }
                umma_commit_warp(&ctl.s_ready[h]);
                if (h == 1 || g >= nst1) umma_commit_warp(&ctl.kempty[n % kStages]);
            };
            auto pv = [&](int h, int nst0, int nst1, int g, int n0) {
                const int n = n0 + g;
                if (!wait(&ctl.p_ready[h], n_p[h]++)) return;
                if ((h == 0 || g >= nst0) && !wait(&ctl.vfull[n % kStages], n / kStages)) return;
                tc_fence_after();
                // 16 tokens a step = two 8-row groups (1024 B apart); the two 64-column
                // halves of V are kHalfBytes apart
                const uint64_t vd0 = umma_sdesc(ring_v(n), kHalfBytes, 1024);
#pragma unroll
                for (int ks = 0; ks < kTokens / 16; ++ks)
                    umma_ts_warp(t_o(h), t_s(h) + 8u * ks, vd0 + static_cast<uint64_t>(ks * 2048 >> 4),
                                 kIdPV, (ks > 0 || g > 0) ? 1u : 0u);
                if (g == (h ? nst1 : nst0) - 1) umma_commit_warp(&ctl.o_done[h]);
                if (h == 1 || g >= nst1) umma_commit_warp(&ctl.vempty[n % kStages]);
            };
            auto usable = [&](int pi) {
                while (pi < n_pieces && list[pi].n_st == 0) ++pi;
                return pi;
            };
            int pi = usable(0), n0 = 0;
            int nst0 = 0, nst1 = 0, next0 = 0, next1 = 0;
            if (pi < n_pieces) {
                next0 = list[pi].nst[0];
                next1 = list[pi].nst[1];
                if (next0 > 0) qk(0, next0, next1, 0, 0);
                if (ok && next1 > 0) qk(1, next0, next1, 0, 0);
            }
            while (pi < n_pieces && ok) {
                nst0 = next0;
                nst1 = next1;
                pi = usable(pi + 1);
                next0 = pi < n_pieces ? list[pi].nst[0] : 0;
                next1 = pi < n_pieces ? list[pi].nst[1] : 0;
                const int n_st = max(nst0, nst1);
                for (int g = 1; g <= n_st && ok; ++g) {
                    if (g - 1 < nst0) pv(0, nst0, nst1, g - 1, n0);
                    if (ok && g < nst0) qk(0, nst0, nst1, g, n0);
                    if (ok && g == n_st && next0 > 0) qk(0, next0, next1, 0, n0 + n_st);
                    if (ok && g - 1 < nst1) pv(1, nst0, nst1, g - 1, n0);
                    if (ok && g < nst1) qk(1, nst0, nst1, g, n0);
                    if (ok && g == n_st && next1 > 0) qk(1, next0, next1, 0, n0 + n_st);
                }
                n0 += n_st;
            }
            if (!ok && lane == 0) {
                flags[0] = 1;
                record_status(p.status, p.epoch, kDeviceWaitTimeout);
            }
            // every MMA completes before the tensor memory is released
            umma_commit_warp(&ctl.mma_done);
            mbar_wait(&ctl.mma_done, 0, nullptr, kWaitTimeoutNs);
        }
        __syncwarp();
    } else {
        // ================================================ softmax warpgroups
        // Warpgroup h (warps 4h .. 4h + 3) owns half h; thread r of it owns row 128 h + r
        // of a tile, TMEM lane r (warp w reads lanes [32 (w % 4), +32)). Every lane waits
        // on each barrier itself; results are AND-ed over the warp so the collective TMEM
        // instructions see one path.
        auto wait_all = [&](uint64_t* bar, int phase) {
            return __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, flags, p.wait_ns));
        };
        const int h = warp >> 2, wq = warp & 3;
        const uint32_t lane_off = static_cast<uint32_t>(32 * wq) << 16;
        const int r = threadIdx.x & 127;
        const int R = 128 * h + r;  // row of the tile: token R / G, head R % G
        const int t = R / G;
        const uint32_t g_magic = (65536u + G - 1) / G;  // R / G = R * magic >> 16 below 256
        const uint32_t ts = t_s(h);
        // (a scale of zero as the smallest normal number: a masked score stays -inf)
        const float sc = p.scale_log2 != 0.f ? p.scale_log2 : 1.17549435e-38f;
        const float hidden = sc > 0.f ? -INFINITY : INFINITY;  // times sc: -inf

        // Copies the half's query rows of piece `c` into shared memory, laid out as the
        // score MMA's A operand: two 64-column halves of [128 rows][128 B] with the
        // 128-byte swizzle (16-byte chunk j of row r at chunk j ^ (r % 8)). Where G divides
        // 128 the half's rows are a box of G heads x 128 / G tokens (rows past the tile are
        // other queries, or zeros behind the last); otherwise a warp copies its 32 rows, 16
        // lanes a row, zeros past the tile.
        const bool boxed = 128 % G == 0;
        auto copy_query = [&](const Piece& c) {
            if (boxed) {
                if (r == 0) {
                    ctl.qissued[h] += 1;
                    mbar_arrive_expect_tx(&ctl.q_ready[h], 2 * kQHalf);
                    tma_load_3d(s_q(h), &tmap_q, &ctl.q_ready[h], 0, c.hkv * G,
                                c.q_begin + h * (128 / G));
                    tma_load_3d(s_q(h) + kQHalf, &tmap_q, &ctl.q_ready[h], 64, c.hkv * G,
                                c.q_begin + h * (128 / G));
                }
                return;
            }
            const int col = lane & 15;
#pragma unroll 1
            for (int i = 0; i < 16; ++i) {
                const uint32_t row = 32 * wq + 2 * i + (lane >> 4);
                const uint32_t RR = 128 * h + row, tt = RR * g_magic >> 16;
                const uint32_t dst = s_q(h) + (col >> 3) * kQHalf + row * 128 +
                                     (((col & 7) ^ (row & 7)) << 4);
                if (static_cast<int>(tt) < c.n_tok)
                    cp_async16(dst, p.q + (static_cast<size_t>(c.q_begin + tt) * p.num_qo_heads +
                                           c.hkv * G + (RR - tt * G)) * kHeadDim + col * 8);
                else
                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0)
                                 : "memory");
            }
        };
        auto query_ready = [&]() {
            if (boxed) return;
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.q_ready[h]);
        };
        auto usable = [&](int pi) {
            while (pi < n_pieces && list[pi].nst[h] == 0) ++pi;
            return pi;
        };

        int n = 0;        // scores of this half so far
        int n_o = 0;      // pieces of this half so far
        bool ok = true;
        if (usable(0) < n_pieces) {
            copy_query(list[usable(0)]);
            query_ready();
        }
        for (int pi = 0; pi < n_pieces && ok; ++pi) {
            const Piece c = list[pi];
            const int nst = c.nst[h];
            // (padding rows see what the tile's last query sees)
            const int pos = c.p0 + min(t, c.n_tok - 1);
            const int w_lo = pos - p.window + 1;  // the row sees [w_lo, pos] and [0, sinks)
            const int pos_a = __shfl_sync(0xffffffffu, pos, 0);   // the warp's first
            const int pos_z = __shfl_sync(0xffffffffu, pos, 31);  // and last position
            const int lo_z = pos_z - p.window + 1;
            // whether every row of the warp sees the columns [c0, c1)
            auto all_see = [&](int c0, int c1) {
                return c1 <= pos_a + 1 && (c0 >= lo_z || c1 <= c.sinks);
            };
            auto sees = [&](int v) {
                return static_cast<unsigned>(v - w_lo) < static_cast<unsigned>(p.window) ||
                       (v < c.sinks && v <= pos);
            };
            float m_ref = -INFINITY, l = 0.f;
            for (int g = 0; g < nst; ++g, ++n) {
                if (!wait_all(&ctl.s_ready[h], n)) {
                    ok = false;
                    break;
                }
                // s_ready(n) also means that every MMA issued before QK_h(n) is done:
                // PV_h of the stage before among them (O_h is up to date)
                tc_fence_after();
                const bool last = g == nst - 1;
                if (last) {
                    // the query rows are read: the next piece's may come
                    const int next = usable(pi + 1);
                    if (next < n_pieces) copy_query(list[next]);
                }
                const int base = g * kTokens;
                float lq[4] = {0.f, 0.f, 0.f, 0.f};
                bool rescale = false, done = false;
                float alpha = 1.f;
                const bool whole = all_see(base, base + kTokens);
                // the columns that the row sees, a bit each
                unsigned long long see[2] = {~0ull, ~0ull};
                if (!whole) {
                    const int from = w_lo - base, to = pos + 1 - base;
                    const int first = min(c.sinks - base, to);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        see[k] = (below(to - 64 * k) & ~below(from - 64 * k)) | below(first - 64 * k);
                }
                if (__any_sync(0xffffffffu, m_ref == -INFINITY)) {
                    // rows without a reference take the maximum of what they see of the last
                    // block of 16 columns of which they see some (one block, where a window
                    // starts or a stage is seen whole; up to three at its end, where a warp's
                    // rows end in different ones: with the last block alone the others' rows
                    // took two passes, 8 prompts of 2048 with 16 query and 8 KV heads at
                    // window 512 165 us, 125 so)
#pragma unroll 1
                    for (int i = 7; i >= 0; --i) {
                        const uint32_t bits =
                            static_cast<uint32_t>((i >= 4 ? see[1] : see[0]) >> (16 * (i & 3))) & 0xffffu;
                        const bool want = m_ref == -INFINITY && bits != 0;
                        if (!__any_sync(0xffffffffu, want)) continue;
                        uint32_t a[16];
                        tmem_ld16_async(ts + lane_off + 16 * i, a);
                        tmem_ld_wait16(a);
                        float mx = -INFINITY;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (bits >> j & 1) mx = fmaxf(mx, __uint_as_float(a[j]) * sc);
                        if (want) m_ref = mx;
                        if (!__any_sync(0xffffffffu, m_ref == -INFINITY)) break;
                    }
                }
                {
                    // P = 2^(s sc - m_ref) for 16 columns at a time (the next 16 loading
                    // meanwhile), kept in registers until the row's sum shows that no
                    // term exceeds 2^64 (nor is infinite). The reference may lag the
                    // row's maximum: every term carries the same factor 2^(m - m_ref),
                    // which the final O / l cancels.
                    uint32_t pk[64];
                    uint32_t a[16], b[16];
                    // (a row that has seen nothing yet keeps a reference of 0 for now)
                    const float mr = m_ref == -INFINITY ? 0.f : m_ref;
                    auto math = [&](uint32_t (&x)[16], int i) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float x0, x1;
                            fma2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]), sc, -mr,
                                 x0, x1);
                            const float p0 = fast_exp2(x0);
                            const float p1 = fast_exp2(x1);
                            add2(lq[(j & 1) * 2], lq[(j & 1) * 2 + 1], p0, p1);
                            pk[8 * i + j] = pack_bf16x2(p0, p1);
                        }
                    };
                    auto edge = [&](uint32_t (&x)[16], int i) {
                        const uint32_t bits = static_cast<uint32_t>(see[i >> 2] >> 16 * (i & 3));
                        if (!__any_sync(0xffffffffu, (bits & 0xffffu) != 0)) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) pk[8 * i + j] = 0u;
                            return;
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (!(bits >> j & 1)) x[j] = __float_as_uint(hidden);
                        math(x, i);
                    };
                    auto pass = [&](auto&& chunk) {
                        tmem_ld16_async(ts + lane_off, a);
                        tmem_ld_wait16(a);
#pragma unroll
                        for (int i = 0; i < 8; i += 2) {
                            tmem_ld16_async(ts + lane_off + 16 * (i + 1), b);
                            chunk(a, i);
                            tmem_ld_wait16(b);
                            if (i + 2 < 8) tmem_ld16_async(ts + lane_off + 16 * (i + 2), a);
                            chunk(b, i + 1);
                            if (i + 2 < 8) tmem_ld_wait16(a);
                        }
                    };
                    if (whole)
                        pass(math);
                    else
                        pass(edge);
                    const float ltot = (lq[0] + lq[1]) + (lq[2] + lq[3]);
                    // (a row without a reference that has seen something goes back too)
                    const bool good = ltot <= 0x1p64f && (m_ref > -INFINITY || ltot == 0.f);
                    if (__all_sync(0xffffffffu, good)) {
                        uint32_t (&p0)[32] = *reinterpret_cast<uint32_t (*)[32]>(&pk[0]);
                        uint32_t (&p1)[32] = *reinterpret_cast<uint32_t (*)[32]>(&pk[32]);
                        tmem_st32(ts + lane_off, p0);
                        tmem_st32(ts + lane_off + 32, p1);
                        done = true;
                    } else {
                        lq[0] = lq[1] = lq[2] = lq[3] = 0.f;
                    }
                }
                if (!done) {
                    // Two passes, 32 columns at a time (P goes over scores already read).
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        uint32_t a[32];
                        tmem_ld32(ts + lane_off + 32 * i, a);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (sees(base + 32 * i + j)) mx = fmaxf(mx, __uint_as_float(a[j]) * sc);
                    }
                    if (g == 0) {
                        m_ref = mx;
                    } else if (mx > m_ref + 8.f) {
                        alpha = fast_exp2(m_ref - mx);  // 0 while nothing was visible
                        m_ref = mx;
                        l *= alpha;
                        rescale = true;
                    }
                    const float mr = m_ref == -INFINITY ? 0.f : m_ref;
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        uint32_t a[32], pk[16];
                        tmem_ld32(ts + lane_off + 32 * i, a);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const int v = base + 32 * i + 2 * j;
                            const float x0 =
                                sees(v) ? __uint_as_float(a[2 * j]) * sc : -INFINITY;
                            const float x1 =
                                sees(v + 1) ? __uint_as_float(a[2 * j + 1]) * sc : -INFINITY;
                            const float p0 = fast_exp2(x0 - mr);
                            const float p1 = fast_exp2(x1 - mr);
                            lq[j & 3] += p0 + p1;
                            pk[j] = pack_bf16x2(p0, p1);
                        }
                        tmem_st16(ts + lane_off + 16 * i, pk);
                    }
                }
                l += (lq[0] + lq[1]) + (lq[2] + lq[3]);
                if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
                    for (int c0 = 0; c0 < kHeadDim; c0 += 32) {
                        uint32_t o[32];
                        tmem_ld32(t_o(h) + lane_off + c0, o);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                        tmem_st32(t_o(h) + lane_off + c0, o);
                    }
                }
                tmem_wait_st();
                if (last && usable(pi + 1) < n_pieces) query_ready();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.p_ready[h]);
            }
            // ---- epilogue: O / l once the half's last PV is done; padding rows take part
            // in the collective loads. A piece that the half's rows see nothing of leaves
            // them an empty state (a split tile's merge weighs it 0).
            if (ok && nst > 0 && !wait_all(&ctl.o_done[h], n_o++)) ok = false;
            if (ok && (nst > 0 || (c.n_st > 0 && c.n_pieces > 1))) {
                tc_fence_after();
                const bool seen = l != 0.f;  // (NaN scores: out and lse are NaN)
                const float inv = seen ? 1.f / l : 0.f;
                const float lse2 = seen ? m_ref + __log2f(l) : -INFINITY;
                // The rows go out through shared memory, 128 bytes of each at a time, so that
                // eight lanes write a whole line (a lane its own row: 32 lines a store,
                // 300 -> 272 us without them). 16-byte chunk j of row i at j ^ (i % 8).
                uint8_t* stage = sm + kOutOff + warp * kOutBytes;
                const bool whole_tile = c.n_pieces == 1;
                const size_t row_bytes = whole_tile ? kHeadDim * 2 : kHeadDim * 4;
                uint8_t* dst0 = whole_tile ? reinterpret_cast<uint8_t*>(p.out)
                                           : reinterpret_cast<uint8_t*>(p.part_o);
                // row of the output, or of the partial states, of row RR of the tile
                auto out_row = [&](uint32_t RR) {
                    const uint32_t tt = RR * g_magic >> 16, gg = RR - tt * G;
                    if (static_cast<int>(tt) >= c.n_tok) return int64_t{-1};
                    return whole_tile
                               ? static_cast<int64_t>(c.q_begin + tt) * p.num_qo_heads + c.hkv * G + gg
                               : (static_cast<int64_t>(c.state) +
                                  static_cast<int64_t>(tt) * c.n_pieces + c.piece) * G + gg;
                };
                auto send = [&](int byte0) {  // 128 bytes of every row, from byte0 on
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int rr = 4 * i + (lane >> 3), j = lane & 7;
                        const uint4 w = *reinterpret_cast<const uint4*>(stage + rr * 128 +
                                                                        ((j ^ (rr & 7)) << 4));
                        const int64_t to = out_row(128 * h + 32 * wq + rr);
                        if (to >= 0)
                            *reinterpret_cast<uint4*>(dst0 + to * row_bytes + byte0 + j * 16) = w;
                    }
                    __syncwarp();
                };
                if (whole_tile) {
#pragma unroll 1
                    for (int c0 = 0; c0 < kHeadDim; c0 += 64) {
                        uint32_t o[64];
                        tmem_ld64(t_o(h) + lane_off + c0, o);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                w[k] = pack_bf16x2(__uint_as_float(o[8 * j + 2 * k]) * inv,
                                                   __uint_as_float(o[8 * j + 2 * k + 1]) * inv);
                            *reinterpret_cast<uint4*>(stage + lane * 128 +
                                                      ((j ^ (lane & 7)) << 4)) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        send(c0 * 2);
                    }
                } else {
#pragma unroll 1
                    for (int c0 = 0; c0 < kHeadDim; c0 += 32) {
                        uint32_t o[32];
                        if (nst > 0) {
                            tmem_ld32(t_o(h) + lane_off + c0, o);
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] = 0u;
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<float4*>(stage + lane * 128 +
                                                       ((j ^ (lane & 7)) << 4)) =
                                make_float4(__uint_as_float(o[4 * j]) * inv,
                                            __uint_as_float(o[4 * j + 1]) * inv,
                                            __uint_as_float(o[4 * j + 2]) * inv,
                                            __uint_as_float(o[4 * j + 3]) * inv);
                        send(c0 * 4);
                    }
                }
                const int64_t row = out_row(R);
                if (row >= 0) {
                    if (!whole_tile)
                        p.part_lse[row] = l != l ? INFINITY : lse2;
                    else if (p.lse != nullptr)
                        p.lse[row] = lse2 * kLn2;
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (!ok && lane == 0) {
            flags[0] = 1;
            record_status(p.status, p.epoch, kDeviceWaitTimeout);
        }
    }
    tc_fence_before();
    __syncthreads();  // every warp has left its loop; the MMAs have completed

    if (flags[0] && threadIdx.x == 0) {
        // Aborted: wait (bounded) for the copies already issued, then leave.
        for (int s = 0; s < kStages; ++s) {
            if (ctl.kissued[s] > 0)
                mbar_wait(&ctl.kfull[s], (ctl.kissued[s] - 1) & 1, nullptr, kWaitTimeoutNs);
            if (ctl.vissued[s] > 0)
                mbar_wait(&ctl.vfull[s], (ctl.vissued[s] - 1) & 1, nullptr, kWaitTimeoutNs);
        }
        if (ctl.landing > ctl.zeroed)
            mbar_wait(&ctl.vland, (ctl.landing - 1) & 1, nullptr, kWaitTimeoutNs);
        for (int h = 0; h < 2; ++h)
            if (ctl.qissued[h] > 0)
                mbar_wait(&ctl.q_ready[h], (ctl.qissued[h] - 1) & 1, nullptr, kWaitTimeoutNs);
    }
    if (warp == kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kTmemCols)
                     : "memory");
    }
}

}  // namespace

cudaError_t launch_prefill_window(const CUtensorMap& tk, const CUtensorMap& tv,
                                  const CUtensorMap& tq, const PrefillParams& p, int grid,
                                  cudaStream_t stream) {
    if (grid < 1 || p.window < 1 || p.cta_begin == nullptr) return cudaErrorInvalidConfiguration;
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
    if (bit == 0 || !(done.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(prefill_window_kernel,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prefill_window_kernel, tk, tv, tq, p);
}

}  // namespace oxd
