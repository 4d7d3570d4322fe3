// Decode attention over a 4-bit paged cache for sm_103a (oxd_quant_decode_run),
// groups of 9 to 32 query heads. The mathematics, the conversion of codes, the
// lazy maximum and the copies are those of oxd_decode_quant.cu; there a warp
// takes its own tokens through both products, which needs 32 accumulator
// registers for every 8 heads. Here
//   * the four warps of a CTA take 64 tokens at a time together. Warp w forms
//     the scores of tokens 16w .. 16w + 15 with every head, and the output
//     columns 32w .. 32w + 31 (a scale group) over all 64 tokens, so a code is
//     converted once whatever the group, a warp's accumulator is 8 registers for
//     every 8 heads, and a unit ends without merging accumulators. Between the
//     halves the weights P go through shared memory: one barrier a stage.
// One kernel for every group was measured: for up to 8 heads the other runs the
// steady stream 1.25 times faster (no barriers, fewer instructions a token), for
// 16 and 32 this one ends a unit in half the time and keeps its accumulators in
// registers (spilled: up to 24 bytes for 16 heads, 28 to 76 for 32). What bounds
// it is issue and latency: 3 to 4 warps a scheduler at half their rate,
// mma.sync at 38 % of its own (32 heads, 16 x 32768 tokens: 45 to 47 us, 25 % of
// the copy rate; four CTAs a SM with a shorter ring 57; 16 heads 3.0 TB/s). On
// tcgen05, a token a thread and K as the A operand in tensor memory, the same
// took 42.5 us, but 16 heads 12 % longer than here and short streams 35 %.
// In an NHD pool the two heads of a pair run on neighbouring CTAs.
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "oxd_decode_quant.cuh"

namespace oxd {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kWarpTokens = 16;                     // a warp's tokens of a stage
constexpr int kStageTokens = kWarps * kWarpTokens;  // 64

// kNT: 8-head tiles. kCtas: resident CTAs a SM, which caps the registers at
// 65536 / (kThreads * kCtas). kPs: page size.
template <int kNT_, int kStages_, int kCtas_, int kPs_>
struct QCfg {
    static constexpr int kNT = kNT_;
    static constexpr int kRows = 8 * kNT;
    static constexpr int kStages = kStages_;
    static constexpr int kCtas = kCtas_;
    static constexpr int kPs = kPs_;
    static constexpr bool kQInRegs = kNT <= 2;  // query fragments, else read from shared memory
    static constexpr int kWarpPages = kPs < kWarpTokens ? kWarpTokens / kPs : 1;
    static constexpr int kRun = 32 / kWarpPages;  // stages whose pages a window of 32 holds
    // stage: K codes | V codes | K scales | V scales of 64 tokens. 16-byte piece
    // i of a token's codes sits at piece i ^ (token / 2 % 4).
    static constexpr int kVOff = kStageTokens * kCodeBytes;
    static constexpr int kKsOff = 2 * kVOff;
    static constexpr int kVsOff = kKsOff + kStageTokens * kScaleBytes;
    static constexpr int kSlotBytes = kVsOff + kStageTokens * kScaleBytes;
    // weights of a stage, as B fragments [16-token block][tile pair][lane] 16 bytes,
    // and V's scales [group][token] f16; two of each
    static constexpr int kPOff = kStages * kSlotBytes;
    static constexpr int kPBytes = kWarps * kNT * 256;
    static constexpr int kTOff = kPOff + 2 * kPBytes;
    static constexpr int kTBytes = kRowScales * kStageTokens * 2;
    // query fragments [group c][tile][lane] 16 bytes, and the next unit's query
    // rows as they come from memory
    static constexpr int kQOff = kTOff + 2 * kTBytes;
    static constexpr int kQBytes = kRows * kHeadDim * 2;
    static constexpr int kRawOff = kQOff + kQBytes;
    static constexpr int kBarOff = kRawOff + kQBytes;            // their mbarrier
    static constexpr int kScOff = kBarOff + 16;                  // logit scales [kRows]
    static constexpr int kMaxOff = kScOff + kRows * 4;           // maxima [warp][kRows]
    static constexpr int kSumOff = kMaxOff + kWarps * kRows * 4; // denominators [warp][kRows]
    static constexpr int kRangeOff = kSumOff + kWarps * kRows * 4;
    static constexpr int kCurOff = kRangeOff + 16;               // the current and next unit
    static constexpr int kListOff = kCurOff + 2 * 32;
    static constexpr int kSmemBytes = kListOff + kListed * 32;
    static_assert(kCtas * (kSmemBytes + 1024) <= 228 * 1024, "the CTAs fit a SM");
};
template <int kPs> using CfgQ16 = QCfg<2, 4, 4, kPs>;
template <int kPs> using CfgQ32 = QCfg<4, 4, 3, kPs>;

using List = UnitList<false>;

__device__ __forceinline__ int stages_of(const Unit& u) {
    return (u.valid + kStageTokens - 1) / kStageTokens;
}

// One warp's stream of copies: its 16 tokens of every stage of the CTA's units,
// ahead of their use. The page indices of a run of stages sit in the lanes
// (`win`, the next run in `ahead`), and the next unit's first indices are read
// while the current unit's stages are still being issued.
template <class C>
struct Stream {
    int u_end, unit;             // unit being issued
    int n_pages, n_stages, first;
    int st;                      // its next stage
    int win_st, win, ahead;      // indices of the stages from win_st on, and of the next run
    int nx_win;                  // unit + 1's first indices
    // this lane's addresses in page 0 of the unit's head: the 16-byte piece
    // lane % 4 of token lane / 4 of K and V, and the scales of tokens
    // 2 (lane % 8), + 1 of K (lanes 0..7) or V (8..15)
    const uint8_t* k;
    const uint8_t* v;
    const uint8_t* sc;

    __device__ __forceinline__ int load_window(const int32_t* indices, int x_first, int x_stages,
                                               int x_pages, int st0, int warp, int lane) const {
        const int s = st0 + lane / C::kWarpPages;
        const int pg = (s * kStageTokens + warp * kWarpTokens) / C::kPs + lane % C::kWarpPages;
        return s < x_stages && pg < x_pages ? __ldg(indices + x_first + pg) : 0;
    }
    // An index outside the pool is recorded and replaced by page 0.
    __device__ __forceinline__ int check(const DecodeParams& p, int i, int lane) const {
        const bool bad = i < 0 || static_cast<int64_t>(i) >= p.num_pages;
        if (__any_sync(0xffffffffu, bad) && lane == 0)
            record_status(p.status, p.epoch, kDeviceBadPage);
        return bad ? 0 : i;
    }
    __device__ __forceinline__ void load_next_window(const QuantDecodeParams& qp,
                                                     const List& units, int warp, int lane) {
        if (unit + 1 < u_end) {
            const Unit x = units.get(qp, unit + 1);
            nx_win = load_window(qp.d.indices, x.first, stages_of(x), x.n_pages, 0, warp, lane);
        }
    }
    // Enters `unit`, whose first indices are in nx_win.
    __device__ __forceinline__ void enter(const QuantDecodeParams& qp, const List& units,
                                          int warp, int lane) {
        const DecodeParams& p = qp.d;
        const Unit u = units.get(qp, unit);
        n_pages = u.n_pages;
        n_stages = stages_of(u);
        first = u.first;
        st = win_st = 0;
        const int h = u.valid > 0 ? u.h : 0;
        // (tokens of a page that a stage's part of a warp may begin in the middle of)
        const int t = (warp * kWarpTokens + (lane >> 2)) % C::kPs;
        const size_t row = row_index(p.layout, 0, t, h, p.num_kv_heads, C::kPs);
        k = qp.k_codes + row * kCodeBytes + (lane & 3) * 16;
        v = qp.v_codes + row * kCodeBytes + (lane & 3) * 16;
        const int ts = (warp * kWarpTokens + 2 * (lane & 7)) % C::kPs;
        sc = reinterpret_cast<const uint8_t*>((lane < 8 ? qp.k_scales : qp.v_scales) +
                                              scale_index(0, ts, h, p.num_kv_heads, C::kPs));
        win = check(p, nx_win, lane);
        ahead = load_window(p.indices, first, n_stages, n_pages, C::kRun, warp, lane);
        load_next_window(qp, units, warp, lane);
    }
    // Issues the next stage's copies into `slot`, if there is one; always one
    // more copy group. dst / sdst: this lane's offsets in it. Pages past the
    // unit's last are read as page 0.
    __device__ __forceinline__ void issue(const QuantDecodeParams& qp, const List& units,
                                          uint32_t slot, uint32_t dst, uint32_t sdst, int warp,
                                          int lane) {
        const DecodeParams& p = qp.d;
        while (unit < u_end && st >= n_stages) {
            ++unit;
            if (unit < u_end) enter(qp, units, warp, lane);
        }
        if (unit < u_end) {
            if (st - win_st >= C::kRun) {
                win = check(p, ahead, lane);
                win_st += C::kRun;
                ahead = load_window(p.indices, first, n_stages, n_pages, win_st + C::kRun, warp, lane);
            }
            const int w0 = (st - win_st) * C::kWarpPages;
            // bytes of one token and of a page
            const uint32_t tok = p.layout == 0 ? p.num_kv_heads * kCodeBytes : kCodeBytes;
            const uint32_t page_bytes = p.num_kv_heads * (C::kPs * kCodeBytes);
#pragma unroll
            for (int i = 0; i < kWarpTokens / 8; ++i) {  // eight tokens of K and of V
                const uint32_t page = __shfl_sync(0xffffffffu, win, w0 + i * 8 / C::kPs % C::kWarpPages);
                const size_t off =
                    static_cast<size_t>(page) * page_bytes + (C::kPs > 8 ? i * 8 * tok : 0);
                cp_async16(slot + dst + i * 8 * kCodeBytes, k + off);
                cp_async16(slot + dst + C::kVOff + i * 8 * kCodeBytes, v + off);
            }
            const uint32_t page = __shfl_sync(
                0xffffffffu, win, w0 + 2 * (lane & 7) / C::kPs % C::kWarpPages);
            if (lane < 16) cp_async16(slot + sdst, sc + static_cast<size_t>(page) * (page_bytes / 8));
            ++st;
        }
        cp_async_commit();
    }
};

template <class C>
struct State {
    uint4 q[C::kQInRegs ? 4 : 1][C::kQInRegs ? C::kNT : 1];
    uint32_t q_addr;           // this lane's query fragments in shared memory
    float sc[C::kNT][2];       // logit scale (log2) of heads 2 tq, 2 tq + 1, positive
    float l[C::kNT][2];        // denominators, this lane's tokens' part
    float mu[C::kNT][2];       // 10 - m (inf: no m yet): from a scaled score to its weight's exponent
    float acc[C::kNT][2][4];   // columns 4 g, 4 g + 1 | 4 g + 2, 4 g + 3 of the warp's 32

    __device__ __forceinline__ void init(uint8_t* base, int lane) {
        q_addr = smem_addr(base) + C::kQOff + lane * 16;
        if constexpr (C::kQInRegs) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int n = 0; n < C::kNT; ++n) q[c][n] = lds128(q_addr + (c * C::kNT + n) * 512);
        }
        const float* s = reinterpret_cast<const float*>(base + C::kScOff);
#pragma unroll
        for (int n = 0; n < C::kNT; ++n) {
            const float2 f = *reinterpret_cast<const float2*>(s + n * 8 + 2 * (lane & 3));
            sc[n][0] = f.x;
            sc[n][1] = f.y;
            mu[n][0] = mu[n][1] = INFINITY;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                acc[n][i][0] = acc[n][i][1] = acc[n][i][2] = acc[n][i][3] = 0.f;
        }
    }

    // Scores of the warp's 16 tokens (rows g and g + 8) with heads 2 tq, 2 tq + 1
    // of each tile. `k_at`: this lane's ldmatrix row, `ks_at`: row g's scales.
    __device__ __forceinline__ void scores(float (&s)[C::kNT][4], uint32_t k_at, uint32_t ks_at) {
        const uint2 ks0 = lds64(ks_at), ks1 = lds64(ks_at + 8 * kScaleBytes);
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
            uint32_t w[4];
            ldsm_x4(k_at ^ (c << 4), w);
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
                const int grp = c + cc;
                uint32_t a[4], b[4];
                codes_to_f16(w[2 * cc], a);
                codes_to_f16(w[2 * cc + 1], b);
                const float2 f0 = f16x2_floats(c ? ks0.y : ks0.x);
                const float2 f1 = f16x2_floats(c ? ks1.y : ks1.x);
                const float e0 = cc ? f0.y : f0.x, e1 = cc ? f1.y : f1.x;
#pragma unroll
                for (int n = 0; n < C::kNT; ++n) {
                    uint4 qf;
                    if constexpr (C::kQInRegs)
                        qf = q[grp][n];
                    else
                        qf = lds128(q_addr + (grp * C::kNT + n) * 512);
                    float t[4];
                    mma_f16_zero(t, a[0], b[0], a[1], b[1], qf.x, qf.y);
                    mma_f16(t, a[2], b[2], a[3], b[3], qf.z, qf.w);
                    if (grp == 0) {
                        s[n][0] = t[0] * e0;
                        s[n][1] = t[1] * e0;
                        s[n][2] = t[2] * e1;
                        s[n][3] = t[3] * e1;
                    } else {
                        fma_pair(s[n][0], s[n][1], t[0], t[1], e0);
                        fma_pair(s[n][2], s[n][3], t[2], t[3], e1);
                    }
                }
            }
        }
    }

    // Weights of the scores (score s counts as s * sc) as P^T fragments at
    // `p_at`, and their sums over this lane's two tokens.
    __device__ __forceinline__ void weights(const float (&s)[C::kNT][4], float (&sum)[C::kNT][2],
                                            uint32_t p_at) {
#pragma unroll
        for (int n = 0; n < C::kNT; n += 2) {
            uint32_t f[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float y[4];
                const float* x = s[n + i];
                fma_pairs(y[0], y[1], x[0], x[1], sc[n + i][0], sc[n + i][1], mu[n + i][0],
                          mu[n + i][1]);
                fma_pairs(y[2], y[3], x[2], x[3], sc[n + i][0], sc[n + i][1], mu[n + i][0],
                          mu[n + i][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = fast_exp2(y[e]);
                f[2 * i] = transpose_8x8(pack_f16x2(y[0], y[1]));
                f[2 * i + 1] = transpose_8x8(pack_f16x2(y[2], y[3]));
                sum[n + i][0] = y[0] + y[2];
                sum[n + i][1] = y[1] + y[3];
            }
            sts128(p_at + n / 2 * 512, f);
        }
    }

    // O^T += V^T P^T over the stage's 64 tokens. `v_at`: this lane's ldmatrix
    // row of the first 32, `p_at`: its fragments of P, `t_at`: the scales of
    // tokens 2 tq, 2 tq + 1 in the warp's group.
    __device__ __forceinline__ void values(uint32_t v_at, uint32_t p_at, uint32_t t_at) {
        constexpr uint32_t kLow = 0x0f0f0f0fu;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t r[4];  // 8 tokens each: four columns of tokens 2 tq | 2 tq + 1
            ldsm_x4_trans(v_at + half * 32 * kCodeBytes, r);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int tb = half * 2 + i;
                const uint32_t s0 = lds32(t_at + tb * 32), s1 = lds32(t_at + tb * 32 + 16);
                // the first tokens of the two 8-token halves, and the second
                const uint32_t x = __byte_perm(r[2 * i], r[2 * i + 1], 0x5410);
                const uint32_t y = __byte_perm(r[2 * i], r[2 * i + 1], 0x7632);
                uint32_t u[4], v[4];
                codes_to_f16((x & kLow) | ((y << 4) & ~kLow), u);  // columns 0, 2 | 0, 2 of 8 on
                codes_to_f16(((x >> 4) & kLow) | (y & ~kLow), v);  // columns 1, 3
                const uint32_t a0 = mul_f16x2(u[0], s0), a1 = mul_f16x2(v[0], s0);
                const uint32_t a2 = mul_f16x2(u[2], s1), a3 = mul_f16x2(v[2], s1);
                const uint32_t b0 = mul_f16x2(u[1], s0), b1 = mul_f16x2(v[1], s0);
                const uint32_t b2 = mul_f16x2(u[3], s1), b3 = mul_f16x2(v[3], s1);
#pragma unroll
                for (int n = 0; n < C::kNT; n += 2) {
                    const uint4 f = lds128(p_at + (tb * C::kNT + n) * 256);
                    mma_f16(acc[n][0], a0, a1, a2, a3, f.x, f.y);
                    mma_f16(acc[n][1], b0, b1, b2, b3, f.x, f.y);
                    mma_f16(acc[n + 1][0], a0, a1, a2, a3, f.z, f.w);
                    mma_f16(acc[n + 1][1], b0, b1, b2, b3, f.z, f.w);
                }
            }
        }
    }
};

template <class C, class WL>
__global__ void __launch_bounds__(kThreads, C::kCtas)
    quant_decode_wide_kernel(const __grid_constant__ QuantDecodeParams qp,
                        const __grid_constant__ WL work) {
    extern __shared__ __align__(128) uint8_t base[];
    const DecodeParams& p = qp.d;
    volatile int* range = reinterpret_cast<volatile int*>(base + C::kRangeOff);
    Unit* cur = reinterpret_cast<Unit*>(base + C::kCurOff);  // [unit & 1]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, tq = lane & 3;

    uint64_t* q_bar = reinterpret_cast<uint64_t*>(base + C::kBarOff);
    if (threadIdx.x == 0) {
        mbar_init(q_bar, 1);
        fence_mbar_init();
    }
    // as a programmatic dependent: nothing in global memory before this
    grid_dependency_wait();
    // This CTA's units, from the parameter buffer or the workspace. Their range
    // and the entries go through shared memory, one thread's reading for all:
    // every warp passes the same number of barriers, whatever happens to the
    // list meanwhile.
    const int4* list = p.units;
    Unit* shared_list = reinterpret_cast<Unit*>(base + C::kListOff);
    int a = 0, b = 0;
    bool listed = false;
    if constexpr (std::is_same<WL, WorkList>::value) {
        if (list == nullptr) {
            list = work.unit;
            a = work.cta_begin[blockIdx.x];
            b = work.cta_begin[blockIdx.x + 1];
            listed = true;
        }
    }
    int4 it0 = make_int4(0, 0, 0, 0);  // the first unit, beside the range
    if (!listed) {
        const int4 r = __ldg(p.cta_rec + 2 * blockIdx.x);
        it0 = __ldg(p.cta_rec + 2 * blockIdx.x + 1);
        a = r.x;
        b = r.y;
    }
    const bool mine = (p.ws_stamp == nullptr || *p.ws_stamp == p.stamp) && a >= 0 &&
                      b <= p.n_units && a <= b;
    if (!mine) a = b = 0;
    Unit own;
    int4 own_it = make_int4(0, 0, 0, 0);
    const bool have = threadIdx.x < kListed && static_cast<int>(threadIdx.x) < b - a;
    if (have) {
        own_it = threadIdx.x == 0 && !listed ? it0 : list[a + threadIdx.x];
        own = decode_unit<false>(qp, own_it);
        shared_list[threadIdx.x] = own;
    }
    if (threadIdx.x == 0) {
        if (blockIdx.x == 0) {
            *p.last_epoch = p.epoch;
            if (p.clear_stamp != nullptr) *p.clear_stamp = 0ull;
        }
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        if (!mine) record_status(p.status, p.epoch, kDevicePlanMismatch);
        range[0] = a;
        range[1] = b;
        if (have) cur[a & 1] = own;
    }
    __syncthreads();
    const int u_begin = range[0], u_end = range[1];
    if (u_begin >= u_end) return;
    const List units{shared_list, list, u_begin};

    // The query rows of a unit (contiguous) come as one bulk copy, a unit ahead;
    // one that is not a unit of this plan has none.
    const int G = p.group;
    auto copy_query = [&](const Unit& u) {  // thread 0
        if (u.valid == 0) return;
        const uint32_t bytes = G * kHeadDim * 2;
        mbar_arrive_expect_tx(q_bar, bytes);
        bulk_load(smem_addr(base) + C::kRawOff,
                  p.q + (static_cast<size_t>(u.b) * p.num_qo_heads + u.h * G) * kHeadDim, bytes,
                  q_bar);
    };
    int q_taken = 0;
    // Waits for the copy of `u`'s rows and makes the fragments. Every thread waits.
    auto take_query = [&](const Unit& u) {
        if (u.valid == 0) return;
        const uint32_t parity = q_taken++ & 1;
        if (!mbar_wait(q_bar, parity, nullptr, p.wait_ns)) {
            record_status(p.status, p.epoch, kDeviceWaitTimeout);
            mbar_wait(q_bar, parity, nullptr, kWaitTimeoutNs);  // the copy still lands first
        }
        convert_query<C::kNT>(base + C::kRawOff, G, p.scale_log2, base + C::kQOff,
                              reinterpret_cast<float*>(base + C::kScOff));
    };
    if (threadIdx.x == 0 && u_begin < u_end) copy_query(cur[u_begin & 1]);

    const uint32_t ring = smem_addr(base);
    // this lane's offsets in a stage: where it copies to, its ldmatrix rows of K
    // (16-byte piece c + 2 is 32 bytes away in the XOR) and V, its K scales
    const int t_cp = warp * kWarpTokens + (lane >> 2);
    const uint32_t dst = t_cp * kCodeBytes + (((lane & 3) ^ ((t_cp >> 1) & 3)) << 4);
    const uint32_t sdst = (lane < 8 ? C::kKsOff : C::kVsOff) +
                          (warp * kWarpTokens + 2 * (lane & 7)) * kScaleBytes;
    const int t_k = warp * kWarpTokens + (lane & 15);
    const uint32_t k_off = t_k * kCodeBytes + (((lane >> 4) ^ ((t_k >> 1) & 3)) << 4);
    const uint32_t v_off = C::kVOff + lane * kCodeBytes + ((warp ^ ((lane >> 1) & 3)) << 4);
    const uint32_t ks_off = C::kKsOff + (warp * kWarpTokens + g) * kScaleBytes;
    Stream<C> in;
    in.u_end = u_end;
    in.unit = u_begin - 1;
    in.load_next_window(qp, units, warp, lane);  // the first unit's
    in.st = in.n_stages = 0;
    for (int i = 0; i < C::kStages - 1; ++i)
        in.issue(qp, units, ring + i * C::kSlotBytes, dst, sdst, warp, lane);
    if (have && !tables_match(p, own, own_it)) record_status(p.status, p.epoch, kDevicePlanMismatch);
    if (u_begin < u_end) take_query(cur[u_begin & 1]);
    cp_async_wait<C::kStages - 2>();  // the first stage
    __syncthreads();

    State<C> st;
    float* maxima = reinterpret_cast<float*>(base + C::kMaxOff);
    float* sums = reinterpret_cast<float*>(base + C::kSumOff);
    int slot = 0;       // of the next stage
    uint32_t flip = 0;  // which of the two weight buffers it takes
    for (int ui = u_begin; ui < u_end; ++ui) {
        const int n_stages = stages_of(cur[ui & 1]);
        int left = cur[ui & 1].valid - warp * kWarpTokens;  // tokens from this warp's next on
        // thread 0 sees to the next unit: its entry, and its query rows
        if (threadIdx.x == 0 && ui + 1 < u_end) {
            const Unit nx = units.get(qp, ui + 1);
            cur[(ui + 1) & 1] = nx;
            copy_query(nx);
            if (ui + 1 - u_begin >= kListed && !tables_match(p, nx, __ldg(list + ui + 1)))
                record_status(p.status, p.epoch, kDevicePlanMismatch);
        }
        st.init(base, lane);
        for (int s = 0; s < n_stages; ++s) {
            const uint32_t stage = ring + slot * C::kSlotBytes;
            const uint32_t p_buf = ring + C::kPOff + flip * C::kPBytes + lane * 16;
            const uint32_t t_buf = ring + C::kTOff + flip * C::kTBytes;
            const uint32_t p_mine = p_buf + warp * C::kNT * 256;
            float x[C::kNT][4], sum[C::kNT][2];
            st.scores(x, stage + k_off, stage + ks_off);
            if (left < kWarpTokens) {
#pragma unroll
                for (int n = 0; n < C::kNT; ++n) {
                    if (g >= left) x[n][0] = x[n][1] = -INFINITY;
                    if (g + 8 >= left) x[n][2] = x[n][3] = -INFINITY;
                }
            }
            // V's scales of this warp's tokens, turned to [group][token]; rows past
            // the last token may hold anything, NaN too
            if (lane < kWarpTokens) {
                uint2 vs = lds64(stage + C::kVsOff + (warp * kWarpTokens + lane) * kScaleBytes);
                if (lane >= left) vs = make_uint2(0u, 0u);
                const uint32_t at = t_buf + (warp * kWarpTokens + lane) * 2;
                sts16(at, vs.x);
                sts16(at + kStageTokens * 2, vs.x >> 16);
                sts16(at + 2 * kStageTokens * 2, vs.y);
                sts16(at + 3 * kStageTokens * 2, vs.y >> 16);
            }
            bool raise = false;
            float mx[C::kNT][2];
#pragma unroll
            for (int n = 0; n < C::kNT; ++n) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    mx[n][j] = fmaxf(x[n][j], x[n][2 + j]);
                    raise |= fmaf(mx[n][j], st.sc[n][j], st.mu[n][j]) > kPOffset + kLazy;
                }
            }
            if (s > 0) st.weights(x, sum, p_mine);
            cp_async_wait<C::kStages - 3>();  // this warp's part of the next stage
            // The barrier: the stage's weights and the next stage are there, every
            // warp is done with the stage before, and whether some maximum rises.
            const bool up = __syncthreads_or(raise) != 0;
            {
                int free = slot - 1;
                if (free < 0) free += C::kStages;
                in.issue(qp, units, ring + free * C::kSlotBytes, dst, sdst, warp, lane);
            }
            if (up || s == 0) {
#pragma unroll
                for (int n = 0; n < C::kNT; ++n) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float t = mx[n][j] * st.sc[n][j];
                        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                        if (g == 0) maxima[warp * C::kRows + n * 8 + 2 * tq + j] = t;
                    }
                }
                __syncthreads();
#pragma unroll
                for (int n = 0; n < C::kNT; ++n) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float was = kPOffset - st.mu[n][j];
                        float t = was;
#pragma unroll
                        for (int w = 0; w < kWarps; ++w)
                            t = fmaxf(t, maxima[w * C::kRows + n * 8 + 2 * tq + j]);
                        const float al = t == -INFINITY ? 1.f : fast_exp2(was - t);
                        st.mu[n][j] = kPOffset - t;
                        st.l[n][j] *= al;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            st.acc[n][i][j] *= al;
                            st.acc[n][i][2 + j] *= al;
                        }
                    }
                }
                st.weights(x, sum, p_mine);
                __syncthreads();
            }
#pragma unroll
            for (int n = 0; n < C::kNT; ++n) {
#pragma unroll
                for (int j = 0; j < 2; ++j) st.l[n][j] += sum[n][j];
            }
            st.values(stage + v_off, p_buf, t_buf + (warp * kStageTokens + 2 * tq) * 2);
            left -= kStageTokens;
            slot = slot + 1 == C::kStages ? 0 : slot + 1;
            flip ^= 1;
        }
        // ---- the unit's end: denominators over the lanes and warps; the columns
        // are whole. Meanwhile the next unit's query rows (no warp reads this
        // unit's fragments any more).
        if (n_stages == 0) __syncthreads();  // (the next unit's entry, and the sums' last readers)
#pragma unroll
        for (int n = 0; n < C::kNT; ++n) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float t = st.l[n][j];
                t += __shfl_xor_sync(0xffffffffu, t, 4);
                t += __shfl_xor_sync(0xffffffffu, t, 8);
                t += __shfl_xor_sync(0xffffffffu, t, 16);
                if (g == 0) sums[warp * C::kRows + n * 8 + 2 * tq + j] = t;
            }
        }
        const Unit u = cur[ui & 1];
        if (ui + 1 < u_end) take_query(cur[(ui + 1) & 1]);
        __syncthreads();
        if (u.valid == 0) continue;
#pragma unroll
        for (int n = 0; n < C::kNT; ++n) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = n * 8 + 2 * tq + j;
                if (r >= G) continue;
                float L = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) L += sums[w * C::kRows + r];
                const float inv = L != 0.f ? __fdividef(1.f, L) : 0.f;
                const float4 o = make_float4(st.acc[n][0][j] * inv, st.acc[n][0][2 + j] * inv,
                                             st.acc[n][1][j] * inv, st.acc[n][1][2 + j] * inv);
                const int col = warp * 32 + g * 4;
                const float lse2 = L != 0.f ? __log2f(L) - st.mu[n][j] : -INFINITY;
                const bool first = warp == 0 && g == 0;
                if (u.slot < 0) {
                    const size_t row =
                        static_cast<size_t>(u.b) * p.num_qo_heads + u.h * G + r;
                    uint2 v;
                    v.x = pack_bf16x2(o.x, o.y);
                    v.y = pack_bf16x2(o.z, o.w);
                    *reinterpret_cast<uint2*>(p.out + row * kHeadDim + col) = v;
                    if (first && p.lse != nullptr) p.lse[row] = lse2 * kLn2;
                } else {
                    // partial states are [slot][heads * G][128]
                    const size_t row = static_cast<size_t>(u.slot) * G * qp.heads + u.row0 + r;
                    *reinterpret_cast<float4*>(p.part_o + row * kHeadDim + col) = o;
                    if (first) p.part_lse[row] = lse2;
                }
            }
        }
    }
    cp_async_wait<0>();
}

template <class C, class WL>
cudaError_t ensure_smem() {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
    if (bit != 0 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(quant_decode_wide_kernel<C, WL>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

template <class C, class WL>
cudaError_t launch_ex(const QuantDecodeParams& p, const WL& w, int grid, cudaStream_t stream,
                      bool pdl) {
    const cudaError_t e = ensure_smem<C, WL>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, quant_decode_wide_kernel<C, WL>, p, w);
}

template <template <int> class C>
cudaError_t launch_ps(const QuantDecodeParams& p, const WorkList* w, int grid, cudaStream_t stream,
                      bool pdl) {
    auto go = [&](auto c) {
        using Cfg = decltype(c);
        if (w != nullptr) return launch_ex<Cfg>(p, *w, grid, stream, pdl);
        return launch_ex<Cfg>(p, NoList{0}, grid, stream, pdl);
    };
    switch (p.d.page_size) {
        case 8: return go(C<8>{});
        case 16: return go(C<16>{});
        case 32: return go(C<32>{});
        case 64: return go(C<64>{});
    }
    return cudaErrorInvalidValue;
}

template <class C>
cudaError_t occupancy(int* n) {
    const cudaError_t e = ensure_smem<C, WorkList>();
    if (e != cudaSuccess) return e;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, quant_decode_wide_kernel<C, WorkList>,
                                                         kThreads, C::kSmemBytes);
}

template <class C>
VariantShape shape() {
    return {kThreads, kStageTokens, C::kStages, C::kSmemBytes};
}

}  // namespace

// The page size changes neither the registers (capped by the launch bound) nor
// the shared memory.
VariantShape quant_wide_shape(int variant) {
    return variant == kVariantQuant16 ? shape<CfgQ16<16>>() : shape<CfgQ32<16>>();
}

cudaError_t quant_wide_occupancy(int variant, int* n) {
    return variant == kVariantQuant16 ? occupancy<CfgQ16<16>>(n) : occupancy<CfgQ32<16>>(n);
}

cudaError_t launch_decode_quant_wide(int variant, const QuantDecodeParams& p, const WorkList* w,
                                     int grid, cudaStream_t stream, bool pdl) {
    return variant == kVariantQuant16 ? launch_ps<CfgQ16>(p, w, grid, stream, pdl)
                                      : launch_ps<CfgQ32>(p, w, grid, stream, pdl);
}

}  // namespace oxd
