// window_sm100.cu -- window attention forward on the sm_100a tensor cores (bfloat16
// inputs, float32 sums and softmax, the probabilities rounded to bfloat16 as
// operands of the second product).
//
// Persistent, 512 threads a CTA, one CTA an SM.  A problem is one head and a pair of
// 128-row query tiles; its keys are the two runs of 128-key chunks that some row of
// the pair sees.  Roles: warp 12 loads keys, warp 14 queries and values (TMA), warps 13
// and 15 issue the products of tile 0 and 1, warps 0-3 and 4-7 are the softmax of tile
// 0 and 1 (one query row a thread), warps 8-11 the epilogue.  Keys go in halves of 64:
// each tile has two S buffers of 64 columns in tensor memory, so the logits of the
// next half are ready while the softmax works on this one; P overwrites S in place.
// The running maximum moves only when it grows by more than 2^8, so O is rarely
// rescaled.  Bound by the exponentials (16 a clock and SM, 2 tiles x 128 x 64 a half)
// together with the issue slots of the softmax warps, then by the products.
#include "window_tc.cuh"

namespace monarch {
namespace win {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 512;
constexpr int kSoftmaxRegs = 136, kEpilogueRegs = 128, kProducerRegs = 112;
static_assert(2 * kSoftmaxRegs + kEpilogueRegs + kProducerRegs == 4 * (65536 / kThreads),
              "the warpgroups' registers must add up to the launch's 128 per thread");

// Shared memory for a head of D columns (tiles of 128 rows).
template <int D> struct Layout {
    static constexpr uint32_t kTile = (D / 64) * kPanel;
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kK = 2 * kTile;
    static constexpr uint32_t kV = kK + 2 * kTile;
    static constexpr uint32_t kL = kV + 2 * kTile;          // row sums [parity][tile][128]
    static constexpr uint32_t kStg = kL + 2048;             // epilogue: 4 warps x 32 rows x 128 B
    static constexpr uint32_t kBar = kStg + 4 * 4096;
    static constexpr uint32_t kSmem = kBar + 512 + 1024;    // + slack to align the base
    static_assert(kSmem <= (uint32_t)kMaxSmem, "window attention shared memory");
};

struct FwdArgs {
    WinProblem p;
    int npairs;     // pairs of 128-row query tiles a head
    int nprob;      // npairs * B * H
    __nv_bfloat16 *out;
    float *lse;     // or null
    int *status;
    long long limit;
    int stall;
};

struct FwdProblem {
    int b, h, i0;
    Sequence seq;
    KeyTiles kt;    // 128-key chunks
    int nh;         // 64-key halves: two a chunk, but for a last one that nobody sees
};

// Later rows see more keys under a causal mask: the pairs go from last to first, so
// that the longest problems start first and the short ones fill the end.
__device__ __forceinline__ FwdProblem fwd_problem(const FwdArgs &a, int unit) {
    const WinProblem &p = a.p;
    FwdProblem q;
    const int bh = unit % (p.B * p.H);
    q.i0 = (a.npairs - 1 - unit / (p.B * p.H)) * 256;
    q.b = bh / p.H;
    q.h = bh % p.H;
    q.seq = sequence(p, q.b);
    q.kt = key_tiles<128>(p, q.seq, q.i0, q.i0 + 256);
    q.nh = 2 * q.kt.count();
    if (q.nh) {
        int r0, r1;
        real_rows(p, q.seq, q.i0, q.i0 + 256, r0, r1);
        const int end = q.kt.nB ? row_keys(p, q.seq, r1 - 1).hi : row_keys(p, q.seq, r1 - 1).sink;
        if (q.kt.tile(q.kt.count() - 1) * 128 + 64 >= end) q.nh--;
    }
    return q;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
tc_window_fwd_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, FwdArgs a) {
    using L = Layout<D>;
    constexpr int PN = D / 64;
    constexpr uint32_t kTile = L::kTile;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = align1024(smem_raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::kBar);
    uint64_t *q_full = bars + 0;     // [2 tiles]
    uint64_t *q_empty = bars + 2;    // [2 tiles]: the tile's last S product of a problem done
    uint64_t *k_full = bars + 4;     // [2 stages]
    uint64_t *k_empty = bars + 6;    // [2 stages], one commit from each issuer
    uint64_t *v_full = bars + 8;     // [2 stages]
    uint64_t *v_empty = bars + 10;   // [2 stages], one commit from each issuer
    uint64_t *s_full = bars + 12;    // [2 tiles][2 S buffers]
    uint64_t *p_full = bars + 16;    // [2 tiles][2 S buffers], one arrival per softmax warp
    uint64_t *o_full = bars + 20;    // [2 tiles]: the last PV product of a problem done
    uint64_t *o_free = bars + 22;    // [2 tiles], one arrival per epilogue warp
    uint64_t *l_full = bars + 24;    // [2 tiles], one arrival per softmax warp
    uint64_t *mma_done = bars + 26;
    uint64_t *stall_bar = bars + 27;   // never completed (fault injection)
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 28);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 29);
    uint64_t *pv_done = bars + 30;   // [2 tiles]: one phase per PV product
    float *lsum = reinterpret_cast<float *>(sm + L::kL);   // [2][2][128]

    const WinProblem &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nmine = a.nprob > (int)blockIdx.x
                          ? (a.nprob - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;

    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; t++) {
            mbar_init(q_full + t, 1);
            mbar_init(q_empty + t, 1);
            mbar_init(k_full + t, 1);
            mbar_init(k_empty + t, 2);
            mbar_init(v_full + t, 1);
            mbar_init(v_empty + t, 2);
            for (int b = 0; b < 2; b++) {
                mbar_init(s_full + 2 * t + b, 1);
                mbar_init(p_full + 2 * t + b, 4);
            }
            mbar_init(pv_done + t, 1);
            mbar_init(o_full + t, 1);
            mbar_init(o_free + t, 4);
            mbar_init(l_full + t, 4);
        }
        mbar_init(mma_done, 2);
        mbar_init(stall_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 13) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx w{a.limit, a.status, abort_flag};
    // Every role walks the same problems and skips those without keys (the softmax
    // warps write their zeros); pc counts the others, and so does every barrier.

    if (warp >= 12) {
        regs_dec<kProducerRegs>();
        if (warp == 12) {
            // ---------------- keys: a chunk as soon as the S products of two chunks
            // back are done
            int issued[2] = {0, 0}, jc = 0;
            bool ok = true;
            for (int pi = 0; ok && pi < nmine; pi++) {
                const FwdProblem pr = fwd_problem(a, blockIdx.x + pi * gridDim.x);
                for (int j = 0; j < (pr.nh + 1) / 2; j++, jc++) {
                    const int sk = jc & 1;
                    if (jc >= 2 && !wait_warp(k_empty + sk, ((jc >> 1) - 1) & 1, w)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        mbar_expect_tx(k_full + sk, kTile);
                        for (int pn = 0; pn < PN; pn++)
                            tma_load_4d(sm + L::kK + sk * kTile + pn * kPanel, &tmK, pn * 64,
                                        pr.kt.tile(j) * 128, pr.h / p.G, pr.b, k_full + sk);
                    }
                    issued[sk]++;
                }
            }
            if (lane == 0)   // every issued copy lands before the CTA may exit
                for (int s = 0; s < 2; s++)
                    if (issued[s] > 0)
                        wait_phase_cleanup(k_full + s, (issued[s] - 1) & 1, kCleanupPolls);
        } else if (warp == 14) {
            // ---------------- queries, then values.  Every wait points at a product
            // that the issuers reach without these loads: a tile's last S of the
            // previous problem follows that problem's values in the issue order.
            int pc = 0, issued[2] = {0, 0}, jc = 0, qloads[2] = {0, 0};
            bool ok = true;
            for (int pi = 0; ok && pi < nmine; pi++) {
                const FwdProblem pr = fwd_problem(a, blockIdx.x + pi * gridDim.x);
                if (!pr.nh) continue;
                for (int t = 0; t < 2; t++) {
                    if (pc > 0 && !wait_warp(q_empty + t, (pc - 1) & 1, w)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        mbar_expect_tx(q_full + t, kTile);
                        for (int pn = 0; pn < PN; pn++)
                            tma_load_4d(sm + L::kQ + t * kTile + pn * kPanel, &tmQ, pn * 64,
                                        pr.i0 + t * 128, pr.h, pr.b, q_full + t);
                    }
                    qloads[t]++;
                }
                if (!ok) break;
                pc++;
                for (int j = 0; j < (pr.nh + 1) / 2; j++, jc++) {
                    const int st = jc & 1;
                    if (jc >= 2 && !wait_warp(v_empty + st, ((jc >> 1) - 1) & 1, w)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        mbar_expect_tx(v_full + st, kTile);
                        for (int pn = 0; pn < PN; pn++)
                            tma_load_4d(sm + L::kV + st * kTile + pn * kPanel, &tmV, pn * 64,
                                        pr.kt.tile(j) * 128, pr.h / p.G, pr.b, v_full + st);
                    }
                    issued[st]++;
                }
            }
            if (lane == 0) {
                for (int t = 0; t < 2; t++)
                    if (qloads[t] > 0)
                        wait_phase_cleanup(q_full + t, (qloads[t] - 1) & 1, kCleanupPolls);
                for (int st = 0; st < 2; st++)
                    if (issued[st] > 0)
                        wait_phase_cleanup(v_full + st, (issued[st] - 1) & 1, kCleanupPolls);
            }
        } else {
            // ---------------- product issuers.  Half hc (over the CTA's problems) of
            // tile t uses S buffer hc & 1.  Order: S of the first two halves, then per
            // half PV(hc), S(hc + 2).  S(hc + 2) overwrites the columns that PV(hc)
            // reads as P: one thread's products execute in issue order.
            if (elect_one()) {
            const int t = warp == 13 ? 0 : 1;
            constexpr uint32_t idS = idesc_bf16(128, 64, 0, 0);
            constexpr uint32_t idO = idesc_bf16(128, D, 0, 1);
            const uint64_t dQ = smem_desc_sw128(smem_u32(sm + L::kQ + t * kTile), 16, 1024);
            const uint64_t dK = smem_desc_sw128(smem_u32(sm + L::kK), 16, 1024);
            const uint64_t dV = smem_desc_sw128(smem_u32(sm + L::kV), kPanel, 1024);
            constexpr uint32_t kTileDesc = kTile >> 4, kHalfDesc = 64 * 128 >> 4;
            const uint32_t tS = tmem + t * 128, tO = tmem + 256 + t * 128;
            bool ok = !a.stall || wait_phase(stall_bar, 0, w);
            struct Cursor {
                int pi, pc, i, hc, jc0;
                FwdProblem pr;
            };
            auto skip_empty = [&](Cursor &c) {
                while (c.pi < nmine) {
                    c.pr = fwd_problem(a, blockIdx.x + c.pi * gridDim.x);
                    if (c.pr.nh) break;
                    c.pi++;
                }
            };
            auto advance = [&](Cursor &c) {
                c.hc++;
                if (++c.i == c.pr.nh) {
                    c.i = 0;
                    c.jc0 += (c.pr.nh + 1) / 2;
                    c.pi++;
                    c.pc++;
                    skip_empty(c);
                }
            };
            auto issue_s = [&](const Cursor &c) -> bool {
                const int jc = c.jc0 + (c.i >> 1), sk = jc & 1, kh = c.i & 1, b = c.hc & 1;
                if (c.i == 0 && !wait_phase(q_full + t, c.pc & 1, w)) return false;
                if (kh == 0 && !wait_phase(k_full + sk, (jc >> 1) & 1, w)) return false;
                tc_fence_after();
                mma_head<D, 128>(tS + b * 64, dQ, dK + sk * kTileDesc + kh * kHalfDesc, idS);
                mma_commit(s_full + 2 * t + b);
                const bool last = c.i == c.pr.nh - 1;
                if (kh == 1 || last) mma_commit(k_empty + sk);
                if (last) mma_commit(q_empty + t);
                return true;
            };
            auto issue_pv = [&](const Cursor &c) -> bool {
                const int jc = c.jc0 + (c.i >> 1), st = jc & 1, kh = c.i & 1, b = c.hc & 1;
                if (kh == 0 && !wait_phase(v_full + st, (jc >> 1) & 1, w)) return false;
                if (!wait_phase(p_full + 2 * t + b, (c.hc >> 1) & 1, w)) return false;
                // the first PV of a problem overwrites O: the epilogue must have read it
                if (c.i == 0 && c.pc > 0 && !wait_phase(o_free + t, (c.pc - 1) & 1, w)) return false;
                tc_fence_after();
                mma_block64<16>(tO, tS + b * 64, dV + st * kTileDesc + kh * kHalfDesc, idO,
                             c.i > 0 ? 1u : 0u);
                mma_commit(pv_done + t);
                const bool last = c.i == c.pr.nh - 1;
                if (kh == 1 || last) mma_commit(v_empty + st);
                if (last) mma_commit(o_full + t);
                return true;
            };
            Cursor cs{0, 0, 0, 0, 0, {}};   // next S to issue
            skip_empty(cs);
            Cursor cp = cs;                 // next PV to issue
            for (int k = 0; ok && k < 2 && cs.pi < nmine; k++) {
                ok = issue_s(cs);
                advance(cs);
            }
            while (ok && cp.pi < nmine) {
                const bool more = cs.pi < nmine;
                ok = issue_pv(cp) && (!more || issue_s(cs));
                if (more) advance(cs);
                advance(cp);
            }
            mma_commit(mma_done);
            wait_phase_cleanup(mma_done, 0, kCleanupPolls);
            }
            __syncwarp();
        }
    } else if (warp >= 8) {
        // ---------------- epilogue: O / l to bfloat16 rows
        regs_dec<kEpilogueRegs>();
        const int wq = warp & 3;
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        bool ok = true;
        int pc = 0;
        for (int pi = 0; ok && pi < nmine; pi++) {
            const FwdProblem pr = fwd_problem(a, blockIdx.x + pi * gridDim.x);
            if (!pr.nh) continue;
            for (int t = 0; t < 2; t++) {
                if (!wait_warp(o_full + t, pc & 1, w) || !wait_warp(l_full + t, pc & 1, w)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float total = lsum[((pc & 1) * 2 + t) * 128 + wq * 32 + lane];
                const float inv_l = 1.f / total;
                uint32_t pk[D / 2];
#pragma unroll
                for (int c = 0; c < D / 32; c++) {
                    float o[32];
                    tmem_ld32f(tmem + lane_off + 256 + t * 128 + c * 32, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; k++)
                        pk[c * 16 + k] = total == 0.f ? 0u   // a row that sees nothing
                                                      : pack_bf16(o[2 * k] * inv_l,
                                                                  o[2 * k + 1] * inv_l);
                }
                tc_fence_before();
                mbar_arrive_warp(o_free + t);
                // the warp's 32 rows leave through shared memory, 128 bytes of a row at a
                // time, so each store instruction covers four runs of 128 bytes
                uint8_t *stg = sm + L::kStg + wq * 4096;
                const int m0 = pr.i0 + t * 128 + wq * 32;
                __nv_bfloat16 *const base = a.out + pr.b * p.o.batch + pr.h * p.o.head;
#pragma unroll
                for (int hf = 0; hf < PN; hf++) {
#pragma unroll
                    for (int c = 0; c < 8; c++)
                        *reinterpret_cast<uint4 *>(stg + lane * 128 + ((c + lane) & 7) * 16) =
                            make_uint4(pk[hf * 32 + 4 * c], pk[hf * 32 + 4 * c + 1],
                                       pk[hf * 32 + 4 * c + 2], pk[hf * 32 + 4 * c + 3]);
                    __syncwarp();
#pragma unroll
                    for (int rr = 0; rr < 8; rr++) {
                        const int row = rr * 4 + (lane >> 3), c = lane & 7;
                        const uint4 val =
                            *reinterpret_cast<const uint4 *>(stg + row * 128 + ((c + row) & 7) * 16);
                        // (d = 32 runs with D = 64: the columns past d are padding)
                        if (m0 + row < p.Nq && hf * 64 + c * 8 < p.d)
                            *reinterpret_cast<uint4 *>(base + (int64_t)(m0 + row) * p.o.token +
                                                       hf * 64 + c * 8) = val;
                    }
                    __syncwarp();
                }
            }
            pc++;
        }
    } else {
        // ---------------- softmax of tile t: one query row a thread
        regs_inc<kSoftmaxRegs>();
        const int t = warp >> 2, wq = warp & 3;
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        const uint32_t tS0 = tmem + lane_off + t * 128;
        const uint32_t tO = tmem + lane_off + 256 + t * 128;
        const float c1 = p.scale_log2;
        const uint64_t c2 = f2_pack(c1, c1);
        bool ok = true;
        int pc = 0, hc = 0, jc0 = 0;
        for (int pi = 0; ok && pi < nmine; pi++) {
            const FwdProblem pr = fwd_problem(a, blockIdx.x + pi * gridDim.x);
            const int m = pr.i0 + t * 128 + wq * 32 + lane;
            if (!pr.nh) {   // no row of the pair sees a key
                if (m < p.Nq) {
                    uint4 *row = reinterpret_cast<uint4 *>(a.out + pr.b * p.o.batch +
                                                           pr.h * p.o.head + (int64_t)m * p.o.token);
                    for (int x = 0; x < p.d / 8; x++) row[x] = make_uint4(0, 0, 0, 0);
                    if (a.lse) a.lse[((int64_t)pr.b * p.H + pr.h) * p.Nq + m] = -INFINITY;
                }
                continue;
            }
            const RowKeys rk = row_keys(p, pr.seq, m);
            float m_run = -INFINITY, l_run = 0.f;
            for (int i = 0; i < pr.nh; i++, hc++) {
                const int b = hc & 1;
                if (!wait_warp(s_full + 2 * t + b, (hc >> 1) & 1, w)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t tS = tS0 + b * 64;
                const int j0 = pr.kt.tile(i >> 1) * 128 + (i & 1) * 64;
                float x[64];
                tmem_ld32f(tS, &x[0]);
                tmem_ld32f(tS + 32, &x[32]);
                tmem_wait_ld();
                const bool all = j0 + 64 <= rk.hi && (j0 >= rk.lo || j0 + 64 <= rk.sink);
                if (!__all_sync(0xffffffffu, all)) {
                    // bit k: the row sees key j0 + k
                    auto below = [](int n) -> uint64_t {
                        return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
                    };
                    const uint64_t see = below(rk.hi - j0) &
                                         (~below(rk.lo - j0) | below(rk.sink - j0));
                    const uint32_t see0 = (uint32_t)see, see1 = (uint32_t)(see >> 32);
#pragma unroll
                    for (int k = 0; k < 32; k++) {
                        x[k] = (see0 >> k) & 1 ? x[k] : -INFINITY;
                        x[k + 32] = (see1 >> k) & 1 ? x[k + 32] : -INFINITY;
                    }
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < 32; k++) mx4[k & 3] = fmax3(mx4[k & 3], x[2 * k], x[2 * k + 1]);
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
                float alpha = 1.f;
                bool rescale = false;
                if ((mx - m_run) * c1 > 8.f) {   // (false for a row without keys so far)
                    alpha = fast_exp2((m_run - mx) * c1);
                    m_run = mx;
                    rescale = true;
                }
                const float mm = m_run == -INFINITY ? 0.f : m_run * c1;
                const uint64_t nmc2 = f2_pack(-mm, -mm);
                uint64_t sum2[4] = {0, 0, 0, 0};
                uint32_t pk[32];
#pragma unroll
                for (int k = 0; k < 32; k++) {
                    const uint64_t d2 = f2_fma(f2_pack(x[2 * k], x[2 * k + 1]), c2, nmc2);
                    float lo, hi;
                    f2_unpack(d2, lo, hi);
                    const uint64_t e2 = f2_pack(fast_exp2(lo), fast_exp2(hi));
                    sum2[k & 3] = f2_add(sum2[k & 3], e2);
                    float p0, p1;
                    f2_unpack(e2, p0, p1);
                    pk[k] = pack_bf16(p0, p1);
                }
                tmem_st32(tS, pk);   // P over the first 32 columns of the buffer
                float s0, s1;
                f2_unpack(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), s0, s1);
                l_run = l_run * alpha + (s0 + s1);
                if (j0 + 64 > pr.seq.len) {
                    // values past the sequence may hold anything, and 0 * NaN is NaN: they
                    // become zeros before this half's PV (both tiles write the same zeros)
                    const int jc = jc0 + (i >> 1), st = jc & 1;
                    if (!wait_warp(v_full + st, (jc >> 1) & 1, w)) {
                        ok = false;
                        break;
                    }
                    zero_rows(sm + L::kV + st * kTile + (i & 1) * 64 * 128,
                              max(0, pr.seq.len - j0), 64, PN, kPanel, wq * 32 + lane, 128);
                    fence_proxy_async_smem();
                }
                if (i > 0 && __any_sync(0xffffffffu, rescale)) {
                    // O holds the products up to the previous half once that PV is done
                    if (!wait_warp(pv_done + t, (hc - 1) & 1, w)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < D / 32; c++) {
                        float o[32];
                        tmem_ld32f(tO + c * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; k++) o[k] *= alpha;
                        tmem_st32f(tO + c * 32, o);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive_warp(p_full + 2 * t + b);
            }
            if (!ok) break;
            jc0 += (pr.nh + 1) / 2;
            if (a.lse && m < p.Nq)
                a.lse[((int64_t)pr.b * p.H + pr.h) * p.Nq + m] =
                    l_run == 0.f ? -INFINITY : (m_run * c1 + log2f(l_run)) * kLn2;
            // the row sums for the epilogue, once it has taken those of the last problem
            if (pc > 0 && !wait_warp(o_free + t, (pc - 1) & 1, w)) break;
            lsum[((pc & 1) * 2 + t) * 128 + wq * 32 + lane] = l_run;
            mbar_arrive_warp(l_full + t);
            pc++;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D>
cudaError_t launch(const WinProblem &p, const void *q, const void *k, const void *v, FwdArgs a,
                   cudaStream_t stream) {
    CUtensorMap mq, mk, mv;
    if (!map_tokens(&mq, q, p.q, p.B, p.H, p.Nq, p.d, 128) ||
        !map_tokens(&mk, k, p.k, p.B, p.Hkv, p.Nk, p.d, 128) ||
        !map_tokens(&mv, v, p.v, p.B, p.Hkv, p.Nk, p.d, 128))
        return cudaErrorInvalidValue;
    cudaError_t e = tcs::set_smem(tc_window_fwd_kernel<D>, Layout<D>::kSmem);
    if (e != cudaSuccess) return e;
    const int grid = min(a.nprob, tcs::sm_count());
    tc_window_fwd_kernel<D><<<grid, kThreads, Layout<D>::kSmem, stream>>>(mq, mk, mv, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t tc_forward(const WinProblem &p, const void *q, const void *k, const void *v, void *out,
                       float *lse, int *status, long long limit, cudaStream_t stream) {
    FwdArgs a;
    a.p = p;
    a.npairs = (p.Nq + 255) / 256;
    a.nprob = a.npairs * p.B * p.H;
    a.out = (__nv_bfloat16 *)out;
    a.lse = lse;
    a.status = status;
    a.limit = limit;
    a.stall = device_inject_stall();
    return p.d == 128 ? launch<128>(p, q, k, v, a, stream) : launch<64>(p, q, k, v, a, stream);
}

}  // namespace win
}  // namespace monarch
