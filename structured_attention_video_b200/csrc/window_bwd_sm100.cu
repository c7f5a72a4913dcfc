// window_bwd_sm100.cu -- backward of the window attention on the sm_100a tensor cores
// (bfloat16 inputs and gradients, float32 sums; P and dS rounded to bfloat16 as
// operands of the accumulating products, from 32-bit values).
//
//   P = exp2(scale_log2 S - lse log2(e)),  dS = P (dO V^T - delta),
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K.
//
// Two kernels, so that every gradient is summed by one CTA in a fixed order (no
// atomics) at the price of forming S and dO V^T twice (7 products instead of 5):
//   tc_window_dkv_kernel  128 keys of one key head against the 128-query tiles of
//                         every head of its group that see them;
//   tc_window_dq_kernel   128 queries of one head against their 128-key tiles.
// 384 threads a CTA, one CTA an SM: warps 0-7 the elementwise work, warp 8 loads
// (TMA), warp 9 issues the products, warp 10 stages lse and delta.
//
// The streamed side goes in blocks of 64 rows (queries in dkv, keys in dq).  Blocks u
// with u % 2 = h belong to warps 4 h .. 4 h + 3 (thread = tensor-memory lane = row of the
// fixed tile) and to half h of the tensor-memory columns, so the two groups work on
// different blocks at different times and the tensor pipe has the products of one
// while the other computes.  Order of the products (fixed, so the sums are too):
//   dkv:  dV(u) S(u+2) after P(u);  dK(u) dP(u+2) after dS(u)
//   dq:   dP(u+2) dQ(u) S(u+3) after dS(u)   (S has four buffers)
// P overwrites S and dS overwrites dP (S in dq) in tensor memory; a later product into
// the same columns follows in issue order.
// The blocks go through two rings of their own, as many as shared memory holds.  A
// block is needed about a block's work after its predecessor, and a load takes about as
// long as a block (16 KB a tensor): with two stages of 128 rows the tensor pipe
// waited for loads and a 128 x 128 tile took 5100 clocks in dkv and 3460 in dq.
//
// delta comes from out as the forward rounded it, an error of 2^-8 |dO.O| at most.  A
// row of n keys of like weight has |O| of about n^(-1/2) |v|, so against dP it matters
// for few keys only.  Query tiles of up to kExactBlocks key blocks therefore first walk
// their keys once for delta = sum P dP from the same products that form dS, and the dq
// kernel runs first to hand it to the dk/dv kernel.  (Two padded causal
// sequences of 1023 and 681 tokens, d = 64: dq is 2.6e-3 from 64 bits without it.)
// Bound by the tensor pipe: 4 (3) products of 128 x 128 x d a tile against 16384
// exponentials at 16 a clock.
#include "window_tc.cuh"

namespace monarch {
namespace win {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 384;
constexpr int kExactBlocks = 6;

// Shared memory: two fixed tiles of 128 rows, two rings of 64-row blocks, and per slot of
// the first ring -lse and -delta of its 64 queries (dkv).
template <int D> struct BwdLayout {
    static constexpr uint32_t kTile = (D / 64) * kPanel;
    static constexpr uint32_t kBlock = kTile / 2;             // panels of 64 rows
    static constexpr uint32_t kBlockPanel = 64 * 128;
    static constexpr int kBlocks = 10;
    static constexpr uint32_t kFix = 0;                       // K, V (dkv) or Q, dO (dq)
    static constexpr uint32_t kRing = 2 * kTile;
    static constexpr uint32_t kStats = kRing + kBlocks * kBlock;
    static constexpr uint32_t kBar = kStats + 5 * 512;
    static constexpr uint32_t kSmem = kBar + 512;   // the base is 1024-aligned (checked)
    static_assert(kSmem <= (uint32_t)kMaxSmem, "window backward shared memory");
};

struct BwdArgs {
    WinProblem p;
    WinGrads g;
    const float *lse;
    float *delta;   // of the rounded out; rows of few keys are written again (dq kernel)
    __nv_bfloat16 *dq, *dk, *dv;
    int *status;
    long long limit;
    int stall;
};

// 32-bit pieces of a 64-bit mask: bit k says whether element first + k of [lo, hi)
// counts.
__device__ __forceinline__ uint64_t below(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// 64 columns of an accumulator row to bfloat16 in global memory (columns below d).
template <int N>
__device__ __forceinline__ void store_row(uint32_t taddr, __nv_bfloat16 *dst, float scale, int d,
                                          bool real) {
#pragma unroll 1
    for (int c = 0; c < N; c += 32) {
        float o[32];
        tmem_ld32f(taddr + c, o);
        tmem_wait_ld();
        if (!real || c >= d) continue;
#pragma unroll
        for (int e = 0; e < 4; e++)
            *reinterpret_cast<uint4 *>(dst + c + 8 * e) =
                make_uint4(pack_bf16(o[8 * e] * scale, o[8 * e + 1] * scale),
                           pack_bf16(o[8 * e + 2] * scale, o[8 * e + 3] * scale),
                           pack_bf16(o[8 * e + 4] * scale, o[8 * e + 5] * scale),
                           pack_bf16(o[8 * e + 6] * scale, o[8 * e + 7] * scale));
    }
}
__device__ __forceinline__ void zero_row(__nv_bfloat16 *dst, int n) {
    for (int c = 0; c < n; c += 8) *reinterpret_cast<uint4 *>(dst + c) = make_uint4(0, 0, 0, 0);
}

// P of 64 columns: x = exp2(c x + nl[column]), masked by `see`.  nl in shared memory.
__device__ __forceinline__ void probabilities(float (&x)[64], float c, const float *nl,
                                              bool all, uint64_t see) {
    const uint64_t c2 = f2_pack(c, c);
#pragma unroll
    for (int k = 0; k < 64; k += 4) {
        const ulonglong2 n2 = *reinterpret_cast<const ulonglong2 *>(nl + k);
        const uint64_t a = f2_fma(f2_pack(x[k], x[k + 1]), c2, n2.x);
        const uint64_t b = f2_fma(f2_pack(x[k + 2], x[k + 3]), c2, n2.y);
        f2_unpack(a, x[k], x[k + 1]);
        f2_unpack(b, x[k + 2], x[k + 3]);
#pragma unroll
        for (int e = 0; e < 4; e++) x[k + e] = fast_exp2(x[k + e]);
    }
    if (!all) {
        const uint32_t s0 = (uint32_t)see, s1 = (uint32_t)(see >> 32);
#pragma unroll
        for (int k = 0; k < 32; k++) {
            x[k] = (s0 >> k) & 1 ? x[k] : 0.f;
            x[k + 32] = (s1 >> k) & 1 ? x[k + 32] : 0.f;
        }
    }
}

// A position in a ring of N blocks: slot and phase of its barriers, without divisions
// (the issuing thread has nothing to hide their latency behind).
template <int N> struct Slot {
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next() {
        if (++s == N) s = 0, ph ^= 1;
    }
};

// Barriers of one CTA.  N1, N2: blocks of the two rings; NS: S buffers.
template <int N1, int N2, int NS> struct Bars {
    uint64_t fix_full;                  // the fixed tiles
    uint64_t full1[N1], empty1[N1];     // Q (dkv) or K (dq)
    uint64_t full2[N2], empty2[N2];     // dO or V
    uint64_t stats_full[N1];            // dkv
    uint64_t s_full[NS];                // S in tensor memory
    uint64_t dp_full[2];
    uint64_t p_full[2], ds_full[2];     // one arrival a warp of the half
    uint64_t delta_bar;                 // the halves' parts of delta (dq), once
    uint64_t acc_full;                  // the last products
    uint64_t stall_bar;                 // never completed (fault injection)
    uint32_t tmem_slot;
    int abort_flag;

    __device__ __forceinline__ void init() {
        mbar_init(&fix_full, 1);
        for (int i = 0; i < N1; i++) {
            mbar_init(full1 + i, 1);
            mbar_init(empty1 + i, 1);
            mbar_init(stats_full + i, 1);
        }
        for (int i = 0; i < N2; i++) {
            mbar_init(full2 + i, 1);
            mbar_init(empty2 + i, 1);
        }
        for (int i = 0; i < NS; i++) mbar_init(s_full + i, 1);
        for (int i = 0; i < 2; i++) {
            mbar_init(dp_full + i, 1);
            mbar_init(p_full + i, 4);
            mbar_init(ds_full + i, 4);
        }
        mbar_init(&delta_bar, 8);
        mbar_init(&acc_full, 1);
        mbar_init(&stall_bar, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    // Every issued copy lands before the CTA may exit (an aborted CTA may not have
    // waited for the last ones).
    __device__ __forceinline__ void drain(int issued1, int issued2) {
        wait_phase_cleanup(&fix_full, 0, kCleanupPolls);
        for (int u = max(0, issued1 - N1); u < issued1; u++)
            wait_phase_cleanup(full1 + u % N1, (u / N1) & 1, kCleanupPolls);
        for (int u = max(0, issued2 - N2); u < issued2; u++)
            wait_phase_cleanup(full2 + u % N2, (u / N2) & 1, kCleanupPolls);
    }
};

// One CTA's loads: the fixed tiles, then the blocks of both rings in the order in which
// the products need them.  coords(u, h, row): head and first row of block u.
template <int D, typename B, int N1, int N2, typename Coords>
__device__ __forceinline__ void load_all(uint8_t *sm, B *bar, const CUtensorMap *fix_a,
                                         const CUtensorMap *fix_b, int fix_row, int fix_head,
                                         const CUtensorMap *ring1, const CUtensorMap *ring2, int b,
                                         int n, const Coords &coords, const WaitCtx &w, int lane) {
    using L = BwdLayout<D>;
    constexpr int PN = D / 64;
    if (lane == 0) {
        mbar_expect_tx(&bar->fix_full, 2 * L::kTile);
        for (int pn = 0; pn < PN; pn++) {
            tma_load_4d(sm + L::kFix + pn * kPanel, fix_a, pn * 64, fix_row, fix_head, b,
                        &bar->fix_full);
            tma_load_4d(sm + L::kFix + L::kTile + pn * kPanel, fix_b, pn * 64, fix_row, fix_head, b,
                        &bar->fix_full);
        }
    }
    int issued1 = 0, issued2 = 0;
    Slot<N1> r1;
    Slot<N2> r2;
    for (int u = 0; u < n; u++) {
        int h, row;
        coords(u, h, row);
        if (u >= N1 && !wait_warp(bar->empty1 + r1.s, r1.ph ^ 1, w)) break;
        if (lane == 0) {
            uint8_t *dst = sm + L::kRing + r1.s * L::kBlock;
            mbar_expect_tx(bar->full1 + r1.s, L::kBlock);
            for (int pn = 0; pn < PN; pn++)
                tma_load_4d(dst + pn * L::kBlockPanel, ring1, pn * 64, row, h, b, bar->full1 + r1.s);
        }
        issued1++;
        r1.next();
        if (u >= N2 && !wait_warp(bar->empty2 + r2.s, r2.ph ^ 1, w)) break;
        if (lane == 0) {
            uint8_t *dst = sm + L::kRing + (N1 + r2.s) * L::kBlock;
            mbar_expect_tx(bar->full2 + r2.s, L::kBlock);
            for (int pn = 0; pn < PN; pn++)
                tma_load_4d(dst + pn * L::kBlockPanel, ring2, pn * 64, row, h, b, bar->full2 + r2.s);
        }
        issued2++;
        r2.next();
    }
    if (lane == 0) bar->drain(issued1, issued2);
}

// The SW128 tiles need a 1024-byte aligned base; the layout leaves no room to align by
// hand, so a misaligned base is reported, not worked around.
__device__ __forceinline__ bool base_aligned(const uint8_t *sm, int *status) {
    if ((smem_u32(sm) & 1023u) == 0) return true;
    if (threadIdx.x == 0) record_status(status, MONARCH_ERR_CUDA);
    return false;
}

// ---------------------------------------------------------------- dk, dv
// Tensor memory, half h: S^T at 64 h (P^T over its first 32 columns), dP^T at 128 + 64 h
// (dS^T over it); dV at 256, dK at 384.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
tc_window_dkv_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmDo, BwdArgs a) {
    using L = BwdLayout<D>;
    constexpr int PN = D / 64, N1 = 5, N2 = 5;
    static_assert(N1 + N2 == L::kBlocks, "ring slots");
    using B = Bars<N1, N2, 2>;
    static_assert(sizeof(B) <= 512, "barriers");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = smem_raw;
    if (!base_aligned(sm, a.status)) return;
    B *bar = reinterpret_cast<B *>(sm + L::kBar);
    float *stats = reinterpret_cast<float *>(sm + L::kStats);   // [slot][-lse | -delta][64]
    const WinProblem &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // (the first key tiles first: they are seen by the most queries under a causal mask)
    const int unit = blockIdx.x % (p.B * p.Hkv), hk = unit % p.Hkv, b = unit / p.Hkv;
    const int j0 = blockIdx.x / (p.B * p.Hkv) * 128;
    const Sequence seq = sequence(p, b);
    int first, last;
    query_rows(p, seq, j0, j0 + 128, first, last);
    const int t0 = first / 64, nt = last > first ? (last + 63) / 64 - t0 : 0;
    const int n = nt * p.G;   // query blocks over the group's heads

    if (n == 0) {             // no query sees these keys (the same for the whole CTA)
        const int j = j0 + threadIdx.x;
        if (threadIdx.x < 128 && j < p.Nk) {
            zero_row(a.dk + b * a.g.dk.batch + hk * a.g.dk.head + (int64_t)j * a.g.dk.token, p.d);
            zero_row(a.dv + b * a.g.dv.batch + hk * a.g.dv.head + (int64_t)j * a.g.dv.token, p.d);
        }
        return;
    }
    if (threadIdx.x == 0) bar->init();
    if (warp == 9) tmem_alloc(&bar->tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem_slot;
    const WaitCtx w{a.limit, a.status, &bar->abort_flag};
    auto coords = [&](int u, int &h, int &row) {
        h = hk * p.G + u / nt;
        row = (t0 + u % nt) * 64;
    };

    if (warp == 8) {
        load_all<D, B, N1, N2>(sm, bar, &tmK, &tmV, j0, hk, &tmQ, &tmDo, b, n, coords, w, lane);
    } else if (warp == 9) {
        if (elect_one()) {
        // ---------------- products
        constexpr uint32_t idS = idesc_bf16(128, 64, 0, 0), idO = idesc_bf16(128, D, 0, 1);
        constexpr uint32_t kBlockDesc = L::kBlock >> 4;
        const uint32_t ring = smem_u32(sm + L::kRing);
        const uint64_t dK = smem_desc_sw128(smem_u32(sm + L::kFix), 16, 1024);
        const uint64_t dV = smem_desc_sw128(smem_u32(sm + L::kFix + L::kTile), 16, 1024);
        const uint64_t dQ = smem_desc_sw128(ring, 16, 1024);
        const uint64_t dO = smem_desc_sw128(ring + N1 * L::kBlock, 16, 1024);
        const uint64_t dQt = smem_desc_sw128(ring, L::kBlockPanel, 1024);
        const uint64_t dOt = smem_desc_sw128(ring + N1 * L::kBlock, L::kBlockPanel, 1024);
        Slot<N1> next_s, cur_q;    // of the next S; of block u
        Slot<N2> next_dp, cur_do;
        auto issue_s = [&](int h) -> bool {
            if (!spin_phase(bar->full1 + next_s.s, next_s.ph, w)) return false;
            tc_fence_after();
            mma_head<D, 64>(tmem + 64 * h, dK, dQ + next_s.s * kBlockDesc, idS);
            mma_commit(bar->s_full + h);
            next_s.next();
            return true;
        };
        auto issue_dp = [&](int h) -> bool {
            if (!spin_phase(bar->full2 + next_dp.s, next_dp.ph, w)) return false;
            tc_fence_after();
            mma_head<D, 64>(tmem + 128 + 64 * h, dV, dO + next_dp.s * kBlockDesc, idS);
            mma_commit(bar->dp_full + h);
            next_dp.next();
            return true;
        };
        bool ok = (!a.stall || spin_phase(&bar->stall_bar, 0, w)) && spin_phase(&bar->fix_full, 0, w);
        for (int u = 0; ok && u < 2 && u < n; u++) ok = issue_s(u) && issue_dp(u);
        for (int u = 0; ok && u < n; u++) {
            const int h = u & 1, ph = (u >> 1) & 1;
            if (!(ok = spin_phase(bar->p_full + h, ph, w))) break;
            tc_fence_after();
            mma_block64(tmem + 256, tmem + 64 * h, dOt + cur_do.s * kBlockDesc, idO, u > 0 ? 1u : 0u);
            mma_commit(bar->empty2 + cur_do.s);
            cur_do.next();
            if (u + 2 < n && !(ok = issue_s(h))) break;
            if (!(ok = spin_phase(bar->ds_full + h, ph, w))) break;
            tc_fence_after();
            mma_block64(tmem + 384, tmem + 128 + 64 * h, dQt + cur_q.s * kBlockDesc, idO,
                        u > 0 ? 1u : 0u);
            mma_commit(bar->empty1 + cur_q.s);
            cur_q.next();
            if (u + 2 < n) ok = issue_dp(h);
        }
        mma_commit(&bar->acc_full);
        wait_phase_cleanup(&bar->acc_full, 0, kCleanupPolls);
        }
        __syncwarp();
    } else if (warp == 10) {
        // ---------------- lse (in log2 units) and delta of each block's queries, negated
        for (int u = 0; u < n; u++) {
            if (u >= N1 && !wait_warp(bar->empty1 + u % N1, (u / N1 - 1) & 1, w)) break;
            int h, i0;
            coords(u, h, i0);
            const int64_t row = ((int64_t)b * p.H + h) * p.Nq;
            float *dst = stats + u % N1 * 128;
#pragma unroll
            for (int x = lane; x < 64; x += 32) {
                const bool in = i0 + x < p.Nq;
                dst[x] = in ? -a.lse[row + i0 + x] * kLog2e : 0.f;
                dst[64 + x] = in ? -a.delta[row + i0 + x] : 0.f;
            }
            mbar_arrive_warp(bar->stats_full + u % N1);
        }
    } else if (warp < 8) {
        // ---------------- elementwise: key row j, the queries of the half's blocks
        const int half = warp >> 2, row = (warp & 3) * 32 + lane, j = j0 + row;
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 64 * half;
        int ilo, ihi, rfirst, rlast;
        query_rows(p, seq, j, j + 1, ilo, ihi);   // the queries that see this key
        real_rows(p, seq, 0, p.Nq, rfirst, rlast);
        bool ok = true;
        for (int u = half; u < n; u += 2) {
            const int ph = (u >> 1) & 1, s1 = u % N1, s2 = u % N2, c0 = (t0 + u % nt) * 64;
            const float *nl = stats + s1 * 128, *nd = nl + 64;
            if (!(ok = wait_warp(bar->s_full + half, ph, w) &&
                       wait_warp(bar->stats_full + s1, (u / N1) & 1, w)))
                break;
            tc_fence_after();
            float x[64];
            tmem_ld32f(tl, &x[0]);
            tmem_ld32f(tl + 32, &x[32]);
            tmem_wait_ld();
            const bool all = __all_sync(0xffffffffu, c0 >= ilo && c0 + 64 <= ihi);
            const uint64_t see = below(ihi - c0) & ~below(ilo - c0);
            probabilities(x, p.scale_log2, nl, all, see);
            uint32_t pk[32];
#pragma unroll
            for (int k = 0; k < 32; k++) pk[k] = pack_bf16(x[2 * k], x[2 * k + 1]);
            tmem_st32(tl, pk);
            if (c0 < rfirst || (rlast < p.Nq && c0 + 64 > rlast)) {
                // rows that are not real may hold anything, and 0 * NaN is NaN: they become
                // zeros before the products over the queries
                if (!(ok = wait_warp(bar->full2 + s2, (u / N2) & 1, w))) break;
                const int za = min(max(rfirst - c0, 0), 64), zb = min(max(rlast - c0, 0), 64);
                for (int x2 = 0; x2 < 2; x2++) {
                    uint8_t *blk = sm + L::kRing + (x2 ? N1 + s2 : s1) * L::kBlock;
                    zero_rows(blk, 0, za, PN, L::kBlockPanel, row, 128);
                    zero_rows(blk, zb, 64, PN, L::kBlockPanel, row, 128);
                }
                fence_proxy_async_smem();
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive_warp(bar->p_full + half);
            if (!(ok = wait_warp(bar->dp_full + half, ph, w))) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
                float y[32];
                tmem_ld32f(tl + 128 + c, y);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    const ulonglong2 d2 = *reinterpret_cast<const ulonglong2 *>(nd + c + k);
                    const uint64_t e = f2_mul(f2_add(f2_pack(y[k], y[k + 1]), d2.x),
                                              f2_pack(x[c + k], x[c + k + 1]));
                    const uint64_t f = f2_mul(f2_add(f2_pack(y[k + 2], y[k + 3]), d2.y),
                                              f2_pack(x[c + k + 2], x[c + k + 3]));
                    f2_unpack(e, y[k], y[k + 1]);
                    f2_unpack(f, y[k + 2], y[k + 3]);
                }
                if (!all) {
                    const uint32_t s = (uint32_t)(see >> c);
#pragma unroll
                    for (int k = 0; k < 32; k++) y[k] = (s >> k) & 1 ? y[k] : 0.f;
                }
#pragma unroll
                for (int k = 0; k < 16; k++) pk[c / 2 + k] = pack_bf16(y[2 * k], y[2 * k + 1]);
            }
            tmem_st32(tl + 128, pk);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive_warp(bar->ds_full + half);
        }
        if (ok && wait_warp(&bar->acc_full, 0, w)) {
            tc_fence_after();
            const uint32_t ta = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * (D / 2);
            const int64_t x = half * (D / 2);
            const bool real = j < p.Nk;
            store_row<D / 2>(ta + 256,
                             a.dv + b * a.g.dv.batch + hk * a.g.dv.head + j * a.g.dv.token + x, 1.f,
                             p.d - (int)x, real);
            store_row<D / 2>(ta + 384,
                             a.dk + b * a.g.dk.batch + hk * a.g.dk.head + j * a.g.dk.token + x,
                             p.scale, p.d - (int)x, real);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- dq
// Tensor memory: S of block u at 64 (u % 4) (dS over its first 32 columns), dP of half h
// at 256 + 64 h, dQ at 384.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
tc_window_dq_kernel(const __grid_constant__ CUtensorMap tmQ,
                    const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ CUtensorMap tmDo, BwdArgs a) {
    using L = BwdLayout<D>;
    // a key block stays from S(u) to dQ(u), three blocks; a value block for dP(u) alone
    constexpr int PN = D / 64, N1 = 6, N2 = 4;
    static_assert(N1 + N2 == L::kBlocks, "ring slots");
    using B = Bars<N1, N2, 4>;
    static_assert(sizeof(B) <= 512, "barriers");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = smem_raw;
    if (!base_aligned(sm, a.status)) return;
    B *bar = reinterpret_cast<B *>(sm + L::kBar);
    float *half_delta = reinterpret_cast<float *>(sm + L::kStats);   // [2 halves][128]
    const WinProblem &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the last tiles first: they see the most keys under a causal mask
    const int unit = blockIdx.x % (p.B * p.H), h = unit % p.H, b = unit / p.H;
    const int i0 = ((int)gridDim.x - 1 - (int)blockIdx.x) / (p.B * p.H) * 128;
    const Sequence seq = sequence(p, b);
    const KeyTiles kt = key_tiles<64>(p, seq, i0, i0 + 128);
    const int nt = kt.count();
    // the first n - nt blocks only sum delta
    const int n = nt <= kExactBlocks ? 2 * nt : nt;
    __nv_bfloat16 *const dq = a.dq + b * a.g.dq.batch + h * a.g.dq.head;

    if (n == 0) {
        const int i = i0 + threadIdx.x;
        if (threadIdx.x < 128 && i < p.Nq) zero_row(dq + (int64_t)i * a.g.dq.token, p.d);
        return;
    }
    if (threadIdx.x == 0) bar->init();
    if (warp == 9) tmem_alloc(&bar->tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem_slot;
    const WaitCtx w{a.limit, a.status, &bar->abort_flag};

    if (warp == 8) {
        auto coords = [&](int u, int &head, int &row) {
            head = h / p.G;
            row = kt.tile(u % nt) * 64;
        };
        load_all<D, B, N1, N2>(sm, bar, &tmQ, &tmDo, i0, h, &tmK, &tmV, b, n, coords, w, lane);
    } else if (warp == 9) {
        if (elect_one()) {
        constexpr uint32_t idS = idesc_bf16(128, 64, 0, 0), idO = idesc_bf16(128, D, 0, 1);
        constexpr uint32_t kBlockDesc = L::kBlock >> 4;
        const uint32_t ring = smem_u32(sm + L::kRing);
        const uint64_t dQ = smem_desc_sw128(smem_u32(sm + L::kFix), 16, 1024);
        const uint64_t dO = smem_desc_sw128(smem_u32(sm + L::kFix + L::kTile), 16, 1024);
        const uint64_t dK = smem_desc_sw128(ring, 16, 1024);
        const uint64_t dV = smem_desc_sw128(ring + N1 * L::kBlock, 16, 1024);
        const uint64_t dKt = smem_desc_sw128(ring, L::kBlockPanel, 1024);
        Slot<N1> next_s, cur_k;    // of the next S; of block u
        Slot<N2> next_dp;
        auto issue_s = [&](int u) -> bool {
            if (!spin_phase(bar->full1 + next_s.s, next_s.ph, w)) return false;
            tc_fence_after();
            mma_head<D, 64>(tmem + 64 * (u & 3), dQ, dK + next_s.s * kBlockDesc, idS);
            mma_commit(bar->s_full + (u & 3));
            next_s.next();
            return true;
        };
        auto issue_dp = [&](int u) -> bool {
            if (!spin_phase(bar->full2 + next_dp.s, next_dp.ph, w)) return false;
            tc_fence_after();
            mma_head<D, 64>(tmem + 256 + 64 * (u & 1), dO, dV + next_dp.s * kBlockDesc, idS);
            mma_commit(bar->dp_full + (u & 1));
            mma_commit(bar->empty2 + next_dp.s);
            next_dp.next();
            return true;
        };
        bool ok = (!a.stall || spin_phase(&bar->stall_bar, 0, w)) && spin_phase(&bar->fix_full, 0, w);
        for (int u = 0; ok && u < 2 && u < n; u++) ok = issue_s(u) && issue_dp(u);
        if (ok && n > 2) ok = issue_s(2);
        for (int u = 0; ok && u < n; u++) {
            // dS(u) is written: the half's dP columns have been read too
            if (!(ok = spin_phase(bar->ds_full + (u & 1), (u >> 1) & 1, w))) break;
            if (u + 2 < n && !(ok = issue_dp(u))) break;   // of block u + 2
            tc_fence_after();
            if (u >= n - nt)
                mma_block64(tmem + 384, tmem + 64 * (u & 3), dKt + cur_k.s * kBlockDesc, idO,
                            u > n - nt ? 1u : 0u);
            mma_commit(bar->empty1 + cur_k.s);
            cur_k.next();
            if (u + 3 < n) ok = issue_s(u + 3);
        }
        mma_commit(&bar->acc_full);
        wait_phase_cleanup(&bar->acc_full, 0, kCleanupPolls);
        }
        __syncwarp();
    } else if (warp < 8) {
        const int half = warp >> 2, row = (warp & 3) * 32 + lane, i = i0 + row;
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const RowKeys rk = row_keys(p, seq, i);
        const int64_t at = ((int64_t)b * p.H + h) * p.Nq + i;
        const bool real = rk.hi > 0;
        const float nl = real ? -a.lse[at] * kLog2e : 0.f;
        float nd = real && n == nt ? -a.delta[at] : 0.f;
        const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2), nl2 = f2_pack(nl, nl);
        bool ok = true, summed = n == nt;
        // (a group without a block of its own still joins delta)
        auto join_delta = [&]() -> bool {
            half_delta[half * 128 + row] = nd;
            mbar_arrive_warp(&bar->delta_bar);
            if (!wait_warp(&bar->delta_bar, 0, w)) return false;
            nd = half_delta[row] + half_delta[128 + row];
            if (half == 0 && real) a.delta[at] = -nd;
            summed = true;
            return true;
        };
        for (int u = half; u < n; u += 2) {
            const int ph = (u >> 1) & 1, c0 = kt.tile(u % nt) * 64;
            if (!summed && u >= n - nt && !(ok = join_delta())) break;
            if (!(ok = wait_warp(bar->s_full + (u & 3), (u >> 2) & 1, w))) break;
            tc_fence_after();
            const uint32_t ts = tl + 64 * (u & 3), td = tl + 256 + 64 * half;
            float x[64];
            tmem_ld32f(ts, &x[0]);
            tmem_ld32f(ts + 32, &x[32]);
            tmem_wait_ld();
            const bool all = __all_sync(0xffffffffu, c0 + 64 <= rk.hi &&
                                                         (c0 >= rk.lo || c0 + 64 <= rk.sink));
            const uint64_t see =
                below(rk.hi - c0) & (~below(rk.lo - c0) | below(rk.sink - c0));
#pragma unroll
            for (int k = 0; k < 64; k += 2) {
                float lo, hi;
                f2_unpack(f2_fma(f2_pack(x[k], x[k + 1]), c2, nl2), lo, hi);
                x[k] = fast_exp2(lo);
                x[k + 1] = fast_exp2(hi);
            }
            if (c0 + 64 > seq.len) {
                // keys past the sequence may hold anything, and 0 * NaN is NaN: they become
                // zeros before the product over the keys (S of this block is done with them)
                zero_rows(sm + L::kRing + u % N1 * L::kBlock, max(0, seq.len - c0), 64, PN,
                          L::kBlockPanel, row, 128);
                fence_proxy_async_smem();
            }
            if (!(ok = wait_warp(bar->dp_full + half, ph, w))) break;
            tc_fence_after();
            if (u < n - nt) {
                // this group's part of delta = sum P dP
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                    float y[32];
                    tmem_ld32f(td + c, y);
                    tmem_wait_ld();
                    const uint32_t s = (uint32_t)(see >> c);
#pragma unroll
                    for (int k = 0; k < 32; k++)
                        sum = fmaf((s >> k) & 1 ? x[c + k] : 0.f, (s >> k) & 1 ? y[k] : 0.f, sum);
                }
                nd -= sum;
                tc_fence_before();
                mbar_arrive_warp(bar->ds_full + half);
                continue;
            }
            const uint64_t nd2 = f2_pack(nd, nd);
            uint32_t pk[32];
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
                float y[32];
                tmem_ld32f(td + c, y);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; k += 2)
                    f2_unpack(f2_mul(f2_add(f2_pack(y[k], y[k + 1]), nd2),
                                     f2_pack(x[c + k], x[c + k + 1])),
                              y[k], y[k + 1]);
                if (!all) {
                    const uint32_t s = (uint32_t)(see >> c);
#pragma unroll
                    for (int k = 0; k < 32; k++) y[k] = (s >> k) & 1 ? y[k] : 0.f;
                }
#pragma unroll
                for (int k = 0; k < 16; k++) pk[c / 2 + k] = pack_bf16(y[2 * k], y[2 * k + 1]);
            }
            tmem_st32(ts, pk);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive_warp(bar->ds_full + half);
        }
        if (ok && !summed) ok = join_delta();
        if (ok && wait_warp(&bar->acc_full, 0, w)) {
            tc_fence_after();
            const int x = half * (D / 2);
            store_row<D / 2>(tl + 384 + x, dq + (int64_t)i * a.g.dq.token + x, p.scale, p.d - x,
                             i < p.Nq);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D>
cudaError_t launch(const WinProblem &p, const WinGrads &g, const void *q, const void *k,
                   const void *v, const void *dout, const BwdArgs &a, cudaStream_t stream) {
    // the fixed tiles have 128 rows, the streamed blocks 64
    CUtensorMap q128, k128, v128, d128, q64, k64, v64, d64;
    if (!map_tokens(&q128, q, p.q, p.B, p.H, p.Nq, p.d, 128) ||
        !map_tokens(&q64, q, p.q, p.B, p.H, p.Nq, p.d, 64) ||
        !map_tokens(&d128, dout, g.dout, p.B, p.H, p.Nq, p.d, 128) ||
        !map_tokens(&d64, dout, g.dout, p.B, p.H, p.Nq, p.d, 64) ||
        !map_tokens(&k128, k, p.k, p.B, p.Hkv, p.Nk, p.d, 128) ||
        !map_tokens(&k64, k, p.k, p.B, p.Hkv, p.Nk, p.d, 64) ||
        !map_tokens(&v128, v, p.v, p.B, p.Hkv, p.Nk, p.d, 128) ||
        !map_tokens(&v64, v, p.v, p.B, p.Hkv, p.Nk, p.d, 64))
        return cudaErrorInvalidValue;
    constexpr uint32_t smem = BwdLayout<D>::kSmem;
    cudaError_t e = tcs::set_smem(tc_window_dkv_kernel<D>, smem);
    if (e == cudaSuccess) e = tcs::set_smem(tc_window_dq_kernel<D>, smem);
    if (e != cudaSuccess) return e;
    const unsigned gk = (unsigned)p.B * p.Hkv * ((p.Nk + 127) / 128);
    const unsigned gq = (unsigned)p.B * p.H * ((p.Nq + 127) / 128);
    // dq first: it completes delta
    tc_window_dq_kernel<D><<<gq, kThreads, smem, stream>>>(q128, k64, v64, d128, a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    tc_window_dkv_kernel<D><<<gk, kThreads, smem, stream>>>(q64, k128, v128, d64, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t tc_backward(const WinProblem &p, const WinGrads &g, const void *q, const void *k,
                        const void *v, const float *lse, float *delta, const void *dout,
                        void *dq, void *dk, void *dv, int *status, long long limit,
                        cudaStream_t stream) {
    BwdArgs a;
    a.p = p;
    a.g = g;
    a.lse = lse;
    a.delta = delta;
    a.dq = (__nv_bfloat16 *)dq;
    a.dk = (__nv_bfloat16 *)dk;
    a.dv = (__nv_bfloat16 *)dv;
    a.status = status;
    a.limit = limit;
    a.stall = device_inject_stall();
    return p.d == 128 ? launch<128>(p, g, q, k, v, dout, a, stream)
                      : launch<64>(p, g, q, k, v, dout, a, stream);
}

}  // namespace win
}  // namespace monarch
