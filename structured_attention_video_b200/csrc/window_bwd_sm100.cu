// window_bwd_sm100.cu -- backward of the window attention on the sm_100a tensor cores
// (bfloat16 inputs and gradients, float32 sums; P and dS rounded to bfloat16 as
// operands of the accumulating products, from 32-bit values).
//
//   P = exp2(scale_log2 S - lse log2(e)),  dS = P (dO V^T - delta),
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K.
//
// Two kernels, so that every gradient is summed by one CTA in a fixed order (no
// atomics) at the price of forming S and dO V^T twice (7 products instead of 5):
//   tc_window_dkv_kernel  128 keys of one key head against the 64-query blocks of
//                         every head of its group that see them;
//   tc_window_dq_kernel   128 queries of one head against their 64-key blocks.
// 640 threads a CTA, one CTA an SM: warps 0-15 the elementwise work, warp 16 loads, one
// thread of warp 17 issues S and dV, one of warp 18 dP and dK (or dQ), warp 19 stages lse
// and delta (dkv).
//
// The streamed side goes in blocks of 64 rows (queries in dkv, keys in dq).  Blocks u
// with u % 2 = h belong to warps 8 h .. 8 h + 7 (a thread has 32 columns of one row, its
// tensor-memory lane, of the fixed tile), so the two groups work on different blocks at
// different times and the tensor pipe has the products of one while the other computes.
// Order of each issuer's products (fixed, and each accumulator has one issuer, so the
// sums are fixed too):
//   dkv:  dV(u) S(u+2) after P(u)         |  dK(u) dP(u+2) after dS(u)
//   dq:   S(u+2) once S(u) is read        |  dQ(u) dP(u+2) after dS(u)
// P lies over S and dS over dP in tensor memory; a later product into the same columns
// follows in issue order.  What shaped this (d = 128, 12 heads, nine 480p frames of which each sees four):
//  - Two stages of 128 rows with 128-column products, all warps in step: dkv 1107 us, dq
//    787; the pipe waited for loads and for the elementwise work in turn.
//  - 64-row blocks, one thread elected for the whole role (an election or a branch per
//    product costs 30 to 80 clocks each): dkv 735, dq 659.
//  - M = 128, N = 64 reads 4 KB of A and 2 KB of B a K-step, 48 clocks of shared memory's
//    128 bytes a clock against 32 of the tensor pipe: Q and dO live in tensor memory in dq
//    (659 -> 648); in dkv the accumulators leave no room.
//  - Sixteen elementwise warps of 32 columns instead of eight of 64: dkv 710, dq 581.  A
//    second issuer, as one thread's barrier polls left the pipe idle: dkv 672, dq 536.
//
// delta comes from out as the forward rounded it, an error of 2^-8 |dO.O| at most.  A
// row of n keys of like weight has |O| of about n^(-1/2) |v|, so against dP it matters
// for few keys only.  Query tiles of up to kExactBlocks key blocks therefore first walk
// their keys once for delta = sum P dP from the same products that form dS, and the dq
// kernel runs first to hand it to the dk/dv kernel.  (Two padded causal
// sequences of 1023 and 681 tokens, d = 64: dq is 2.6e-3 from 64 bits without it.)
// Bound by the tensor pipe and, nearly as long, the elementwise warps' issue slots: 4 (3)
// products of 128 x 128 x d a tile against 16384 exponentials at 16 a clock.  The same
// frames, forward included: 1667 us in a burst and 1913 in a long run, where the power
// limit lowers the clocks, against 967 of the fewest products at the rate of a large matrix
// product.
#include "window_tc.cuh"

namespace monarch {
namespace win {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 640;
constexpr int kLoadWarp = 16, kIssueWarp = 17, kIssueWarp2 = 18, kStatsWarp = 19;
constexpr int kExactBlocks = 6;
constexpr int kDkvRing1 = 5, kDkvRing2 = 5, kDqRing1 = 8, kDqRing2 = 6;

// Shared memory: FIX fixed tiles of 128 rows (K and V of dkv), two rings of N1 and N2
// 64-row blocks, then per slot of the first ring -lse and -delta of its 64 queries (dkv) or the
// warps' parts of delta (dq).
template <int D, int FIX, int N1, int N2> struct BwdLayout {
    static constexpr uint32_t kTile = (D / 64) * kPanel;
    static constexpr uint32_t kBlock = kTile / 2;             // panels of 64 rows
    static constexpr uint32_t kBlockPanel = 64 * 128;
    static constexpr uint32_t kRing = FIX * kTile;
    static constexpr uint32_t kStats = kRing + (N1 + N2) * kBlock;
    static constexpr uint32_t kBar = kStats + (FIX ? N1 * 512 : 2048);
    static constexpr uint32_t kSmem = kBar + 512;   // the base is 1024-aligned (checked)
    static_assert(kSmem <= (uint32_t)kMaxSmem, "window backward shared memory");
};

struct BwdArgs {
    WinProblem p;
    WinGrads g;
    const float *lse;
    float *delta;   // of the rounded out; rows of few keys are written again (dq kernel)
    const __nv_bfloat16 *q, *dout;
    __nv_bfloat16 *dq, *dk, *dv;
    int splits;     // parts of a key tile's query blocks, a CTA each (dkv)
    float *parts;   // splits > 1: [key tile, batch, head][split][128][dV | dK of D]
    int *status;
    long long limit;
    int stall;
};

// The lowest n bits, n clamped to [0, 32].
__device__ __forceinline__ uint32_t below(int n) {
    return n >= 32 ? ~0u : (1u << max(n, 0)) - 1;
}

// N columns of an accumulator row to bfloat16 in global memory (columns below d), if the
// row is in the tensor; zeros if it is not real.
template <int N>
__device__ __forceinline__ void store_row(uint32_t taddr, __nv_bfloat16 *dst, float scale, int d,
                                          bool in, bool real) {
#pragma unroll 1
    for (int c = 0; c < N; c += 16) {
        float o[16];
        tmem_ld16f(taddr + c, o);
        tmem_wait_ld();
        if (!in || c >= d) continue;
#pragma unroll
        for (int e = 0; e < 16; e++) o[e] = real ? o[e] : 0.f;
#pragma unroll
        for (int e = 0; e < 2; e++)
            *reinterpret_cast<uint4 *>(dst + c + 8 * e) =
                make_uint4(pack_bf16(o[8 * e] * scale, o[8 * e + 1] * scale),
                           pack_bf16(o[8 * e + 2] * scale, o[8 * e + 3] * scale),
                           pack_bf16(o[8 * e + 4] * scale, o[8 * e + 5] * scale),
                           pack_bf16(o[8 * e + 6] * scale, o[8 * e + 7] * scale));
    }
}
// N columns of an accumulator row as they are.
template <int N> __device__ __forceinline__ void store_part(uint32_t taddr, float *dst) {
#pragma unroll 1
    for (int c = 0; c < N; c += 16) {
        float o[16];
        tmem_ld16f(taddr + c, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<float4 *>(dst + c + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
    }
}
__device__ __forceinline__ void zero_row(__nv_bfloat16 *dst, int n) {
    for (int c = 0; c < n; c += 8) *reinterpret_cast<uint4 *>(dst + c) = make_uint4(0, 0, 0, 0);
}

// Elements whose bit of `see` is 0 become 0, whatever they were.
__device__ __forceinline__ void keep_seen(float (&x)[32], uint32_t see) {
#pragma unroll
    for (int k = 0; k < 32; k++) x[k] = (see >> k) & 1 ? x[k] : 0.f;
}

// 32 columns as bfloat16 pairs over 16 columns of tensor memory.
__device__ __forceinline__ void pack_to_tmem(uint32_t taddr, const float (&x)[32]) {
    uint32_t pk[16];
#pragma unroll
    for (int k = 0; k < 16; k++) pk[k] = pack_bf16(x[2 * k], x[2 * k + 1]);
    tmem_st8(taddr, *reinterpret_cast<const uint32_t(*)[8]>(&pk[0]));
    tmem_st8(taddr + 8, *reinterpret_cast<const uint32_t(*)[8]>(&pk[8]));
    tmem_wait_st();
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

// Barriers of one CTA.  N1, N2: blocks of the two rings.
// READERS: issuers that read a block of the second ring.
template <int N1, int N2, int READERS> struct Bars {
    uint64_t fix_full;                  // the fixed tiles
    uint64_t tmem_full;                 // Q and dO in tensor memory (dq), 8 warps
    uint64_t full1[N1], empty1[N1];     // Q (dkv) or K (dq)
    uint64_t full2[N2], empty2[N2];     // dO or V
    uint64_t stats_full[N1];            // dkv
    uint64_t s_full[2], dp_full[2];     // products in tensor memory, per half
    uint64_t s_free[2];                 // S is read (dq), the half's 8 warps
    uint64_t p_full[2], ds_full[2];     // the half's 8 warps
    uint64_t delta_bar;                 // the parts of delta (dq), 16 warps, once
    uint64_t done[2];                   // each issuer's last products
    uint64_t stall_bar;                 // never completed (fault injection)
    uint32_t tmem_slot;
    int abort_flag;
    Sequence seq;                       // of the whole CTA

    __device__ __forceinline__ void init() {
        mbar_init(&fix_full, 1);
        mbar_init(&tmem_full, 8);
        for (int i = 0; i < N1; i++) {
            mbar_init(full1 + i, 1);
            mbar_init(empty1 + i, 1);
            mbar_init(stats_full + i, 1);
        }
        for (int i = 0; i < N2; i++) {
            mbar_init(full2 + i, 1);
            mbar_init(empty2 + i, READERS);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(s_full + i, 1);
            mbar_init(dp_full + i, 1);
            mbar_init(s_free + i, 8);
            mbar_init(p_full + i, 8);
            mbar_init(ds_full + i, 8);
        }
        mbar_init(&delta_bar, 16);
        mbar_init(done, 1);
        mbar_init(done + 1, 1);
        mbar_init(&stall_bar, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    // Every issued copy lands before the CTA may exit (an aborted CTA may not have
    // waited for the last ones).
    __device__ __forceinline__ void drain(int issued1, int issued2) {
        for (int u = max(0, issued1 - N1); u < issued1; u++)
            wait_phase_cleanup(full1 + u % N1, (u / N1) & 1, kCleanupPolls);
        for (int u = max(0, issued2 - N2); u < issued2; u++)
            wait_phase_cleanup(full2 + u % N2, (u / N2) & 1, kCleanupPolls);
    }
};

// A role of one thread of a warp: waits and issues until body() is done or gives up,
// then waits for its own products, which the CTA's exit must not overtake.
template <typename Body>
__device__ __forceinline__ void issuer(uint64_t *done, const Body &body) {
    if (elect_one()) {
        body();
        mma_commit(done);
        wait_phase_cleanup(done, 0, kCleanupPolls);
    }
    __syncwarp();
}

// One CTA's loads of the blocks of both rings, in the order in which the products need
// them.  coords(u, h, row): head and first row of block u.
template <int D, typename L, int N1, int N2, int RD, typename Coords>
__device__ __forceinline__ void load_blocks(uint8_t *sm, Bars<N1, N2, RD> *bar,
                                            const CUtensorMap *ring1, const CUtensorMap *ring2,
                                            int b, int n, const Coords &coords, const WaitCtx &w,
                                            int lane) {
    constexpr int PN = D / 64;
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
// Tensor memory: S^T of half h at 64 h, dP^T at 128 + 64 h, dV at 256, dK at 384.  P^T and
// dS^T of each 32 columns lie over the first 16 of them.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
tc_window_dkv_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmDo, BwdArgs a) {
    constexpr int PN = D / 64, N1 = kDkvRing1, N2 = kDkvRing2;
    using L = BwdLayout<D, 2, N1, N2>;
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
    const int tile_unit = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
    const int unit = tile_unit % (p.B * p.Hkv), hk = unit % p.Hkv, b = unit / p.Hkv;
    const int j0 = tile_unit / (p.B * p.Hkv) * 128;
    Sequence seq = first_threads_sequence(p, b);
    if (threadIdx.x == 32) bar->init();
    share_sequence(seq, &bar->seq);
    int first, last;
    query_rows(p, seq, j0, j0 + 128, first, last);
    const int t0 = first / 64, nt = last > first ? (last + 63) / 64 - t0 : 0;
    // query blocks over the group's heads; this CTA's
    const int u0 = (int)((int64_t)nt * p.G * split / a.splits);
    const int n = (int)((int64_t)nt * p.G * (split + 1) / a.splits) - u0;
    // (row of this CTA's part: dV, then dK, in 32 bits)
    float *const part_base = a.parts + (int64_t)blockIdx.x * 128 * 2 * D;

    if (n == 0) {             // no query sees these keys (the same for the whole CTA)
        const int j = j0 + threadIdx.x;
        if (a.splits > 1) {
            for (int x = threadIdx.x; x < 128 * 2 * D / 4; x += kThreads)
                reinterpret_cast<float4 *>(part_base)[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        } else if (threadIdx.x < 128 && j < p.Nk) {
            zero_row(a.dk + b * a.g.dk.batch + hk * a.g.dk.head + (int64_t)j * a.g.dk.token, p.d);
            zero_row(a.dv + b * a.g.dv.batch + hk * a.g.dv.head + (int64_t)j * a.g.dv.token, p.d);
        }
        return;
    }
    if (warp == kIssueWarp) tmem_alloc(&bar->tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem_slot;
    const WaitCtx w{a.limit, a.status, &bar->abort_flag};
    auto coords = [&](int u, int &h, int &row) {
        h = hk * p.G + (u0 + u) / nt;
        row = (t0 + (u0 + u) % nt) * 64;
    };

    constexpr uint32_t idS = idesc_bf16(128, 64, 0, 0), idO = idesc_bf16(128, D, 0, 1);
    constexpr uint32_t kBlockDesc = L::kBlock >> 4;
    const uint32_t ring = smem_u32(sm + L::kRing);
    const uint64_t dK = smem_desc_sw128(smem_u32(sm), 16, 1024);
    const uint64_t dV = smem_desc_sw128(smem_u32(sm + L::kTile), 16, 1024);
    const uint64_t dQ = smem_desc_sw128(ring, 16, 1024);
    const uint64_t dO = smem_desc_sw128(ring + N1 * L::kBlock, 16, 1024);
    const uint64_t dQt = smem_desc_sw128(ring, L::kBlockPanel, 1024);
    const uint64_t dOt = smem_desc_sw128(ring + N1 * L::kBlock, L::kBlockPanel, 1024);

    if (warp == kLoadWarp) {
        if (lane == 0) {
            mbar_expect_tx(&bar->fix_full, 2 * L::kTile);
            for (int pn = 0; pn < PN; pn++) {
                tma_load_4d(sm + pn * kPanel, &tmK, pn * 64, j0, hk, b, &bar->fix_full);
                tma_load_4d(sm + L::kTile + pn * kPanel, &tmV, pn * 64, j0, hk, b, &bar->fix_full);
            }
        }
        load_blocks<D, L>(sm, bar, &tmQ, &tmDo, b, n, coords, w, lane);
        if (lane == 0) wait_phase_cleanup(&bar->fix_full, 0, kCleanupPolls);
    } else if (warp == kStatsWarp) {
        // -lse (in log2 units) and -delta of each block's queries.  (A warp of its own: in
        // the loading warp, its global reads held up the copies, 722 -> 915 us.)
        Slot<N1> cur;
        for (int u = 0; u < n; u++) {
            int h, i0;
            coords(u, h, i0);
            const int64_t at = ((int64_t)b * p.H + h) * p.Nq + i0;
            float2 st[2];
#pragma unroll
            for (int x = 0; x < 2; x++) {
                const int i = lane + 32 * x;
                st[x] = i0 + i < p.Nq ? make_float2(-a.lse[at + i] * kLog2e, -a.delta[at + i])
                                      : make_float2(0.f, 0.f);
            }
            if (u >= N1 && !wait_warp(bar->empty1 + cur.s, cur.ph ^ 1, w)) break;
            float *dst = stats + cur.s * 128;
#pragma unroll
            for (int x = 0; x < 2; x++) {
                dst[lane + 32 * x] = st[x].x;
                dst[64 + lane + 32 * x] = st[x].y;
            }
            mbar_arrive_warp(bar->stats_full + cur.s);
            cur.next();
        }
    } else if (warp == kIssueWarp) {
        issuer(bar->done, [&]() {
            if ((a.stall && !spin_phase(&bar->stall_bar, 0, w)) || !spin_phase(&bar->fix_full, 0, w))
                return;
            Slot<N1> next;   // of the next S
            Slot<N2> cur;    // dO of block u
            auto issue_s = [&](int h) -> bool {
                if (!spin_phase(bar->full1 + next.s, next.ph, w)) return false;
                tc_fence_after();
                mma_head<D, 64>(tmem + 64 * h, dK, dQ + next.s * kBlockDesc, idS);
                mma_commit(bar->s_full + h);
                next.next();
                return true;
            };
            if (!issue_s(0) || (n > 1 && !issue_s(1))) return;
            for (int u = 0; u < n; u++) {
                const int h = u & 1;
                if (!spin_phase(bar->full2 + cur.s, cur.ph, w) ||
                    !spin_phase(bar->p_full + h, (u >> 1) & 1, w))
                    return;
                tc_fence_after();
                mma_block64<32>(tmem + 256, tmem + 64 * h, dOt + cur.s * kBlockDesc, idO, u > 0);
                mma_commit(bar->empty2 + cur.s);
                cur.next();
                if (u + 2 < n && !issue_s(h)) return;
            }
        });
    } else if (warp == kIssueWarp2) {
        issuer(bar->done + 1, [&]() {
            if (!spin_phase(&bar->fix_full, 0, w)) return;
            Slot<N2> next;   // of the next dP
            Slot<N1> cur;    // Q of block u
            auto issue_dp = [&](int h) -> bool {
                if (!spin_phase(bar->full2 + next.s, next.ph, w)) return false;
                tc_fence_after();
                mma_head<D, 64>(tmem + 128 + 64 * h, dV, dO + next.s * kBlockDesc, idS);
                mma_commit(bar->dp_full + h);
                mma_commit(bar->empty2 + next.s);
                next.next();
                return true;
            };
            if (!issue_dp(0) || (n > 1 && !issue_dp(1))) return;
            for (int u = 0; u < n; u++) {
                const int h = u & 1;
                if (!spin_phase(bar->full1 + cur.s, cur.ph, w) ||
                    !spin_phase(bar->ds_full + h, (u >> 1) & 1, w))
                    return;
                tc_fence_after();
                mma_block64<32>(tmem + 384, tmem + 128 + 64 * h, dQt + cur.s * kBlockDesc, idO, u > 0);
                mma_commit(bar->empty1 + cur.s);
                cur.next();
                if (u + 2 < n && !issue_dp(h)) return;
            }
        });
    } else if (warp < kLoadWarp) {
        // ---------------- elementwise: key row j, 32 queries of each of the half's blocks
        const int half = warp >> 3, part = (warp >> 2) & 1, row = (warp & 3) * 32 + lane;
        const int j = j0 + row;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ts = lanes + 64 * half, td = ts + 128;
        int ilo, ihi, rfirst, rlast;
        // the queries that see this key; a row that is not a key takes them all, so that its
        // warp needs no masks (its sums touch nothing else), and zeros are stored
        query_rows(p, seq, j, j + 1, ilo, ihi);
        const bool key = j < seq.len;
        if (!key) ilo = 0, ihi = 0x7fffffff;
        real_rows(p, seq, 0, p.Nq, rfirst, rlast);
        const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2);
        bool ok = true;
        int x0 = (u0 + half) % nt;   // block of its head
        for (int u = half; u < n; u += 2) {
            const int ph = (u >> 1) & 1, s1 = u % N1, c0 = (t0 + x0) * 64 + 32 * part;
            x0 += 2;
            while (x0 >= nt) x0 -= nt;
            const float *nl = stats + s1 * 128 + 32 * part, *nd = nl + 64;
            const bool all = __all_sync(0xffffffffu, c0 >= ilo && c0 + 32 <= ihi);
            const uint32_t see = below(ihi - c0) & ~below(ilo - c0);
            if (!(ok = wait_warp(bar->stats_full + s1, (u / N1) & 1, w) &&
                       wait_warp(bar->s_full + half, ph, w)))
                break;
            tc_fence_after();
            float x[32];
            tmem_ld32f(ts + 32 * part, x);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
                const ulonglong2 n2 = *reinterpret_cast<const ulonglong2 *>(nl + k);
                f2_unpack(f2_fma(f2_pack(x[k], x[k + 1]), c2, n2.x), x[k], x[k + 1]);
                f2_unpack(f2_fma(f2_pack(x[k + 2], x[k + 3]), c2, n2.y), x[k + 2], x[k + 3]);
#pragma unroll
                for (int e = 0; e < 4; e++) x[k + e] = fast_exp2(x[k + e]);
            }
            if (!all) keep_seen(x, see);
            pack_to_tmem(ts + 32 * part, x);   // over the part's own columns of S
            if (c0 < rfirst || (rlast < p.Nq && c0 + 32 > rlast)) {
                // rows that are not real may hold anything, and 0 * NaN is NaN: they become
                // zeros before the products over the queries
                const int s2 = u % N2;
                if (!(ok = wait_warp(bar->full2 + s2, (u / N2) & 1, w))) break;
                const int za = min(max(rfirst - c0, 0), 32), zb = min(max(rlast - c0, 0), 32);
                for (int x2 = 0; x2 < 2; x2++) {
                    uint8_t *blk = sm + L::kRing + (x2 ? N1 + s2 : s1) * L::kBlock + part * 32 * 128;
                    zero_rows(blk, 0, za, PN, L::kBlockPanel, row, 128);
                    zero_rows(blk, zb, 32, PN, L::kBlockPanel, row, 128);
                }
                fence_proxy_async_smem();
            }
            tc_fence_before();
            mbar_arrive_warp(bar->p_full + half);
            if (!(ok = wait_warp(bar->dp_full + half, ph, w))) break;
            tc_fence_after();
            float y[32];
            tmem_ld32f(td + 32 * part, y);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
                const ulonglong2 d2 = *reinterpret_cast<const ulonglong2 *>(nd + k);
                f2_unpack(f2_mul(f2_add(f2_pack(y[k], y[k + 1]), d2.x), f2_pack(x[k], x[k + 1])),
                          y[k], y[k + 1]);
                f2_unpack(f2_mul(f2_add(f2_pack(y[k + 2], y[k + 3]), d2.y),
                                 f2_pack(x[k + 2], x[k + 3])),
                          y[k + 2], y[k + 3]);
            }
            if (!all) keep_seen(y, see);
            pack_to_tmem(td + 32 * part, y);
            tc_fence_before();
            mbar_arrive_warp(bar->ds_full + half);
        }
        if (ok && wait_warp(bar->done, 0, w) && wait_warp(bar->done + 1, 0, w)) {
            tc_fence_after();
            // a quarter of the head's columns, of dV and dK, for each group of four warps
            constexpr int W = D / 4;
            const int64_t x = (half * 2 + part) * W;
            const bool real = j < p.Nk;
            if (a.splits > 1) {
                float *dst = part_base + row * 2 * D + x;
                store_part<W>(lanes + 256 + x, dst);
                store_part<W>(lanes + 384 + x, dst + D);
            } else {
                store_row<W>(lanes + 256 + x,
                             a.dv + b * a.g.dv.batch + hk * a.g.dv.head + j * a.g.dv.token + x, 1.f,
                             p.d - (int)x, real, key);
                store_row<W>(lanes + 384 + x,
                             a.dk + b * a.g.dk.batch + hk * a.g.dk.head + j * a.g.dk.token + x,
                             p.scale, p.d - (int)x, real, key);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kIssueWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// dk and dv from the parts of each key tile's query blocks, added in order.
template <int D>
__global__ void __launch_bounds__(256) window_dkv_join_kernel(BwdArgs a) {
    const WinProblem &p = a.p;
    const int tile_unit = blockIdx.x, unit = tile_unit % (p.B * p.Hkv);
    const int hk = unit % p.Hkv, b = unit / p.Hkv, j0 = tile_unit / (p.B * p.Hkv) * 128;
    const Sequence seq = sequence(p, b);
    const float *base = a.parts + (int64_t)tile_unit * a.splits * 128 * 2 * D;
    const int at = blockIdx.y * 256 + threadIdx.x;   // 4 columns of a row
    const int row = at / (2 * D / 4), x = at % (2 * D / 4) * 4, j = j0 + row;
    const bool is_k = x >= D;
    const int col = is_k ? x - D : x;
    if (j >= p.Nk || col >= p.d) return;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    if (j < seq.len)
        for (int s = 0; s < a.splits; s++) {
            const float4 y = *reinterpret_cast<const float4 *>(base + ((int64_t)s * 128 + row) * 2 * D + x);
            sum.x += y.x, sum.y += y.y, sum.z += y.z, sum.w += y.w;
        }
    const float f = is_k ? p.scale : 1.f;
    __nv_bfloat16 *dst =
        is_k ? a.dk + b * a.g.dk.batch + hk * a.g.dk.head + (int64_t)j * a.g.dk.token
             : a.dv + b * a.g.dv.batch + hk * a.g.dv.head + (int64_t)j * a.g.dv.token;
    *reinterpret_cast<uint2 *>(dst + col) =
        make_uint2(pack_bf16(sum.x * f, sum.y * f), pack_bf16(sum.z * f, sum.w * f));
}

// ---------------------------------------------------------------- dq
// Tensor memory: S of half h at 64 h, dP at 128 + 64 h (dS of each 32 columns over the
// first 16), dQ at 256, Q at 384, dO at 448.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
tc_window_dq_kernel(const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, BwdArgs a) {
    // a key block stays from S(u) to dQ(u), a value block for dP(u) alone
    constexpr int PN = D / 64, N1 = kDqRing1, N2 = kDqRing2;
    using L = BwdLayout<D, 0, N1, N2>;
    using B = Bars<N1, N2, 1>;
    static_assert(sizeof(B) <= 512, "barriers");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = smem_raw;
    if (!base_aligned(sm, a.status)) return;
    B *bar = reinterpret_cast<B *>(sm + L::kBar);
    float *part_delta = reinterpret_cast<float *>(sm + L::kStats);   // [half, part][128]
    const WinProblem &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the last tiles first: they see the most keys under a causal mask
    const int unit = blockIdx.x % (p.B * p.H), h = unit % p.H, b = unit / p.H;
    const int i0 = ((int)gridDim.x - 1 - (int)blockIdx.x) / (p.B * p.H) * 128;
    Sequence seq = first_threads_sequence(p, b);
    if (threadIdx.x == 32) bar->init();
    share_sequence(seq, &bar->seq);
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
    if (warp == kIssueWarp) tmem_alloc(&bar->tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem_slot;
    const WaitCtx w{a.limit, a.status, &bar->abort_flag};

    constexpr uint32_t idS = idesc_bf16(128, 64, 0, 0), idO = idesc_bf16(128, D, 0, 1);
    constexpr uint32_t kBlockDesc = L::kBlock >> 4;
    const uint32_t ring = smem_u32(sm + L::kRing);
    const uint64_t dK = smem_desc_sw128(ring, 16, 1024);
    const uint64_t dV = smem_desc_sw128(ring + N1 * L::kBlock, 16, 1024);
    const uint64_t dKt = smem_desc_sw128(ring, L::kBlockPanel, 1024);

    if (warp == kLoadWarp) {
        auto coords = [&](int u, int &head, int &row) {
            head = h / p.G;
            row = kt.tile(u % nt) * 64;
        };
        load_blocks<D, L>(sm, bar, &tmK, &tmV, b, n, coords, w, lane);
    } else if (warp == kIssueWarp) {
        issuer(bar->done, [&]() {
            if ((a.stall && !spin_phase(&bar->stall_bar, 0, w)) || !spin_phase(&bar->tmem_full, 0, w))
                return;
            Slot<N1> next;
            for (int u = 0; u < n; u++) {
                const int h = u & 1;
                if (!spin_phase(bar->full1 + next.s, next.ph, w) ||
                    (u >= 2 && !spin_phase(bar->s_free + h, ((u - 2) >> 1) & 1, w)))
                    return;
                tc_fence_after();
                mma_head_ts<D, 64>(tmem + 64 * h, tmem + 384, dK + next.s * kBlockDesc, idS);
                mma_commit(bar->s_full + h);
                next.next();
            }
        });
    } else if (warp == kIssueWarp2) {
        issuer(bar->done + 1, [&]() {
            if (!spin_phase(&bar->tmem_full, 0, w)) return;
            Slot<N2> next;   // of the next dP
            Slot<N1> cur;    // K of block u
            auto issue_dp = [&](int h) -> bool {
                if (!spin_phase(bar->full2 + next.s, next.ph, w)) return false;
                tc_fence_after();
                mma_head_ts<D, 64>(tmem + 128 + 64 * h, tmem + 448, dV + next.s * kBlockDesc, idS);
                mma_commit(bar->dp_full + h);
                mma_commit(bar->empty2 + next.s);
                next.next();
                return true;
            };
            if (!issue_dp(0) || (n > 1 && !issue_dp(1))) return;
            for (int u = 0; u < n; u++) {
                const int h = u & 1;
                if (!spin_phase(bar->full1 + cur.s, cur.ph, w) ||
                    !spin_phase(bar->ds_full + h, (u >> 1) & 1, w))
                    return;
                tc_fence_after();
                if (u >= n - nt)
                    mma_block64<32>(tmem + 256, tmem + 128 + 64 * h, dKt + cur.s * kBlockDesc, idO,
                                    u > n - nt);
                mma_commit(bar->empty1 + cur.s);
                cur.next();
                if (u + 2 < n && !issue_dp(h)) return;
            }
        });
    } else if (warp < kLoadWarp) {
        // ---------------- elementwise: query row i, 32 keys of each of the half's blocks
        const int half = warp >> 3, part = (warp >> 2) & 1, row = (warp & 3) * 32 + lane;
        const int i = i0 + row;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ts = lanes + 64 * half + 32 * part, td = ts + 128;
        if (half == 0) {   // Q's rows to tensor memory (warps 0-3) and dO's (warps 4-7)
            row_to_tmem<D>(lanes + 384 + 64 * part,
                           part ? a.dout + b * a.g.dout.batch + h * a.g.dout.head + i * a.g.dout.token
                                : a.q + b * p.q.batch + h * p.q.head + i * p.q.token,
                           p.d, i < p.Nq);
            tc_fence_before();
            mbar_arrive_warp(&bar->tmem_full);
        }
        RowKeys rk = row_keys(p, seq, i);
        const int64_t at = ((int64_t)b * p.H + h) * p.Nq + i;
        const bool real = rk.hi > 0;   // (others take every key, and zeros are stored)
        if (!real) rk = RowKeys{0, 0x7fffffff, 0};
        const float nl = real ? -a.lse[at] * kLog2e : 0.f;
        float nd = real && n == nt ? -a.delta[at] : 0.f;
        const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2), nl2 = f2_pack(nl, nl);
        bool ok = true, summed = n == nt;
        // (warps without a block of their own still join delta)
        auto join_delta = [&]() -> bool {
            part_delta[(warp >> 2) * 128 + row] = nd;
            mbar_arrive_warp(&bar->delta_bar);
            if (!wait_warp(&bar->delta_bar, 0, w)) return false;
            nd = (part_delta[row] + part_delta[128 + row]) +
                 (part_delta[256 + row] + part_delta[384 + row]);
            if (warp < 4 && real) a.delta[at] = -nd;
            summed = true;
            return true;
        };
        for (int u = half; u < n; u += 2) {
            const int ph = (u >> 1) & 1, c0 = kt.tile(u < nt ? u : u - nt) * 64 + 32 * part;
            const bool all = __all_sync(0xffffffffu, c0 + 32 <= rk.hi &&
                                                         (c0 >= rk.lo || c0 + 32 <= rk.sink));
            const uint32_t see =
                below(rk.hi - c0) & (~below(rk.lo - c0) | below(rk.sink - c0));
            if (!summed && u >= n - nt && !(ok = join_delta())) break;
            if (!(ok = wait_warp(bar->s_full + half, ph, w))) break;
            tc_fence_after();
            float x[32];
            tmem_ld32f(ts, x);
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive_warp(bar->s_free + half);
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
                float lo, hi;
                f2_unpack(f2_fma(f2_pack(x[k], x[k + 1]), c2, nl2), lo, hi);
                x[k] = fast_exp2(lo);
                x[k + 1] = fast_exp2(hi);
            }
            if (c0 + 32 > seq.len) {
                // keys past the sequence may hold anything, and 0 * NaN is NaN: they become
                // zeros before the product over the keys (S of this block is done with them)
                zero_rows(sm + L::kRing + u % N1 * L::kBlock + part * 32 * 128, max(0, seq.len - c0),
                          32, PN, L::kBlockPanel, row, 128);
                fence_proxy_async_smem();
            }
            if (!(ok = wait_warp(bar->dp_full + half, ph, w))) break;
            tc_fence_after();
            float y[32];
            tmem_ld32f(td, y);
            tmem_wait_ld();
            if (u < n - nt) {
                // this part of delta = sum P dP
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < 32; k++)
                    sum = fmaf((see >> k) & 1 ? x[k] : 0.f, (see >> k) & 1 ? y[k] : 0.f, sum);
                nd -= sum;
            } else {
                const uint64_t nd2 = f2_pack(nd, nd);
#pragma unroll
                for (int k = 0; k < 32; k += 2)
                    f2_unpack(f2_mul(f2_add(f2_pack(y[k], y[k + 1]), nd2), f2_pack(x[k], x[k + 1])),
                              y[k], y[k + 1]);
                if (!all) keep_seen(y, see);
                pack_to_tmem(td, y);
            }
            tc_fence_before();
            mbar_arrive_warp(bar->ds_full + half);
        }
        if (ok && !summed) ok = join_delta();
        if (ok && wait_warp(bar->done + 1, 0, w)) {
            tc_fence_after();
            constexpr int W = D / 4;   // columns of dQ for each group of four warps
            const int x = (warp >> 2) * W;
            store_row<W>(lanes + 256 + x, dq + (int64_t)i * a.g.dq.token + x, p.scale, p.d - x,
                         i < p.Nq, real);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kIssueWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D>
cudaError_t launch(const WinProblem &p, const WinGrads &g, const void *q, const void *k,
                   const void *v, const void *dout, const BwdArgs &a, cudaStream_t stream) {
    // the fixed tiles have 128 rows, the streamed blocks 64
    CUtensorMap k128, v128, q64, k64, v64, d64;
    if (!map_tokens(&q64, q, p.q, p.B, p.H, p.Nq, p.d, 64) ||
        !map_tokens(&d64, dout, g.dout, p.B, p.H, p.Nq, p.d, 64) ||
        !map_tokens(&k128, k, p.k, p.B, p.Hkv, p.Nk, p.d, 128) ||
        !map_tokens(&k64, k, p.k, p.B, p.Hkv, p.Nk, p.d, 64) ||
        !map_tokens(&v128, v, p.v, p.B, p.Hkv, p.Nk, p.d, 128) ||
        !map_tokens(&v64, v, p.v, p.B, p.Hkv, p.Nk, p.d, 64))
        return cudaErrorInvalidValue;
    constexpr uint32_t smem_dkv = BwdLayout<D, 2, kDkvRing1, kDkvRing2>::kSmem;
    constexpr uint32_t smem_dq = BwdLayout<D, 0, kDqRing1, kDqRing2>::kSmem;
    cudaError_t e = tcs::set_smem(tc_window_dkv_kernel<D>, smem_dkv);
    if (e == cudaSuccess) e = tcs::set_smem(tc_window_dq_kernel<D>, smem_dq);
    if (e != cudaSuccess) return e;
    const unsigned key_tiles = (unsigned)p.B * p.Hkv * ((p.Nk + 127) / 128);
    const unsigned gk = key_tiles * a.splits;
    const unsigned gq = (unsigned)p.B * p.H * ((p.Nq + 127) / 128);
    // dq first: it completes delta
    tc_window_dq_kernel<D><<<gq, kThreads, smem_dq, stream>>>(k64, v64, a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    tc_window_dkv_kernel<D><<<gk, kThreads, smem_dkv, stream>>>(q64, k128, v128, d64, a);
    e = cudaGetLastError();
    if (e != cudaSuccess || a.splits == 1) return e;
    window_dkv_join_kernel<D><<<dim3(key_tiles, 128 * 2 * D / 4 / 256), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

// Parts of a key tile's query blocks in the dk/dv kernel: where the key tiles are fewer
// than the SMs, as many as fill them, of eight blocks at least (a part's prologue, its
// store and the join cost about four).  Two causal sequences of 1023 tokens, 8 heads on 2
// key heads, d = 64: 32 tiles of up to 64 blocks, 49 us whole, 20 and 4.5 for the join split.
int dkv_splits(const WinProblem &p) {
    const int64_t tiles = (int64_t)p.B * p.Hkv * ((p.Nk + 127) / 128);
    const int64_t blocks = (int64_t)((p.Nq + 63) / 64) * p.G;
    const int64_t fill = tcs::sm_count() / tiles;
    return (int)max((int64_t)1, min(fill, blocks / 8));
}

}  // namespace

size_t tc_backward_bytes(const WinProblem &p) {
    const int splits = dkv_splits(p);
    if (splits == 1) return 0;
    const size_t tiles = (size_t)p.B * p.Hkv * ((p.Nk + 127) / 128);
    return tiles * splits * 128 * 2 * (p.d == 128 ? 128 : 64) * sizeof(float);
}

cudaError_t tc_backward(const WinProblem &p, const WinGrads &g, const void *q, const void *k,
                        const void *v, const float *lse, float *delta, const void *dout,
                        void *dq, void *dk, void *dv, void *parts, int *status, long long limit,
                        cudaStream_t stream) {
    BwdArgs a;
    a.splits = dkv_splits(p);
    a.parts = (float *)parts;
    a.p = p;
    a.g = g;
    a.lse = lse;
    a.delta = delta;
    a.q = (const __nv_bfloat16 *)q;
    a.dout = (const __nv_bfloat16 *)dout;
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
