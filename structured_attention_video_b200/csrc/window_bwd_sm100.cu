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
// 384 threads a CTA, one CTA an SM: warps 0-7 the elementwise work (two warps a group
// of 32 tensor-memory lanes, each half of the 128 columns), warp 8 loads (TMA), warp 9
// issues the products, warp 10 stages lse and delta.
//
// Order of the products (dkv), chosen so that the tensor pipe always has one that
// does not wait for the elementwise work on the previous one:
//   S(0) dP(0)  |  dV(i) S(i+1) dK(i) dP(i+1)  |  ...
// While the warps form P(i + 1) the pipe runs dK(i) and dP(i + 1), while they form
// dS(i) it runs dV(i) and S(i + 1).  P overwrites S and dS overwrites dP in tensor
// memory, each half of the columns in its own place, so no warp waits for another
// before it writes; a later product into the same columns follows in issue order.
// In the dq kernel S has two buffers: dP(j+1) dQ(j) S(j+2) after dS(j).
//
// delta comes from out as the forward rounded it, an error of 2^-8 |dO.O| at most.  A
// row of n keys of like weight has |O| of about n^(-1/2) |v|, so against dP it matters
// for few keys only.  Query tiles of up to kExactTiles key tiles therefore first walk
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
constexpr int kExactTiles = 3;

// Shared memory: two fixed tiles of 128 rows, two stages of two streamed ones.
template <int D> struct BwdLayout {
    static constexpr uint32_t kTile = (D / 64) * kPanel;
    static constexpr uint32_t kFix = 0;                       // K, V (dkv) or Q, dO (dq)
    static constexpr uint32_t kRing = 2 * kTile;              // stage s: 2 tiles
    static constexpr uint32_t kStats = kRing + 4 * kTile;     // [stage][-lse | -delta][128] floats
    static constexpr uint32_t kBar = kStats + 2 * 2 * 512;
    static constexpr uint32_t kSmem = kBar + 256 + 1024;      // + slack to align the base
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

// Everything one CTA's roles share.
struct Bars {
    uint64_t *fix_full;      // the fixed tiles
    uint64_t *first_full;    // [2 stages]: Q (dkv) or K (dq)
    uint64_t *second_full;   // [2 stages]: dO or V
    uint64_t *stage_empty;   // [2 stages]: the products have read the stage
    uint64_t *stats_full;    // [2 stages] (dkv)
    uint64_t *s_full;        // [2] S in tensor memory (dkv uses the first)
    uint64_t *dp_full;
    uint64_t *p_full;        // 8 warps (dkv; in dq the halves of delta, once)
    uint64_t *ds_full;       // 8 warps
    uint64_t *acc_full;      // the last products
    uint64_t *stall_bar;
    uint32_t *tmem_slot;
    volatile int *abort_flag;
};

__device__ __forceinline__ Bars make_bars(uint8_t *at) {
    uint64_t *b = reinterpret_cast<uint64_t *>(at);
    return {b, b + 1, b + 3, b + 5, b + 7, b + 9, b + 11, b + 12, b + 13, b + 14, b + 15,
            reinterpret_cast<uint32_t *>(b + 16), reinterpret_cast<volatile int *>(b + 17)};
}
__device__ __forceinline__ void init_bars(const Bars &b) {
    for (int i = 0; i < 2; i++) {
        mbar_init(b.first_full + i, 1);
        mbar_init(b.second_full + i, 1);
        mbar_init(b.stage_empty + i, 1);
        mbar_init(b.stats_full + i, 1);
        mbar_init(b.s_full + i, 1);
    }
    mbar_init(b.fix_full, 1);
    mbar_init(b.dp_full, 1);
    mbar_init(b.p_full, 8);
    mbar_init(b.ds_full, 8);
    mbar_init(b.acc_full, 1);
    mbar_init(b.stall_bar, 1);
    *b.abort_flag = 0;
    fence_mbar_init();
}

// Every issued copy lands before the CTA may exit (an aborted CTA may not have
// waited for the last ones).
__device__ __forceinline__ void drain_loads(const Bars &b, const int (&issued)[2]) {
    wait_phase_cleanup(b.fix_full, 0, kCleanupPolls);
    for (int s = 0; s < 2; s++)
        if (issued[s] > 0) {
            wait_phase_cleanup(b.first_full + s, (issued[s] - 1) & 1, kCleanupPolls);
            wait_phase_cleanup(b.second_full + s, (issued[s] - 1) & 1, kCleanupPolls);
        }
}

// ---------------------------------------------------------------- dk, dv
// Tensor memory: S^T at 0, dP^T at 128, dV at 256, dK at 384.  P^T of the half h of
// the queries lies at 64 h, dS^T at 128 + 64 h (32 columns each).
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
tc_window_dkv_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmDo, BwdArgs a) {
    using L = BwdLayout<D>;
    constexpr int PN = D / 64;
    constexpr uint32_t kTile = L::kTile;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = align1024(smem_raw);
    const Bars bar = make_bars(sm + L::kBar);
    float *stats = reinterpret_cast<float *>(sm + L::kStats);   // [stage][2][128]
    const WinProblem &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // (the first key tiles first: they are seen by the most queries under a causal mask)
    const int unit = blockIdx.x % (p.B * p.Hkv), hk = unit % p.Hkv, b = unit / p.Hkv;
    const int j0 = blockIdx.x / (p.B * p.Hkv) * 128;
    const Sequence seq = sequence(p, b);
    int first, last;
    query_rows(p, seq, j0, j0 + 128, first, last);
    const int t0 = first / 128, nt = last > first ? (last + 127) / 128 - t0 : 0;
    const int n = nt * p.G;   // query tiles over the group's heads

    if (n == 0) {             // no query sees these keys (the same for the whole CTA)
        const int j = j0 + threadIdx.x;
        if (threadIdx.x < 128 && j < p.Nk) {
            zero_row(a.dk + b * a.g.dk.batch + hk * a.g.dk.head + (int64_t)j * a.g.dk.token, p.d);
            zero_row(a.dv + b * a.g.dv.batch + hk * a.g.dv.head + (int64_t)j * a.g.dv.token, p.d);
        }
        return;
    }
    if (threadIdx.x == 0) init_bars(bar);
    if (warp == 9) tmem_alloc(bar.tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *bar.tmem_slot;
    const WaitCtx w{a.limit, a.status, bar.abort_flag};

    if (warp == 8) {
        // ---------------- loads
        int issued[2] = {0, 0};
        if (lane == 0) {
            mbar_expect_tx(bar.fix_full, 2 * kTile);
            for (int pn = 0; pn < PN; pn++) {
                tma_load_4d(sm + L::kFix + pn * kPanel, &tmK, pn * 64, j0, hk, b, bar.fix_full);
                tma_load_4d(sm + L::kFix + kTile + pn * kPanel, &tmV, pn * 64, j0, hk, b,
                            bar.fix_full);
            }
        }
        for (int i = 0; i < n; i++) {
            const int st = i & 1;
            if (i >= 2 && !wait_warp(bar.stage_empty + st, ((i >> 1) - 1) & 1, w)) break;
            if (lane == 0) {
                const int h = hk * p.G + i / nt, i0 = (t0 + i % nt) * 128;
                uint8_t *dst = sm + L::kRing + st * 2 * kTile;
                mbar_expect_tx(bar.first_full + st, kTile);
                for (int pn = 0; pn < PN; pn++)
                    tma_load_4d(dst + pn * kPanel, &tmQ, pn * 64, i0, h, b, bar.first_full + st);
                mbar_expect_tx(bar.second_full + st, kTile);
                for (int pn = 0; pn < PN; pn++)
                    tma_load_4d(dst + kTile + pn * kPanel, &tmDo, pn * 64, i0, h, b,
                                bar.second_full + st);
            }
            issued[st]++;
        }
        if (lane == 0) drain_loads(bar, issued);
    } else if (warp == 9) {
        // ---------------- products
        constexpr uint32_t idS = idesc_bf16(128, 128, 0, 0);
        constexpr uint32_t idO = idesc_bf16(128, D, 0, 1);
        constexpr uint32_t kStageDesc = 2 * kTile >> 4, kHalfDesc = 64 * 128 >> 4;
        const uint64_t dK = smem_desc_sw128(smem_u32(sm + L::kFix), 16, 1024);
        const uint64_t dV = smem_desc_sw128(smem_u32(sm + L::kFix + kTile), 16, 1024);
        const uint64_t dQ = smem_desc_sw128(smem_u32(sm + L::kRing), 16, 1024);
        const uint64_t dO = smem_desc_sw128(smem_u32(sm + L::kRing + kTile), 16, 1024);
        const uint64_t dQt = smem_desc_sw128(smem_u32(sm + L::kRing), kPanel, 1024);
        const uint64_t dOt = smem_desc_sw128(smem_u32(sm + L::kRing + kTile), kPanel, 1024);
        auto issue_s = [&](int i) -> bool {
            const int st = i & 1;
            if (!spin_warp(bar.first_full + st, (i >> 1) & 1, w)) return false;
            tc_fence_after();
            mma_ss_head<D>(tmem, dK, dQ + st * kStageDesc, idS);
            mma_commit_warp(bar.s_full);
            return true;
        };
        auto issue_dp = [&](int i) -> bool {
            const int st = i & 1;
            if (!spin_warp(bar.second_full + st, (i >> 1) & 1, w)) return false;
            tc_fence_after();
            mma_ss_head<D>(tmem + 128, dV, dO + st * kStageDesc, idS);
            mma_commit_warp(bar.dp_full);
            return true;
        };
        bool ok = (!a.stall || spin_warp(bar.stall_bar, 0, w)) && spin_warp(bar.fix_full, 0, w);
        ok = ok && issue_s(0) && issue_dp(0);
        for (int i = 0; ok && i < n; i++) {
            const int st = i & 1;
            if (!(ok = spin_warp(bar.p_full, i & 1, w))) break;
            tc_fence_after();
            for (int h = 0; h < 2; h++)
                mma4_ts_mn64(tmem + 256, tmem + 64 * h, dOt + st * kStageDesc + h * kHalfDesc, idO,
                             i > 0 || h > 0 ? 1u : 0u);
            if (i + 1 < n && !(ok = issue_s(i + 1))) break;
            if (!(ok = spin_warp(bar.ds_full, i & 1, w))) break;
            tc_fence_after();
            for (int h = 0; h < 2; h++)
                mma4_ts_mn64(tmem + 384, tmem + 128 + 64 * h,
                             dQt + st * kStageDesc + h * kHalfDesc, idO, i > 0 || h > 0 ? 1u : 0u);
            mma_commit_warp(bar.stage_empty + st);
            if (i + 1 < n) ok = issue_dp(i + 1);
        }
        mma_commit_warp(bar.acc_full);
        wait_phase_cleanup(bar.acc_full, 0, kCleanupPolls);
    } else if (warp == 10) {
        // ---------------- lse (in log2 units) and delta of each tile's queries, negated
        for (int i = 0; i < n; i++) {
            const int st = i & 1;
            if (i >= 2 && !wait_warp(bar.stage_empty + st, ((i >> 1) - 1) & 1, w)) break;
            const int h = hk * p.G + i / nt, i0 = (t0 + i % nt) * 128;
            const int64_t row = ((int64_t)b * p.H + h) * p.Nq;
            float *dst = stats + st * 256;
#pragma unroll
            for (int x = lane; x < 128; x += 32) {
                const bool in = i0 + x < p.Nq;
                dst[x] = in ? -a.lse[row + i0 + x] * kLog2e : 0.f;
                dst[128 + x] = in ? -a.delta[row + i0 + x] : 0.f;
            }
            mbar_arrive_warp(bar.stats_full + st);
        }
    } else if (warp < 8) {
        // ---------------- elementwise: key row j, queries of one half of the tile
        const int half = warp >> 2, row = (warp & 3) * 32 + lane, j = j0 + row;
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 64 * half;
        int ilo, ihi, rfirst, rlast;
        query_rows(p, seq, j, j + 1, ilo, ihi);   // the queries that see this key
        real_rows(p, seq, 0, p.Nq, rfirst, rlast);
        bool ok = true;
        for (int i = 0; i < n; i++) {
            const int st = i & 1, i0 = (t0 + i % nt) * 128, c0 = i0 + 64 * half;
            const float *nl = stats + st * 256 + 64 * half, *nd = nl + 128;
            if (!(ok = wait_warp(bar.s_full, i & 1, w) &&
                       wait_warp(bar.stats_full + st, (i >> 1) & 1, w)))
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
            const int rl = min(rlast, p.Nq), rf = rfirst;
            if (i0 < rf || (rl < p.Nq && i0 + 128 > rl)) {
                // rows that are not real may hold anything, and 0 * NaN is NaN: they become
                // zeros before the products over the queries
                if (!(ok = wait_warp(bar.second_full + st, (i >> 1) & 1, w))) break;
                uint8_t *tile = sm + L::kRing + st * 2 * kTile;
                const int za = min(max(rf - i0, 0), 128), zb = min(max(rl - i0, 0), 128);
                const int id = half * 128 + row;
                zero_rows(tile, 0, za, PN, kPanel, id, 256);
                zero_rows(tile, zb, 128, PN, kPanel, id, 256);
                zero_rows(tile + kTile, 0, za, PN, kPanel, id, 256);
                zero_rows(tile + kTile, zb, 128, PN, kPanel, id, 256);
                fence_proxy_async_smem();
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive_warp(bar.p_full);
            if (!(ok = wait_warp(bar.dp_full, i & 1, w))) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
                float y[32];
                tmem_ld32f(tl + 128 + c, y);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    const ulonglong2 d2 = *reinterpret_cast<const ulonglong2 *>(nd + c + k);
                    const uint64_t u = f2_mul(f2_add(f2_pack(y[k], y[k + 1]), d2.x),
                                              f2_pack(x[c + k], x[c + k + 1]));
                    const uint64_t v = f2_mul(f2_add(f2_pack(y[k + 2], y[k + 3]), d2.y),
                                              f2_pack(x[c + k + 2], x[c + k + 3]));
                    f2_unpack(u, y[k], y[k + 1]);
                    f2_unpack(v, y[k + 2], y[k + 3]);
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
            mbar_arrive_warp(bar.ds_full);
        }
        if (ok && wait_warp(bar.acc_full, 0, w)) {
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
// Tensor memory: S at 0 and 128 (two buffers; dS over S, half h at + 64 h), dP at 256,
// dQ at 384.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
tc_window_dq_kernel(const __grid_constant__ CUtensorMap tmQ,
                    const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ CUtensorMap tmDo, BwdArgs a) {
    using L = BwdLayout<D>;
    constexpr int PN = D / 64;
    constexpr uint32_t kTile = L::kTile;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = align1024(smem_raw);
    const Bars bar = make_bars(sm + L::kBar);
    float *half_delta = reinterpret_cast<float *>(sm + L::kStats);   // [2 halves][128]
    const WinProblem &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the last tiles first: they see the most keys under a causal mask
    const int unit = blockIdx.x % (p.B * p.H), h = unit % p.H, b = unit / p.H;
    const int i0 = ((int)gridDim.x - 1 - (int)blockIdx.x) / (p.B * p.H) * 128;
    const Sequence seq = sequence(p, b);
    const KeyTiles kt = key_tiles<128>(p, seq, i0, i0 + 128);
    const int nt = kt.count();
    // the first n - nt steps only sum delta
    const int n = nt <= kExactTiles ? 2 * nt : nt;
    __nv_bfloat16 *const dq = a.dq + b * a.g.dq.batch + h * a.g.dq.head;

    if (n == 0) {
        const int i = i0 + threadIdx.x;
        if (threadIdx.x < 128 && i < p.Nq) zero_row(dq + (int64_t)i * a.g.dq.token, p.d);
        return;
    }
    if (threadIdx.x == 0) init_bars(bar);
    if (warp == 9) tmem_alloc(bar.tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *bar.tmem_slot;
    const WaitCtx w{a.limit, a.status, bar.abort_flag};

    if (warp == 8) {
        int issued[2] = {0, 0};
        if (lane == 0) {
            mbar_expect_tx(bar.fix_full, 2 * kTile);
            for (int pn = 0; pn < PN; pn++) {
                tma_load_4d(sm + L::kFix + pn * kPanel, &tmQ, pn * 64, i0, h, b, bar.fix_full);
                tma_load_4d(sm + L::kFix + kTile + pn * kPanel, &tmDo, pn * 64, i0, h, b,
                            bar.fix_full);
            }
        }
        for (int i = 0; i < n; i++) {
            const int st = i & 1;
            if (i >= 2 && !wait_warp(bar.stage_empty + st, ((i >> 1) - 1) & 1, w)) break;
            if (lane == 0) {
                const int j0 = kt.tile(i % nt) * 128;
                uint8_t *dst = sm + L::kRing + st * 2 * kTile;
                mbar_expect_tx(bar.first_full + st, kTile);
                for (int pn = 0; pn < PN; pn++)
                    tma_load_4d(dst + pn * kPanel, &tmK, pn * 64, j0, h / p.G, b,
                                bar.first_full + st);
                mbar_expect_tx(bar.second_full + st, kTile);
                for (int pn = 0; pn < PN; pn++)
                    tma_load_4d(dst + kTile + pn * kPanel, &tmV, pn * 64, j0, h / p.G, b,
                                bar.second_full + st);
            }
            issued[st]++;
        }
        if (lane == 0) drain_loads(bar, issued);
    } else if (warp == 9) {
        constexpr uint32_t idS = idesc_bf16(128, 128, 0, 0);
        constexpr uint32_t idO = idesc_bf16(128, D, 0, 1);
        constexpr uint32_t kStageDesc = 2 * kTile >> 4, kHalfDesc = 64 * 128 >> 4;
        const uint64_t dQ = smem_desc_sw128(smem_u32(sm + L::kFix), 16, 1024);
        const uint64_t dO = smem_desc_sw128(smem_u32(sm + L::kFix + kTile), 16, 1024);
        const uint64_t dK = smem_desc_sw128(smem_u32(sm + L::kRing), 16, 1024);
        const uint64_t dV = smem_desc_sw128(smem_u32(sm + L::kRing + kTile), 16, 1024);
        const uint64_t dKt = smem_desc_sw128(smem_u32(sm + L::kRing), kPanel, 1024);
        auto issue_s = [&](int i) -> bool {
            const int st = i & 1;
            if (!spin_warp(bar.first_full + st, (i >> 1) & 1, w)) return false;
            tc_fence_after();
            mma_ss_head<D>(tmem + 128 * st, dQ, dK + st * kStageDesc, idS);
            mma_commit_warp(bar.s_full + st);
            return true;
        };
        auto issue_dp = [&](int i) -> bool {
            const int st = i & 1;
            if (!spin_warp(bar.second_full + st, (i >> 1) & 1, w)) return false;
            tc_fence_after();
            mma_ss_head<D>(tmem + 256, dO, dV + st * kStageDesc, idS);
            mma_commit_warp(bar.dp_full);
            return true;
        };
        bool ok = (!a.stall || spin_warp(bar.stall_bar, 0, w)) && spin_warp(bar.fix_full, 0, w);
        ok = ok && issue_s(0) && issue_dp(0);
        if (ok && n > 1) ok = issue_s(1);
        for (int i = 0; ok && i < n; i++) {
            const int st = i & 1;
            // dS(i) is written: dP's columns have been read too
            if (!(ok = spin_warp(bar.ds_full, i & 1, w))) break;
            if (i + 1 < n && !(ok = issue_dp(i + 1))) break;
            tc_fence_after();
            for (int hh = 0; hh < 2 && i >= n - nt; hh++)
                mma4_ts_mn64(tmem + 384, tmem + 128 * st + 64 * hh,
                             dKt + st * kStageDesc + hh * kHalfDesc, idO,
                             i > n - nt || hh > 0 ? 1u : 0u);
            mma_commit_warp(bar.stage_empty + st);
            if (i + 2 < n) ok = issue_s(i + 2);
        }
        mma_commit_warp(bar.acc_full);
        wait_phase_cleanup(bar.acc_full, 0, kCleanupPolls);
    } else if (warp < 8) {
        const int half = warp >> 2, row = (warp & 3) * 32 + lane, i = i0 + row;
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 64 * half;
        const RowKeys rk = row_keys(p, seq, i);
        const int64_t at = ((int64_t)b * p.H + h) * p.Nq + i;
        const bool real = rk.hi > 0;
        const float nl = real ? -a.lse[at] * kLog2e : 0.f;
        float nd = real && n == nt ? -a.delta[at] : 0.f;
        const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2), nl2 = f2_pack(nl, nl);
        bool ok = true;
        for (int it = 0; it < n; it++) {
            const int st = it & 1, c0 = kt.tile(it % nt) * 128 + 64 * half;
            if (!(ok = wait_warp(bar.s_full + st, (it >> 1) & 1, w))) break;
            tc_fence_after();
            float x[64];
            tmem_ld32f(tl + 128 * st, &x[0]);
            tmem_ld32f(tl + 128 * st + 32, &x[32]);
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
            if (kt.tile(it % nt) * 128 + 128 > seq.len) {
                // keys past the sequence may hold anything, and 0 * NaN is NaN: they become
                // zeros before the product over the keys (S of this tile is done with them)
                zero_rows(sm + L::kRing + st * 2 * kTile, max(0, seq.len - kt.tile(it % nt) * 128), 128,
                          PN, kPanel, half * 128 + row, 256);
                fence_proxy_async_smem();
            }
            if (!(ok = wait_warp(bar.dp_full, it & 1, w))) break;
            tc_fence_after();
            if (it < n - nt) {
                // this half's part of delta = sum P dP; the halves meet in shared memory
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                    float y[32];
                    tmem_ld32f(tl + 256 + c, y);
                    tmem_wait_ld();
                    const uint32_t s = (uint32_t)(see >> c);
#pragma unroll
                    for (int k = 0; k < 32; k++)
                        sum = fmaf((s >> k) & 1 ? x[c + k] : 0.f, (s >> k) & 1 ? y[k] : 0.f, sum);
                }
                nd -= sum;
                if (it == n - nt - 1) {
                    half_delta[half * 128 + row] = nd;
                    mbar_arrive_warp(bar.p_full);
                    if (!(ok = wait_warp(bar.p_full, 0, w))) break;
                    nd = half_delta[row] + half_delta[128 + row];
                    if (half == 0 && real) a.delta[at] = -nd;
                }
                tc_fence_before();
                mbar_arrive_warp(bar.ds_full);
                continue;
            }
            const uint64_t nd2 = f2_pack(nd, nd);
            uint32_t pk[32];
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
                float y[32];
                tmem_ld32f(tl + 256 + c, y);
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
            tmem_st32(tl + 128 * st, pk);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive_warp(bar.ds_full);
        }
        if (ok && wait_warp(bar.acc_full, 0, w)) {
            tc_fence_after();
            const int x = half * (D / 2);
            store_row<D / 2>(tmem + ((uint32_t)((warp & 3) * 32) << 16) + 384 + x,
                             dq + (int64_t)i * a.g.dq.token + x, p.scale, p.d - x, i < p.Nq);
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
    CUtensorMap mq, mk, mv, md;
    if (!map_tokens(&mq, q, p.q, p.B, p.H, p.Nq, p.d, 128) ||
        !map_tokens(&mk, k, p.k, p.B, p.Hkv, p.Nk, p.d, 128) ||
        !map_tokens(&mv, v, p.v, p.B, p.Hkv, p.Nk, p.d, 128) ||
        !map_tokens(&md, dout, g.dout, p.B, p.H, p.Nq, p.d, 128))
        return cudaErrorInvalidValue;
    constexpr uint32_t smem = BwdLayout<D>::kSmem;
    cudaError_t e = tcs::set_smem(tc_window_dkv_kernel<D>, smem);
    if (e == cudaSuccess) e = tcs::set_smem(tc_window_dq_kernel<D>, smem);
    if (e != cudaSuccess) return e;
    const unsigned gk = (unsigned)p.B * p.Hkv * ((p.Nk + 127) / 128);
    const unsigned gq = (unsigned)p.B * p.H * ((p.Nq + 127) / 128);
    // dq first: it completes delta
    tc_window_dq_kernel<D><<<gq, kThreads, smem, stream>>>(mq, mk, mv, md, a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    tc_window_dkv_kernel<D><<<gk, kThreads, smem, stream>>>(mq, mk, mv, md, a);
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
