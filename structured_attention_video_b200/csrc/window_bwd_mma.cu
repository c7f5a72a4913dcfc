// window_bwd_mma.cu -- backward of the window attention in bfloat16 on mma.sync (float32
// sums; P and dS rounded to bfloat16 as operands of the accumulating products, from 32-bit
// values).
//
//   P = exp2(scale_log2 S - lse log2(e)),  dS = P (dO V^T - delta),
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K.
//
// Two kernels, so that every gradient is summed by one warp in a fixed order (no atomics) at
// the price of forming S and dO V^T twice (7 products instead of 5):
//   mma_dq_kernel    64 queries of one head against their 64-key tiles;
//   mma_dkv_kernel   64 keys of one key head against the query blocks of every head of its
//                    group that see them.
// Four warps of 16 rows each.  A warp's logits stay in its registers: the accumulator of the
// first product is, packed, the left operand of the second.  Tiles of the other side come
// through two stages of asynchronous copies, in rows padded by 16 bytes, so that eight rows of
// an ldmatrix cover all banks.
//
// Not on tcgen05.  A form with tensor memory and TMA (dq and dk/dv with two issuing threads
// and sixteen elementwise warps) took 1.2 ms instead of 6.4 on nine 480p frames, but about one
// call in 400 on small ragged batches ended in an illegal address, its cause not found by
// reading, and with checks in the kernels it did not show.  These kernels have no waits, no
// tensor memory and no asynchronous copy that outlives its CTA.
//
// Bound by the products of mma.sync (45 to 47% of that pipe, about 540 TFLOP/s at most) with
// the reads of their fragments from shared memory close behind.  Nine 480p frames, each seeing
// four, 12 heads, d = 128: dq 2.81 ms, dk/dv 3.59; 2 x 1023 causal tokens, 8 heads on 2 key
// heads, d = 64: 40, 41 and 5 us for the join.
//
// delta comes from out as the forward rounded it, an error of 2^-8 |dO.O| at most.  A
// row of n keys of like weight has |O| of about n^(-1/2) |v|, so against dP it matters
// for few keys only.  Query tiles of up to kExactTiles key tiles therefore first walk their
// keys once for delta = sum P dP from the same products that form dS, and the dq kernel
// runs first to hand it to the dk/dv kernel.
#include "window_mma.cuh"
#include "window_tc.cuh"

namespace monarch {
namespace win {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 128, kRows = 64;
constexpr int kExactTiles = 6;

// Elements between rows in shared memory.
template <int D> constexpr int kPitch = D + 8;
// Queries of one block of the dk/dv kernel: at d = 128 its accumulators leave room for 32.
template <int D> constexpr int kBlock = D == 128 ? 32 : 64;

struct BwdArgs {
    WinProblem p;
    WinGrads g;
    const float *lse;
    float *delta;   // of the real rows, from the dq kernel
    const __nv_bfloat16 *q, *k, *v, *out, *dout;
    __nv_bfloat16 *dq, *dk, *dv;
    int splits;     // parts of a key tile's query blocks, a CTA each (dkv)
    float *parts;   // splits > 1: [key tile, batch, head][split][64][dV | dK]
    int *status;
    long long limit;
    int stall;
};

// Rows [r0, r0 + R) of a [tokens][D] matrix into shared memory, asynchronously; rows outside
// [low, high) become zero.
template <int D, int R>
__device__ __forceinline__ void load_rows(__nv_bfloat16 *sm, const __nv_bfloat16 *base,
                                          int64_t stride, int r0, int low, int high) {
    constexpr int kChunks = D / 8;
#pragma unroll
    for (int x = threadIdx.x; x < R * kChunks; x += kThreads) {
        const int r = x / kChunks, c = x % kChunks;
        const bool in = r0 + r >= low && r0 + r < high;
        const __nv_bfloat16 *src = base + (in ? (int64_t)(r0 + r) * stride + c * 8 : 0);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         smem_u32(sm + r * kPitch<D> + c * 8)),
                     "l"(src), "r"(in ? 16 : 0)
                     : "memory");
    }
}

// s = A B^T: 16 rows of a (this warp's) against NT x 8 rows of b, over D columns.
template <int D, int NT>
__device__ __forceinline__ void product_nt(float (&s)[NT][4], uint32_t a, uint32_t b, int lane) {
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
        for (int c = 0; c < 4; c++) s[j][c] = 0.f;
    const int r8 = lane & 7, mi = lane >> 3;
    const uint32_t ar = a + (((mi & 1) * 8 + r8) * kPitch<D> + (mi >> 1) * 8) * 2;
    const uint32_t br = b + (((mi >> 1) * 8 + r8) * kPitch<D> + (mi & 1) * 8) * 2;
#pragma unroll
    for (int kk = 0; kk < D / 16; kk++) {
        uint32_t af[4];
        ldmatrix4(af, ar + kk * 32);
#pragma unroll
        for (int j = 0; j < NT / 2; j++) {
            uint32_t bf[4];
            ldmatrix4(bf, br + j * 16 * kPitch<D> * 2 + kk * 32);
            mma16816(s[2 * j], af, bf[0], bf[1]);
            mma16816(s[2 * j + 1], af, bf[2], bf[3]);
        }
    }
}

// o += W B: W 16 x (NT x 8), packed from an accumulator; b NT x 8 rows of D columns.
template <int D, int NT>
__device__ __forceinline__ void product_nn(float (&o)[D / 8][4], const float (&w)[NT][4], uint32_t b,
                                           int lane) {
    const int r8 = lane & 7, mi = lane >> 3;
    const uint32_t br = b + (((mi & 1) * 8 + r8) * kPitch<D> + (mi >> 1) * 8) * 2;
#pragma unroll
    for (int j = 0; j < NT / 2; j++) {
        const uint32_t af[4] = {pack_bf16(w[2 * j][0], w[2 * j][1]),
                                pack_bf16(w[2 * j][2], w[2 * j][3]),
                                pack_bf16(w[2 * j + 1][0], w[2 * j + 1][1]),
                                pack_bf16(w[2 * j + 1][2], w[2 * j + 1][3])};
#pragma unroll
        for (int x = 0; x < D / 16; x++) {
            uint32_t bf[4];
            ldmatrix4_trans(bf, br + (j * 16 * kPitch<D> + x * 16) * 2);
            mma16816(o[2 * x], af, bf[0], bf[1]);
            mma16816(o[2 * x + 1], af, bf[2], bf[3]);
        }
    }
}

// This warp's 16 x D accumulator times `scale` to global memory through its 16 rows of
// shared memory; rows from `valid` on are not there.
template <int D>
__device__ __forceinline__ void store_rows(__nv_bfloat16 *sm, const float (&o)[D / 8][4], float scale,
                                           __nv_bfloat16 *base, int64_t stride, int r0, int valid,
                                           int lane) {
    const int n = lane >> 2, t = lane & 3;
    __syncwarp();
#pragma unroll
    for (int x = 0; x < D / 8; x++)
#pragma unroll
        for (int y = 0; y < 2; y++)
            *reinterpret_cast<uint32_t *>(sm + (n + 8 * y) * kPitch<D> + x * 8 + 2 * t) =
                pack_bf16(o[x][2 * y] * scale, o[x][2 * y + 1] * scale);
    __syncwarp();
    for (int x = lane; x < 16 * (D / 8); x += 32) {
        const int r = x / (D / 8), c = x % (D / 8) * 8;
        if (r0 + r < valid)
            *reinterpret_cast<uint4 *>(base + (int64_t)(r0 + r) * stride + c) =
                *reinterpret_cast<const uint4 *>(sm + r * kPitch<D> + c);
    }
}

// The product of 8 elements of two rows.
__device__ __forceinline__ float dot8(const __nv_bfloat16 *a, const __nv_bfloat16 *b) {
    const uint4 x = *reinterpret_cast<const uint4 *>(a), y = *reinterpret_cast<const uint4 *>(b);
    const uint32_t u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        sum = fmaf(__uint_as_float(u[i] << 16), __uint_as_float(v[i] << 16), sum);
        sum = fmaf(__uint_as_float(u[i] & 0xFFFF0000u), __uint_as_float(v[i] & 0xFFFF0000u), sum);
    }
    return sum;
}

// Rows [r0, r0 + 64) become zero, those below `valid`.
template <int D>
__device__ __forceinline__ void zero_rows64(__nv_bfloat16 *base, int64_t stride, int r0, int valid) {
    for (int x = threadIdx.x; x < kRows * (D / 8); x += kThreads) {
        const int r = r0 + x / (D / 8);
        if (r < valid)
            *reinterpret_cast<uint4 *>(base + (int64_t)r * stride + x % (D / 8) * 8) =
                make_uint4(0, 0, 0, 0);
    }
}

// Fault injection: a wait on a barrier that nothing completes, until it gives up and says so.
__device__ __forceinline__ void stalled(const BwdArgs &a) {
    __shared__ uint64_t never;
    __shared__ int abort_flag;
    if (threadIdx.x != 0) return;
    abort_flag = 0;
    mbar_init(&never, 1);
    fence_mbar_init();
    wait_phase(&never, 0, WaitCtx{a.limit, a.status, &abort_flag});
}

// ---------------------------------------------------------------- dq
template <int D> constexpr uint32_t dq_smem() { return 6 * kRows * kPitch<D> * 2; }

template <int D>
__global__ void __launch_bounds__(kThreads, 2) mma_dq_kernel(BwdArgs a) {
    extern __shared__ __align__(16) __nv_bfloat16 smb[];
    constexpr int kTile = kRows * kPitch<D>, NT = 8;
    __nv_bfloat16 *sq = smb, *sdo = sq + kTile, *skv = sdo + kTile;   // [stage][K, V]
    __shared__ Sequence shared_seq;
    const WinProblem &p = a.p;
    if (a.stall) return stalled(a);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = lane >> 2, t = lane & 3;
    // the last tiles first: they see the most keys under a causal mask
    const int unit = blockIdx.x % (p.B * p.H), h = unit % p.H, b = unit / p.H;
    const int i0 = ((int)gridDim.x - 1 - (int)blockIdx.x) / (p.B * p.H) * kRows;
    Sequence seq = first_threads_sequence(p, b);
    share_sequence(seq, &shared_seq);
    const KeyTiles kt = key_tiles<64>(p, seq, i0, i0 + kRows);
    const int nt = kt.count();
    const bool exact = nt <= kExactTiles;
    const int total = exact ? 2 * nt : nt;   // the first total - nt tiles only sum delta
    __nv_bfloat16 *const dq = a.dq + b * a.g.dq.batch + h * a.g.dq.head;
    if (nt == 0) {   // (the same for the whole CTA)
        zero_rows64<D>(dq, a.g.dq.token, i0, p.Nq);
        return;
    }
    const __nv_bfloat16 *kb = a.k + b * p.k.batch + (h / p.G) * p.k.head;
    const __nv_bfloat16 *vb = a.v + b * p.v.batch + (h / p.G) * p.v.head;
    auto load = [&](int u) {
        const int j0 = kt.tile(u < nt ? u : u - nt) * 64;
        __nv_bfloat16 *dst = skv + (u & 1) * 2 * kTile;
        load_rows<D, 64>(dst, kb, p.k.token, j0, 0, seq.len);
        load_rows<D, 64>(dst + kTile, vb, p.v.token, j0, 0, seq.len);
    };
    load_rows<D, kRows>(sq, a.q + b * p.q.batch + h * p.q.head, p.q.token, i0, 0, p.Nq);
    load_rows<D, kRows>(sdo, a.dout + b * a.g.dout.batch + h * a.g.dout.head, a.g.dout.token, i0, 0,
                        p.Nq);
    load(0);
    copies_commit();

    // rows n and n + 8 of the warp's 16
    RowKeys rk[2];
    float nl[2], dl[2], sum[2] = {0.f, 0.f};
#pragma unroll
    for (int y = 0; y < 2; y++) {
        const int i = i0 + warp * 16 + n + 8 * y;
        const int64_t at = ((int64_t)b * p.H + h) * p.Nq + i;
        rk[y] = row_keys(p, seq, i);
        const bool real = rk[y].hi > 0;
        nl[y] = real ? a.lse[at] * kLog2e : 0.f;
        dl[y] = 0.f;
        if (real && !exact) {   // a quarter of the row a lane
            const __nv_bfloat16 *po = a.out + b * p.o.batch + h * p.o.head + i * p.o.token;
            const __nv_bfloat16 *pd =
                a.dout + b * a.g.dout.batch + h * a.g.dout.head + i * a.g.dout.token;
#pragma unroll
            for (int c = 8 * t; c < D; c += 32) dl[y] += dot8(po + c, pd + c);
        }
        dl[y] += __shfl_xor_sync(0xffffffffu, dl[y], 1);
        dl[y] += __shfl_xor_sync(0xffffffffu, dl[y], 2);
        if (t == 0 && real && !exact) a.delta[at] = dl[y];
    }
    float o[D / 8][4];
#pragma unroll
    for (int x = 0; x < D / 8; x++)
#pragma unroll
        for (int c = 0; c < 4; c++) o[x][c] = 0.f;
    const uint32_t aq = smem_u32(sq + warp * 16 * kPitch<D>);
    const uint32_t ado = smem_u32(sdo + warp * 16 * kPitch<D>);
    for (int u = 0; u < total; u++) {
        const int j0 = kt.tile(u < nt ? u : u - nt) * 64;
        __syncthreads();   // the other stage's last readers are done
        if (u + 1 < total) load(u + 1);
        copies_commit();
        copies_wait<1>();
        __syncthreads();
        if (exact && u == nt) {   // delta of both rows, over the four lanes of each
#pragma unroll
            for (int y = 0; y < 2; y++) {
                sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], 1);
                sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], 2);
                dl[y] = sum[y];
                const int i = i0 + warp * 16 + n + 8 * y;
                if (t == 0 && rk[y].hi > 0) a.delta[((int64_t)b * p.H + h) * p.Nq + i] = dl[y];
            }
        }
        const uint32_t sk = smem_u32(skv + (u & 1) * 2 * kTile), sv = sk + kTile * 2;
        float s[NT][4], dp[NT][4];
        product_nt<D, NT>(s, aq, sk, lane);
        product_nt<D, NT>(dp, ado, sv, lane);
        const bool first_pass = u < total - nt;
#pragma unroll
        for (int j = 0; j < NT; j++)
#pragma unroll
            for (int c = 0; c < 4; c++) {
                const int y = c >> 1;
                const bool see = rk[y].sees(j0 + 8 * j + 2 * t + (c & 1));
                const float e = fast_exp2(fmaf(s[j][c], p.scale_log2, -nl[y]));
                if (first_pass)
                    sum[y] += see ? e * dp[j][c] : 0.f;
                else
                    dp[j][c] = see ? e * (dp[j][c] - dl[y]) : 0.f;
            }
        if (!first_pass) product_nn<D, NT>(o, dp, sk, lane);
    }
    copies_wait<0>();
    // (rows that are not real have dS = 0 and so zeros)
    store_rows<D>(sq + warp * 16 * kPitch<D>, o, p.scale, dq, a.g.dq.token, i0 + warp * 16, p.Nq,
                  lane);
}

// ---------------------------------------------------------------- dk, dv
template <int D> constexpr uint32_t dkv_smem() {
    return (2 * kRows + 4 * kBlock<D>) * kPitch<D> * 2 + 4 * kBlock<D> * 4;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) mma_dkv_kernel(BwdArgs a) {
    extern __shared__ __align__(16) __nv_bfloat16 smb[];
    constexpr int Q = kBlock<D>, NT = Q / 8, kTile = kRows * kPitch<D>, kQTile = Q * kPitch<D>;
    __nv_bfloat16 *sk = smb, *sv = sk + kTile, *sqd = sv + kTile;   // [stage][Q, dO]
    float *stats = reinterpret_cast<float *>(sqd + 4 * kQTile);     // [stage][lse, delta][Q]
    __shared__ Sequence shared_seq;
    const WinProblem &p = a.p;
    if (a.stall) return stalled(a);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = lane >> 2, t = lane & 3;
    // (the first key tiles first: they are seen by the most queries under a causal mask)
    const int tile_unit = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
    const int unit = tile_unit % (p.B * p.Hkv), hk = unit % p.Hkv, b = unit / p.Hkv;
    const int j0 = tile_unit / (p.B * p.Hkv) * kRows;
    Sequence seq = first_threads_sequence(p, b);
    share_sequence(seq, &shared_seq);
    int first, last, rfirst, rlast;
    query_rows(p, seq, j0, j0 + kRows, first, last);
    real_rows(p, seq, 0, p.Nq, rfirst, rlast);
    const int t0 = first / Q, nt = last > first ? (last + Q - 1) / Q - t0 : 0;
    // query blocks over the group's heads; this CTA's
    const int u0 = (int)((int64_t)nt * p.G * split / a.splits);
    const int u1 = (int)((int64_t)nt * p.G * (split + 1) / a.splits);
    __nv_bfloat16 *const dk = a.dk + b * a.g.dk.batch + hk * a.g.dk.head;
    __nv_bfloat16 *const dv = a.dv + b * a.g.dv.batch + hk * a.g.dv.head;
    if (nt == 0 && a.splits == 1) {   // no query sees these keys (the same for the whole CTA)
        zero_rows64<D>(dk, a.g.dk.token, j0, p.Nk);
        zero_rows64<D>(dv, a.g.dv.token, j0, p.Nk);
        return;
    }
    auto load = [&](int u) {
        const int st = u & 1, h = hk * p.G + u / nt, i0 = (t0 + u % nt) * Q;
        __nv_bfloat16 *dst = sqd + st * 2 * kQTile;
        // rows that are not real enter as zeros, whatever they hold
        load_rows<D, Q>(dst, a.q + b * p.q.batch + h * p.q.head, p.q.token, i0, rfirst, rlast);
        load_rows<D, Q>(dst + kQTile, a.dout + b * a.g.dout.batch + h * a.g.dout.head,
                        a.g.dout.token, i0, rfirst, rlast);
        if (threadIdx.x < Q) {
            const int i = i0 + threadIdx.x;
            const bool real = i >= rfirst && i < rlast;
            const int64_t at = ((int64_t)b * p.H + h) * p.Nq + i;
            stats[st * 2 * Q + threadIdx.x] = real ? a.lse[at] * kLog2e : 0.f;
            stats[st * 2 * Q + Q + threadIdx.x] = real ? a.delta[at] : 0.f;
        }
    };
    load_rows<D, kRows>(sk, a.k + b * p.k.batch + hk * p.k.head, p.k.token, j0, 0, seq.len);
    load_rows<D, kRows>(sv, a.v + b * p.v.batch + hk * p.v.head, p.v.token, j0, 0, seq.len);
    if (u0 < u1) load(u0);
    copies_commit();
    // the queries that see keys n and n + 8 of the warp's 16
    int ilo[2], ihi[2];
#pragma unroll
    for (int y = 0; y < 2; y++) {
        const int j = j0 + warp * 16 + n + 8 * y;
        query_rows(p, seq, j, j + 1, ilo[y], ihi[y]);
    }
    float ok[D / 8][4], ov[D / 8][4];
#pragma unroll
    for (int x = 0; x < D / 8; x++)
#pragma unroll
        for (int c = 0; c < 4; c++) ok[x][c] = ov[x][c] = 0.f;
    const uint32_t ak = smem_u32(sk + warp * 16 * kPitch<D>);
    const uint32_t av = smem_u32(sv + warp * 16 * kPitch<D>);
    for (int u = u0; u < u1; u++) {
        const int st = u & 1, i0 = (t0 + u % nt) * Q;
        __syncthreads();   // the other stage's last readers are done
        if (u + 1 < u1) load(u + 1);
        copies_commit();
        copies_wait<1>();
        __syncthreads();
        const uint32_t bq = smem_u32(sqd + st * 2 * kQTile), bdo = bq + kQTile * 2;
        const float *ls = stats + st * 2 * Q, *ds = ls + Q;
        float s[NT][4], dp[NT][4];
        product_nt<D, NT>(s, ak, bq, lane);
        product_nt<D, NT>(dp, av, bdo, lane);
#pragma unroll
        for (int j = 0; j < NT; j++)
#pragma unroll
            for (int c = 0; c < 4; c++) {
                const int y = c >> 1, x = 8 * j + 2 * t + (c & 1);
                const bool see = i0 + x >= ilo[y] && i0 + x < ihi[y];
                const float e = see ? fast_exp2(fmaf(s[j][c], p.scale_log2, -ls[x])) : 0.f;
                s[j][c] = e;
                dp[j][c] = see ? e * (dp[j][c] - ds[x]) : 0.f;
            }
        product_nn<D, NT>(ov, s, bdo, lane);
        product_nn<D, NT>(ok, dp, bq, lane);
    }
    copies_wait<0>();
    if (a.splits > 1) {
        float *dst = a.parts + ((int64_t)blockIdx.x * kRows + warp * 16) * 2 * D;
#pragma unroll
        for (int x = 0; x < D / 8; x++)
#pragma unroll
            for (int y = 0; y < 2; y++) {
                float *row = dst + (n + 8 * y) * 2 * D + x * 8 + 2 * t;
                *reinterpret_cast<float2 *>(row) = make_float2(ov[x][2 * y], ov[x][2 * y + 1]);
                *reinterpret_cast<float2 *>(row + D) = make_float2(ok[x][2 * y], ok[x][2 * y + 1]);
            }
        return;
    }
    // (keys past the sequence are seen by no query: zeros)
    __syncthreads();
    store_rows<D>(sk + warp * 16 * kPitch<D>, ok, p.scale, dk, a.g.dk.token, j0 + warp * 16, p.Nk,
                  lane);
    store_rows<D>(sv + warp * 16 * kPitch<D>, ov, 1.f, dv, a.g.dv.token, j0 + warp * 16, p.Nk, lane);
}

// dk and dv from the parts of each key tile's query blocks, added in order.
template <int D>
__global__ void __launch_bounds__(256) mma_dkv_join_kernel(BwdArgs a) {
    const WinProblem &p = a.p;
    const int tile_unit = blockIdx.x, unit = tile_unit % (p.B * p.Hkv);
    const int hk = unit % p.Hkv, b = unit / p.Hkv, j0 = tile_unit / (p.B * p.Hkv) * kRows;
    const float *base = a.parts + (int64_t)tile_unit * a.splits * kRows * 2 * D;
    const int at = blockIdx.y * 256 + threadIdx.x;   // 4 columns of a row
    const int row = at / (2 * D / 4), x = at % (2 * D / 4) * 4, j = j0 + row;
    const bool is_k = x >= D;
    const int col = is_k ? x - D : x;
    if (row >= kRows || j >= p.Nk) return;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < a.splits; s++) {
        const float4 y =
            *reinterpret_cast<const float4 *>(base + ((int64_t)s * kRows + row) * 2 * D + x);
        sum.x += y.x, sum.y += y.y, sum.z += y.z, sum.w += y.w;
    }
    const float f = is_k ? p.scale : 1.f;
    __nv_bfloat16 *dst = is_k ? a.dk + b * a.g.dk.batch + hk * a.g.dk.head + (int64_t)j * a.g.dk.token
                              : a.dv + b * a.g.dv.batch + hk * a.g.dv.head + (int64_t)j * a.g.dv.token;
    *reinterpret_cast<uint2 *>(dst + col) =
        make_uint2(pack_bf16(sum.x * f, sum.y * f), pack_bf16(sum.z * f, sum.w * f));
}

template <int D> cudaError_t launch(const BwdArgs &a, cudaStream_t stream) {
    const WinProblem &p = a.p;
    cudaError_t e = tcs::set_smem(mma_dq_kernel<D>, dq_smem<D>());
    if (e == cudaSuccess) e = tcs::set_smem(mma_dkv_kernel<D>, dkv_smem<D>());
    if (e != cudaSuccess) return e;
    const unsigned key_tiles = (unsigned)p.B * p.Hkv * ((p.Nk + kRows - 1) / kRows);
    const unsigned query_tiles = (unsigned)p.B * p.H * ((p.Nq + kRows - 1) / kRows);
    // dq first: it completes delta
    mma_dq_kernel<D><<<query_tiles, kThreads, dq_smem<D>(), stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    mma_dkv_kernel<D><<<key_tiles * a.splits, kThreads, dkv_smem<D>(), stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess || a.splits == 1) return e;
    mma_dkv_join_kernel<D><<<dim3(key_tiles, (kRows * 2 * D / 4 + 255) / 256), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

// Parts of a key tile's query blocks in the dk/dv kernel: where the key tiles are fewer than
// two CTAs an SM, as many as fill those, of four blocks at least (a part's prologue, its
// store and the join cost about two).
int dkv_splits(const WinProblem &p) {
    const int64_t tiles = (int64_t)p.B * p.Hkv * ((p.Nk + kRows - 1) / kRows);
    const int block = p.d == 128 ? kBlock<128> : kBlock<64>;
    const int64_t blocks = (int64_t)((p.Nq + block - 1) / block) * p.G;
    const int64_t fill = 2 * tcs::sm_count() / tiles;
    return (int)max((int64_t)1, min(fill, blocks / 4));
}

}  // namespace

size_t mma_backward_bytes(const WinProblem &p) {
    const int splits = dkv_splits(p);
    if (splits == 1) return 0;
    const size_t tiles = (size_t)p.B * p.Hkv * ((p.Nk + kRows - 1) / kRows);
    return tiles * splits * kRows * 2 * p.d * sizeof(float);
}

cudaError_t mma_backward(const WinProblem &p, const WinGrads &g, const void *q, const void *k,
                         const void *v, const void *out, const float *lse, float *delta,
                         const void *dout, void *dq, void *dk, void *dv, void *parts, int *status,
                         long long limit, cudaStream_t stream) {
    BwdArgs a;
    a.p = p;
    a.g = g;
    a.lse = lse;
    a.delta = delta;
    a.q = (const __nv_bfloat16 *)q;
    a.k = (const __nv_bfloat16 *)k;
    a.v = (const __nv_bfloat16 *)v;
    a.out = (const __nv_bfloat16 *)out;
    a.dout = (const __nv_bfloat16 *)dout;
    a.dq = (__nv_bfloat16 *)dq;
    a.dk = (__nv_bfloat16 *)dk;
    a.dv = (__nv_bfloat16 *)dv;
    a.splits = dkv_splits(p);
    a.parts = (float *)parts;
    a.status = status;
    a.limit = limit;
    a.stall = device_inject_stall();
    return p.d == 32   ? launch<32>(a, stream)
           : p.d == 64 ? launch<64>(a, stream)
                       : launch<128>(a, stream);
}

}  // namespace win
}  // namespace monarch
