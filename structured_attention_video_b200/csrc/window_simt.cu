// window_simt.cu -- window attention in 32-bit arithmetic on the FMA pipes, forward
// and backward (float32 inputs; the tensor cores round operands to fewer bits).
//
// One CTA of 256 threads takes 16 RT rows of one side (queries; keys for dk and dv)
// and walks tiles of the other side.  Thread (ty, tx) of a 16 x 16 grid owns rows
// RT ty .. RT ty + RT - 1: in the logit products columns tx, tx + 16, ..., in the
// accumulating products d/16 columns of the head dimension.  The products run on
// packed pairs of float32 (fma.rn.f32x2).  The 16 threads of a row are half a warp,
// so softmax rows reduce with shuffles and the probabilities pass from the first
// product to the second through shared memory without a CTA barrier.
// No atomics: each output element is summed by one thread in a fixed order.
//
// Bound by the FMA pipes (128 a clock and SM, packed or not) with shared memory close
// behind: a step of 4 columns reads 12 rows' wavefronts for 16 clocks of FMAs.  8 heads of
// 4096 tokens, all keys seen: forward 34 TFLOP/s at d = 128, 30 at 64, 26 at 32; backward 22.5, 21
// and 18.  Rejected: lanes of 4 x 8 logits, which halve those reads (d = 128 backward
// 7.6 -> 9.2 ms, 1024 tokens at d = 64 forward 111 -> 173 us: fewer, longer-lived rows a warp).
#include "tc_primitives.cuh"
#include "window_common.cuh"

namespace monarch {
namespace win {
namespace {

using tc::f2_add;
using tc::f2_fma;
using tc::f2_mul;
using tc::f2_pack;
using tc::f2_unpack;

constexpr float kLn2 = 0.6931471805599453f;

// Shared-memory row of D floats, padded so that 16-byte reads of 8 consecutive rows
// cover all banks.
template <int D> constexpr int kPitch = D + 4;

// Rows [r0, r0 + R) of a [tokens][D] matrix into shared memory, asynchronously (16-byte
// copies of one group per thread); rows outside [low, valid) become zero.
template <int D, int R>
__device__ __forceinline__ void load_rows(float *sm, const float *base, int64_t stride, int r0,
                                          int valid, int low = 0) {
    constexpr int kChunks = D / 4;
    for (int i = threadIdx.x; i < R * kChunks; i += 256) {
        const int r = i / kChunks, c = i % kChunks;
        const bool in = r0 + r >= low && r0 + r < valid;
        const float *src = base + (in ? (int64_t)(r0 + r) * stride + c * 4 : 0);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         tc::smem_u32(sm + r * kPitch<D> + c * 4)),
                     "l"(src), "r"(in ? 16 : 0)
                     : "memory");
    }
}
// Two stages of the streamed tiles, the next one's copies behind this one's arithmetic,
// where two CTAs with them fit on an SM; at d = 128 two CTAs of one stage do instead.
template <int D> constexpr int kStages = D == 128 ? 1 : 2;

// s[i][j] = row (RT ty + i) of a . row (tx + 16 j) of b.
template <int D, int RT, int NC>
__device__ __forceinline__ void dot_tile(const float *a, const float *b, int ty, int tx,
                                         float (&s)[RT][NC]) {
    uint64_t acc[RT][NC];
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
        for (int j = 0; j < NC; j++) acc[i][j] = 0;
    const float *ap = a + RT * ty * kPitch<D>, *bp = b + tx * kPitch<D>;
#pragma unroll 4
    for (int x = 0; x < D; x += 4) {
        ulonglong2 av[RT], bv[NC];
#pragma unroll
        for (int i = 0; i < RT; i++)
            av[i] = *reinterpret_cast<const ulonglong2 *>(ap + i * kPitch<D> + x);
#pragma unroll
        for (int j = 0; j < NC; j++)
            bv[j] = *reinterpret_cast<const ulonglong2 *>(bp + j * 16 * kPitch<D> + x);
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
            for (int j = 0; j < NC; j++) {
                acc[i][j] = f2_fma(av[i].x, bv[j].x, acc[i][j]);
                acc[i][j] = f2_fma(av[i].y, bv[j].y, acc[i][j]);
            }
    }
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
        for (int j = 0; j < NC; j++) {
            float lo, hi;
            f2_unpack(acc[i][j], lo, hi);
            s[i][j] = lo + hi;
        }
}

// Columns of the head dimension that thread tx owns: pair q of D/32 covers
// columns 2 tx + 32 q and the next.
// o[i][q] += sum over the C columns of w of w[RT ty + i][c] * b[c][columns].
template <int D, int RT, int C, int PW>
__device__ __forceinline__ void add_product(const float *w, const float *b, int ty, int tx,
                                            uint64_t (&o)[RT][D / 32]) {
    const float *wp = w + RT * ty * PW, *bp = b + 2 * tx;
#pragma unroll 2
    for (int c = 0; c < C; c += 4) {
        float4 wv[RT];
#pragma unroll
        for (int i = 0; i < RT; i++) wv[i] = *reinterpret_cast<const float4 *>(wp + i * PW + c);
#pragma unroll
        for (int cc = 0; cc < 4; cc++) {
            uint64_t bv[D / 32];
#pragma unroll
            for (int q = 0; q < D / 32; q++)
                bv[q] = *reinterpret_cast<const uint64_t *>(bp + (c + cc) * kPitch<D> + 32 * q);
#pragma unroll
            for (int i = 0; i < RT; i++) {
                const float x = cc == 0 ? wv[i].x : cc == 1 ? wv[i].y : cc == 2 ? wv[i].z : wv[i].w;
                const uint64_t xx = f2_pack(x, x);
#pragma unroll
                for (int q = 0; q < D / 32; q++) o[i][q] = f2_fma(xx, bv[q], o[i][q]);
            }
        }
    }
}

template <int D, int RT>
__device__ __forceinline__ void store_rows(float *base, int64_t stride, int r0, int valid, int ty,
                                           int tx, const uint64_t (&o)[RT][D / 32],
                                           const float (&scale)[RT]) {
#pragma unroll
    for (int i = 0; i < RT; i++) {
        const int r = r0 + RT * ty + i;
        if (r >= valid) continue;
#pragma unroll
        for (int q = 0; q < D / 32; q++) {
            float lo, hi;
            f2_unpack(o[i][q], lo, hi);
            *reinterpret_cast<float2 *>(base + (int64_t)r * stride + 2 * tx + 32 * q) =
                make_float2(lo * scale[i], hi * scale[i]);
        }
    }
}

__device__ __forceinline__ float half_warp_max(float x) {
#pragma unroll
    for (int m = 8; m > 0; m >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, m));
    return x;
}
__device__ __forceinline__ float half_warp_sum(float x) {
#pragma unroll
    for (int m = 8; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// The streamed tiles of part blockIdx.z of gridDim.z: [part_begin, part_end) of n.
// (One part, which short calls have, spares the divisions: 8.3 -> 7.7 us.)
__device__ __forceinline__ int part_begin(int n) {
    return gridDim.z == 1 ? 0 : (int)((int64_t)n * blockIdx.z / gridDim.z);
}
__device__ __forceinline__ int part_end(int n) {
    return gridDim.z == 1 ? n : (int)((int64_t)n * (blockIdx.z + 1) / gridDim.z);
}
// This part's rows of this head: [part][head][row][D].
template <int D> __device__ __forceinline__ float *part_rows(float *parts, int rows) {
    return parts + ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * rows * D;
}

// ---------------------------------------------------------------- forward
// 16 RT queries of one head against tiles of 64 keys.  With one stage K and V take turns
// in one buffer.
template <int D, int RT>
constexpr int fwd_smem() {
    return ((16 * RT + 64 * (kStages<D> == 2 ? 4 : 1)) * kPitch<D> + 16 * RT * 68) * 4;
}

template <int D, int RT>
__global__ void __launch_bounds__(256, 2)
simt_fwd_kernel(WinProblem p, const float *q, const float *k, const float *v, float *out,
                float *lse, float *parts) {
    extern __shared__ __align__(16) float smf[];
    constexpr int kTileFloats = 64 * kPitch<D>;
    float *sq = smf, *sp = sq + 16 * RT * kPitch<D>, *skv = sp + 16 * RT * 68;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int h = blockIdx.y % p.H, b = blockIdx.y / p.H;
    const int i0 = blockIdx.x * 16 * RT;
    __shared__ Sequence shared_seq;
    Sequence seq = first_threads_sequence(p, b);
    load_rows<D, 16 * RT>(sq, q + b * p.q.batch + h * p.q.head, p.q.token, i0, p.Nq);
    share_sequence(seq, &shared_seq);
    const KeyTiles kt = key_tiles<64>(p, seq, i0, i0 + 16 * RT);
    const float *kb = k + b * p.k.batch + (h / p.G) * p.k.head;
    const float *vb = v + b * p.v.batch + (h / p.G) * p.v.head;
    const int first = part_begin(kt.count()), n = part_end(kt.count()) - first;
    auto load = [&](float *dst, const float *src, int64_t stride, int it) {
        load_rows<D, 64>(dst, src, stride, kt.tile(first + it) * 64, seq.len);
    };
    if (kStages<D> == 2 && n > 0) {
        load(skv, kb, p.k.token, 0);
        load(skv + kTileFloats, vb, p.v.token, 0);
    }
    copies_commit();
    RowKeys rk[RT];
    float m[RT], l[RT];
    uint64_t o[RT][D / 32];
#pragma unroll
    for (int i = 0; i < RT; i++) {
        rk[i] = row_keys(p, seq, i0 + RT * ty + i);
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int x = 0; x < D / 32; x++) o[i][x] = 0;
    }
    for (int it = 0; it < n; it++) {
        const int j0 = kt.tile(first + it) * 64;
        const float *sk = skv, *sv = skv;
        __syncthreads();   // the buffer's last readers are done
        if (kStages<D> == 2) {
            float *next = skv + ((it + 1) & 1) * 2 * kTileFloats;
            if (it + 1 < n) {
                load(next, kb, p.k.token, it + 1);
                load(next + kTileFloats, vb, p.v.token, it + 1);
            }
            copies_commit();
            copies_wait<1>();
            sk = skv + (it & 1) * 2 * kTileFloats;
            sv = sk + kTileFloats;
        } else {
            load(skv, kb, p.k.token, it);
            copies_commit();
            copies_wait<0>();
        }
        __syncthreads();
        float s[RT][4];
        dot_tile<D, RT, 4>(sq, sk, ty, tx, s);
#pragma unroll
        for (int i = 0; i < RT; i++) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                // a key outside the row's window never enters, whatever its value
                s[i][j] = rk[i].sees(j0 + tx + 16 * j) ? s[i][j] * p.scale_log2 : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
            mx = fmaxf(m[i], half_warp_max(mx));
            const float safe = mx == -INFINITY ? 0.f : mx;   // a row without keys so far
            const float alpha = exp2f(m[i] - safe);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float e = exp2f(s[i][j] - safe);
                sum += e;
                sp[(RT * ty + i) * 68 + tx + 16 * j] = e;
            }
            l[i] = l[i] * alpha + sum;   // this thread's columns; joined at the end
            m[i] = mx;
            const uint64_t aa = f2_pack(alpha, alpha);
#pragma unroll
            for (int x = 0; x < D / 32; x++) o[i][x] = f2_mul(o[i][x], aa);
        }
        if (kStages<D> == 2) {
            __syncwarp();      // the row's probabilities come from its own half warp
        } else {
            __syncthreads();   // K is read
            load(skv, vb, p.v.token, it);
            copies_commit();
            copies_wait<0>();
            __syncthreads();
        }
        add_product<D, RT, 64, 68>(sp, sv, ty, tx, o);
    }
    copies_wait<0>();   // without keys the queries' copies may still be under way
    float inv[RT];
#pragma unroll
    for (int i = 0; i < RT; i++) {
        const float total = half_warp_sum(l[i]);
        if (gridDim.z > 1) {   // the unscaled sums, and behind all of them (maximum, sum)
            const int64_t row = ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * p.Nq + i0 + RT * ty + i;
            inv[i] = 1.f;
            if (tx == 0 && i0 + RT * ty + i < p.Nq)
                *reinterpret_cast<float2 *>(parts + (int64_t)gridDim.z * gridDim.y * p.Nq * D + 2 * row) =
                    make_float2(m[i], total);
            continue;
        }
        inv[i] = total > 0.f ? 1.f / total : 0.f;
        if (total != total) inv[i] = total;   // NaN inputs stay visible
        const int r = i0 + RT * ty + i;
        if (lse && tx == 0 && r < p.Nq)
            lse[((int64_t)b * p.H + h) * p.Nq + r] =
                total == 0.f ? -INFINITY : (m[i] + log2f(total)) * kLn2;
    }
    if (gridDim.z > 1)
        store_rows<D, RT>(part_rows<D>(parts, p.Nq), D, i0, p.Nq, ty, tx, o, inv);
    else
        store_rows<D, RT>(out + b * p.o.batch + h * p.o.head, p.o.token, i0, p.Nq, ty, tx, o, inv);
}

// Rows from the parts of their keys, in order; a thread has 4 columns.
template <int D>
__global__ void __launch_bounds__(256)
simt_fwd_join_kernel(WinProblem p, int splits, const float *parts, float *out, float *lse) {
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, rows = (int64_t)p.B * p.H * p.Nq;
    const int64_t row = at / (D / 4);
    const int c = (int)(at % (D / 4)) * 4;
    if (row >= rows) return;
    const float2 *ml = reinterpret_cast<const float2 *>(parts + splits * rows * D);
    float mx = -INFINITY, sum = 0.f;
    for (int s = 0; s < splits; s++) mx = fmaxf(mx, ml[s * rows + row].x);
    const float safe = mx == -INFINITY ? 0.f : mx;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < splits; s++) {
        const float2 y = ml[s * rows + row];
        const float4 x = *reinterpret_cast<const float4 *>(parts + (s * rows + row) * D + c);
        const float f = exp2f(y.x - safe);
        sum = fmaf(f, y.y, sum);
        acc.x = fmaf(f, x.x, acc.x);
        acc.y = fmaf(f, x.y, acc.y);
        acc.z = fmaf(f, x.z, acc.z);
        acc.w = fmaf(f, x.w, acc.w);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;   // (a NaN stays visible)
    const int i = (int)(row % p.Nq), h = (int)(row / p.Nq % p.H), b = (int)(row / p.Nq / p.H);
    *reinterpret_cast<float4 *>(out + b * p.o.batch + h * p.o.head + i * p.o.token + c) =
        make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (lse && c == 0) lse[row] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

// ---------------------------------------------------------------- backward
// dq: 16 RT queries against tiles of 32 keys.  dS = P (dO.V - delta) with
// P = exp(S - lse); dq = scale * dS K.
template <int D, int RT>
constexpr int dq_smem() {
    return ((2 * 16 * RT + 2 * 32 * kStages<D>) * kPitch<D> + 16 * RT * 36) * 4;
}

template <int D, int RT>
__global__ void __launch_bounds__(256, 2)
simt_dq_kernel(WinProblem p, WinGrads g, const float *q, const float *k, const float *v,
               const float *lse, const float *delta, const float *dout, float *dq, float *parts) {
    extern __shared__ __align__(16) float smf[];
    constexpr int kTileFloats = 32 * kPitch<D>;
    float *sq = smf, *sdo = sq + 16 * RT * kPitch<D>, *sds = sdo + 16 * RT * kPitch<D>;
    float *skv = sds + 16 * RT * 36;   // [stage][K, V]
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int h = blockIdx.y % p.H, b = blockIdx.y / p.H;
    const int i0 = blockIdx.x * (16 * RT);
    __shared__ Sequence shared_seq;
    Sequence seq = first_threads_sequence(p, b);
    load_rows<D, 16 * RT>(sq, q + b * p.q.batch + h * p.q.head, p.q.token, i0, p.Nq);
    load_rows<D, 16 * RT>(sdo, dout + b * g.dout.batch + h * g.dout.head, g.dout.token, i0, p.Nq);
    share_sequence(seq, &shared_seq);
    const KeyTiles kt = key_tiles<32>(p, seq, i0, i0 + (16 * RT));
    const float *kb = k + b * p.k.batch + (h / p.G) * p.k.head;
    const float *vb = v + b * p.v.batch + (h / p.G) * p.v.head;
    const int first = part_begin(kt.count()), n = part_end(kt.count()) - first;
    auto load = [&](int it) {
        float *dst = skv + it % kStages<D> * 2 * kTileFloats;
        load_rows<D, 32>(dst, kb, p.k.token, kt.tile(first + it) * 32, seq.len);
        load_rows<D, 32>(dst + kTileFloats, vb, p.v.token, kt.tile(first + it) * 32, seq.len);
    };
    if (kStages<D> == 2 && n > 0) load(0);
    copies_commit();
    RowKeys rk[RT];
    float lm[RT], dl[RT];
    uint64_t o[RT][D / 32];
#pragma unroll
    for (int i = 0; i < RT; i++) {
        const int r = i0 + RT * ty + i;
        rk[i] = row_keys(p, seq, r);
        const int64_t at = ((int64_t)b * p.H + h) * p.Nq + r;
        lm[i] = r < p.Nq ? lse[at] * (1.f / kLn2) : 0.f;
        dl[i] = r < p.Nq ? delta[at] : 0.f;
#pragma unroll
        for (int x = 0; x < D / 32; x++) o[i][x] = 0;
    }
    for (int it = 0; it < n; it++) {
        const int j0 = kt.tile(first + it) * 32;
        const float *sk = skv + it % kStages<D> * 2 * kTileFloats, *sv = sk + kTileFloats;
        __syncthreads();
        if (it + kStages<D> - 1 < n) load(it + kStages<D> - 1);
        copies_commit();
        copies_wait<kStages<D> - 1>();
        __syncthreads();
        float s[RT][2], dp[RT][2];
        dot_tile<D, RT, 2>(sq, sk, ty, tx, s);
        dot_tile<D, RT, 2>(sdo, sv, ty, tx, dp);
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const float e = exp2f(fmaf(s[i][j], p.scale_log2, -lm[i]));
                sds[(RT * ty + i) * 36 + tx + 16 * j] =
                    rk[i].sees(j0 + tx + 16 * j) ? e * (dp[i][j] - dl[i]) : 0.f;
            }
        __syncwarp();
        add_product<D, RT, 32, 36>(sds, sk, ty, tx, o);
    }
    copies_wait<0>();   // (see the forward)
    float sc[RT];
#pragma unroll
    for (int i = 0; i < RT; i++) sc[i] = gridDim.z > 1 ? 1.f : p.scale;
    if (gridDim.z > 1)
        store_rows<D, RT>(part_rows<D>(parts, p.Nq), D, i0, p.Nq, ty, tx, o, sc);
    else
        store_rows<D, RT>(dq + b * g.dq.batch + h * g.dq.head, g.dq.token, i0, p.Nq, ty, tx, o, sc);
}

// dk, dv: 16 RT keys of one key head against tiles of 32 queries of every head of its
// group.  dv += P^T dO, dk += dS^T q (times scale at the end).
template <int D, int RT>
constexpr int dkv_smem() {
    return ((2 * 16 * RT + 2 * 32 * kStages<D>) * kPitch<D> + 16 * RT * 36) * 4;
}

template <int D, int RT>
__global__ void __launch_bounds__(256, 2)
simt_dkv_kernel(WinProblem p, WinGrads g, const float *q, const float *k, const float *v,
                const float *lse, const float *delta, const float *dout, float *dk, float *dv,
                float *parts) {
    extern __shared__ __align__(16) float smf[];
    constexpr int kTileFloats = 32 * kPitch<D>;
    float *sk = smf, *sv = sk + 16 * RT * kPitch<D>, *sw = sv + 16 * RT * kPitch<D>;
    float *sqd = sw + 16 * RT * 36;   // [stage][Q, dO]
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int hk = blockIdx.y % p.Hkv, b = blockIdx.y / p.Hkv;
    const int j0 = blockIdx.x * (16 * RT);
    __shared__ Sequence shared_seq;
    Sequence seq = first_threads_sequence(p, b);
    share_sequence(seq, &shared_seq);
    int first, last;
    query_rows(p, seq, j0, j0 + (16 * RT), first, last);
    load_rows<D, 16 * RT>(sk, k + b * p.k.batch + hk * p.k.head, p.k.token, j0, seq.len);
    load_rows<D, 16 * RT>(sv, v + b * p.v.batch + hk * p.v.head, p.v.token, j0, seq.len);
    uint64_t ok[RT][D / 32], ov[RT][D / 32];
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
        for (int x = 0; x < D / 32; x++) ok[i][x] = ov[i][x] = 0;
    int rfirst, rlast;
    real_rows(p, seq, 0, p.Nq, rfirst, rlast);
    // tiles of 32 queries of every head of the group
    const int t0 = first / 32, nt = last > first ? (last + 31) / 32 - t0 : 0;
    const int u0 = part_begin(nt * p.G), u1 = part_end(nt * p.G);
    auto load = [&](int u) {
        float *dst = sqd + u % kStages<D> * 2 * kTileFloats;
        const int h = hk * p.G + u / nt, i0 = (t0 + u % nt) * 32;
        // rows that are not real enter as zeros, whatever they hold
        load_rows<D, 32>(dst, q + b * p.q.batch + h * p.q.head, p.q.token, i0, rlast, rfirst);
        load_rows<D, 32>(dst + kTileFloats, dout + b * g.dout.batch + h * g.dout.head, g.dout.token,
                         i0, rlast, rfirst);
    };
    if (kStages<D> == 2 && u0 < u1) load(u0);
    copies_commit();
    for (int u = u0; u < u1; u++) {
        const int64_t row = ((int64_t)b * p.H + hk * p.G + u / nt) * p.Nq;
        const int i0 = (t0 + u % nt) * 32;
        const float *sq = sqd + u % kStages<D> * 2 * kTileFloats, *sdo = sq + kTileFloats;
        __syncthreads();
        if (u + kStages<D> - 1 < u1) load(u + kStages<D> - 1);
        copies_commit();
        copies_wait<kStages<D> - 1>();
        __syncthreads();
        {
            float s[RT][2], dp[RT][2];
            dot_tile<D, RT, 2>(sk, sq, ty, tx, s);
            dot_tile<D, RT, 2>(sv, sdo, ty, tx, dp);
#pragma unroll
            for (int c = 0; c < 2; c++) {
                const int i = i0 + tx + 16 * c;
                const RowKeys rk = row_keys(p, seq, i);
                const bool real = rk.hi > 0;
                const float lm = real ? lse[row + i] * (1.f / kLn2) : 0.f;
                const float dl = real ? delta[row + i] : 0.f;
#pragma unroll
                for (int r = 0; r < RT; r++) {
                    const bool see = rk.sees(j0 + RT * ty + r);
                    const float e = see ? exp2f(fmaf(s[r][c], p.scale_log2, -lm)) : 0.f;
                    s[r][c] = e;
                    dp[r][c] = see ? e * (dp[r][c] - dl) : 0.f;
                    sw[(RT * ty + r) * 36 + tx + 16 * c] = e;
                }
            }
            __syncwarp();
            add_product<D, RT, 32, 36>(sw, sdo, ty, tx, ov);
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 2; c++)
#pragma unroll
                for (int r = 0; r < RT; r++) sw[(RT * ty + r) * 36 + tx + 16 * c] = dp[r][c];
            __syncwarp();
            add_product<D, RT, 32, 36>(sw, sq, ty, tx, ok);
        }
    }
    copies_wait<0>();   // (see the forward)
    float sc[RT], one[RT];
#pragma unroll
    for (int i = 0; i < RT; i++) sc[i] = gridDim.z > 1 ? 1.f : p.scale, one[i] = 1.f;
    if (gridDim.z > 1) {   // all parts of dk, then those of dv
        float *rows = part_rows<D>(parts, p.Nk);
        store_rows<D, RT>(rows, D, j0, p.Nk, ty, tx, ok, sc);
        store_rows<D, RT>(rows + (int64_t)gridDim.z * gridDim.y * p.Nk * D, D, j0, p.Nk, ty, tx, ov, one);
        return;
    }
    store_rows<D, RT>(dk + b * g.dk.batch + hk * g.dk.head, g.dk.token, j0, p.Nk, ty, tx, ok, sc);
    store_rows<D, RT>(dv + b * g.dv.batch + hk * g.dv.head, g.dv.token, j0, p.Nk, ty, tx, ov, one);
}

// A gradient's rows [B][heads][tokens] from their parts, added in order; a thread has 4
// columns.
template <int D>
__global__ void __launch_bounds__(256)
simt_sum_kernel(const float *parts, int splits, int B, int heads, int tokens, float scale,
                Strides to, float *grad) {
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, rows = (int64_t)B * heads * tokens;
    const int64_t row = at / (D / 4);
    const int c = (int)(at % (D / 4)) * 4;
    if (row >= rows) return;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < splits; s++) {
        const float4 x = *reinterpret_cast<const float4 *>(parts + (s * rows + row) * D + c);
        acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
    }
    const int i = (int)(row % tokens), h = (int)(row / tokens % heads), b = (int)(row / tokens / heads);
    *reinterpret_cast<float4 *>(grad + b * to.batch + h * to.head + i * to.token + c) =
        make_float4(acc.x * scale, acc.y * scale, acc.z * scale, acc.w * scale);
}

// ---------------------------------------------------------------- delta
// delta_i = dO_i . O_i: 16-byte loads, d / 4 lanes a row; rows without keys get 0 (their dO
// may be anything).  Bound by memory: dO and O are read once.
template <int D>
__global__ void __launch_bounds__(256)
row_delta_kernel(WinProblem p, WinGrads g, const float *out, const float *dout, float *delta) {
    constexpr int LANES = D / 4, ROWS = 256 / LANES;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES;
    const int c = threadIdx.x % LANES * 4;
    float sum = 0.f;
    if (row < (int64_t)p.B * p.H * p.Nq) {
        const int i = (int)(row % p.Nq), bh = (int)(row / p.Nq), h = bh % p.H, b = bh / p.H;
        const Sequence seq = sequence(p, b);
        const int64_t pos = seq.start + i;
        if (pos >= 0 && pos < seq.len) {   // a real row
            const float4 x = *reinterpret_cast<const float4 *>(
                out + b * p.o.batch + h * p.o.head + i * p.o.token + c);
            const float4 y = *reinterpret_cast<const float4 *>(
                dout + b * g.dout.batch + h * g.dout.head + i * g.dout.token + c);
            sum = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, x.w * y.w)));
        }
    }
#pragma unroll
    for (int m = LANES / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (c == 0 && row < (int64_t)p.B * p.H * p.Nq) delta[row] = sum;
}

template <typename K>
cudaError_t allow_smem(K kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// How a kernel divides its work.  Rows a thread: 4 (tiles of 64 rows), or 2 where those
// tiles, and parts of them, would leave SMs without a CTA.  A tile's time is its
// shared-memory reads, most of them of the streamed side and the same for any number of
// rows, next to the FMAs, which halve; with 1 row a thread two CTAs share an SM's shared
// memory and take longer (4 heads of 780 tokens, 255 keys a row, d = 64: forward 43 us at 4
// rows, 33 at 1).  Parts of a tile's walk over the other side: as many as make the CTAs that
// run at once (two an SM), of four streamed tiles at least, or of `shared` where they would
// share SMs and gain less than the join takes.  d = 64: 12 heads of 100 queries over 9000
// keys forward 520 -> 113 us, backward 1049 -> 407; 4 heads of 1000 tokens backward 234 ->
// 139.  Backward without / with short parts that share SMs: 780 tokens of 4 heads, 255 keys a
// row, d = 64 79 / 89 us; 1000 tokens of 3 heads, 201 keys, d = 128 127 / 138; 2 x 400 tokens,
// 4 heads, d = 64 109 / 111; but 780 tokens of 2 heads, 511 keys, d = 128 140 / 130 and 3 x 512
// tokens, 2 heads, d = 64 123 / 95.  148 and 296 are the device's SMs and two CTAs on each.
struct Division {
    int rows, parts;
};
Division divide(int64_t heads, int rows, int64_t streamed, int shared) {
    const int64_t tiles = heads * ((rows + 63) / 64), most = std::max<int64_t>(1, streamed / 4);
    Division d;
    d.rows = tiles >= 148 || tiles * most >= 296 ? 4 : 2;
    const int64_t ctas = heads * ((rows + 16 * d.rows - 1) / (16 * d.rows));
    d.parts = (int)std::max<int64_t>(1, std::min(296 / ctas, most));
    while (d.parts > 1 && ctas * d.parts > 148 && streamed / d.parts < shared) d.parts--;
    return d;
}
Division forward_division(const WinProblem &p) {
    return divide((int64_t)p.B * p.H, p.Nq, most_keys(p, 64) / 64, 4);
}
Division dq_division(const WinProblem &p) {
    return divide((int64_t)p.B * p.H, p.Nq, most_keys(p, 64) / 32, 7);
}
Division dkv_division(const WinProblem &p) {
    return divide((int64_t)p.B * p.Hkv, p.Nk, most_queries(p, 64) / 32 * p.G, 7);
}

template <int D>
unsigned join_grid(int64_t rows) { return (unsigned)((rows * (D / 4) + 255) / 256); }

template <int D, int RT>
cudaError_t forward_rt(const WinProblem &p, const float *q, const float *k, const float *v,
                       float *out, float *lse, float *parts, cudaStream_t stream) {
    constexpr int smem = fwd_smem<D, RT>();
    cudaError_t e = allow_smem(simt_fwd_kernel<D, RT>, smem);
    if (e != cudaSuccess) return e;
    const int splits = forward_division(p).parts;
    const dim3 grid((p.Nq + 16 * RT - 1) / (16 * RT), p.B * p.H, splits);
    simt_fwd_kernel<D, RT><<<grid, 256, smem, stream>>>(p, q, k, v, out, lse, parts);
    e = cudaGetLastError();
    if (e != cudaSuccess || splits == 1) return e;
    simt_fwd_join_kernel<D><<<join_grid<D>((int64_t)p.B * p.H * p.Nq), 256, 0, stream>>>(
        p, splits, parts, out, lse);
    return cudaGetLastError();
}
template <int D, int RT>
cudaError_t dq_rt(const WinProblem &p, const WinGrads &g, const float *q, const float *k,
                  const float *v, const float *lse, const float *delta, const float *dout,
                  float *dq, float *parts, cudaStream_t stream) {
    constexpr int smem = dq_smem<D, RT>();
    cudaError_t e = allow_smem(simt_dq_kernel<D, RT>, smem);
    if (e != cudaSuccess) return e;
    const int splits = dq_division(p).parts;
    const dim3 grid((p.Nq + 16 * RT - 1) / (16 * RT), p.B * p.H, splits);
    simt_dq_kernel<D, RT><<<grid, 256, smem, stream>>>(p, g, q, k, v, lse, delta, dout, dq, parts);
    e = cudaGetLastError();
    if (e != cudaSuccess || splits == 1) return e;
    simt_sum_kernel<D><<<join_grid<D>((int64_t)p.B * p.H * p.Nq), 256, 0, stream>>>(
        parts, splits, p.B, p.H, p.Nq, p.scale, g.dq, dq);
    return cudaGetLastError();
}
template <int D, int RT>
cudaError_t dkv_rt(const WinProblem &p, const WinGrads &g, const float *q, const float *k,
                   const float *v, const float *lse, const float *delta, const float *dout,
                   float *dk, float *dv, float *parts, cudaStream_t stream) {
    constexpr int smem = dkv_smem<D, RT>();
    cudaError_t e = allow_smem(simt_dkv_kernel<D, RT>, smem);
    if (e != cudaSuccess) return e;
    const int splits = dkv_division(p).parts;
    const dim3 grid((p.Nk + 16 * RT - 1) / (16 * RT), p.B * p.Hkv, splits);
    simt_dkv_kernel<D, RT><<<grid, 256, smem, stream>>>(p, g, q, k, v, lse, delta, dout, dk, dv, parts);
    e = cudaGetLastError();
    if (e != cudaSuccess || splits == 1) return e;
    const int64_t rows = (int64_t)p.B * p.Hkv * p.Nk;
    simt_sum_kernel<D><<<join_grid<D>(rows), 256, 0, stream>>>(parts, splits, p.B, p.Hkv, p.Nk,
                                                               p.scale, g.dk, dk);
    simt_sum_kernel<D><<<join_grid<D>(rows), 256, 0, stream>>>(parts + splits * rows * D, splits, p.B,
                                                               p.Hkv, p.Nk, 1.f, g.dv, dv);
    return cudaGetLastError();
}

template <int D>
cudaError_t forward_d(const WinProblem &p, const float *q, const float *k, const float *v,
                      float *out, float *lse, float *parts, cudaStream_t stream) {
    if (forward_division(p).rows == 4) return forward_rt<D, 4>(p, q, k, v, out, lse, parts, stream);
    return forward_rt<D, 2>(p, q, k, v, out, lse, parts, stream);
}

template <int D>
cudaError_t backward_d(const WinProblem &p, const WinGrads &g, const float *q, const float *k,
                       const float *v, const float *out, const float *lse, float *delta,
                       const float *dout, float *dq, float *dk, float *dv, float *parts,
                       cudaStream_t stream) {
    const int64_t rows = (int64_t)p.B * p.H * p.Nq, per = 256 / (D / 4);
    row_delta_kernel<D><<<(unsigned)((rows + per - 1) / per), 256, 0, stream>>>(p, g, out, dout, delta);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = dq_division(p).rows == 4
            ? dq_rt<D, 4>(p, g, q, k, v, lse, delta, dout, dq, parts, stream)
            : dq_rt<D, 2>(p, g, q, k, v, lse, delta, dout, dq, parts, stream);
    if (e != cudaSuccess) return e;
    if (dkv_division(p).rows == 4)
        return dkv_rt<D, 4>(p, g, q, k, v, lse, delta, dout, dk, dv, parts, stream);
    return dkv_rt<D, 2>(p, g, q, k, v, lse, delta, dout, dk, dv, parts, stream);
}

}  // namespace

size_t simt_forward_bytes(const WinProblem &p) {
    const int splits = forward_division(p).parts;
    return splits == 1 ? 0 : (size_t)splits * p.B * p.H * p.Nq * (p.d + 2) * sizeof(float);
}
size_t simt_backward_bytes(const WinProblem &p) {
    // dq's parts are joined before those of dk and dv are written
    const int sq = dq_division(p).parts, sk = dkv_division(p).parts;
    const size_t q = sq == 1 ? 0 : (size_t)sq * p.B * p.H * p.Nq;
    const size_t k = sk == 1 ? 0 : (size_t)sk * p.B * p.Hkv * p.Nk * 2;
    return std::max(q, k) * p.d * sizeof(float);
}

cudaError_t simt_forward(const WinProblem &p, const float *q, const float *k, const float *v,
                         float *out, float *lse, void *workspace, cudaStream_t stream) {
    float *parts = (float *)workspace;
    if (p.d == 32) return forward_d<32>(p, q, k, v, out, lse, parts, stream);
    if (p.d == 64) return forward_d<64>(p, q, k, v, out, lse, parts, stream);
    return forward_d<128>(p, q, k, v, out, lse, parts, stream);
}

cudaError_t simt_backward(const WinProblem &p, const WinGrads &g, const float *q, const float *k,
                          const float *v, const float *out, const float *lse, float *delta,
                          const float *dout, float *dq, float *dk, float *dv, void *workspace,
                          cudaStream_t stream) {
    float *parts = (float *)workspace;
    return p.d == 32 ? backward_d<32>(p, g, q, k, v, out, lse, delta, dout, dq, dk, dv, parts, stream)
           : p.d == 64
               ? backward_d<64>(p, g, q, k, v, out, lse, delta, dout, dq, dk, dv, parts, stream)
               : backward_d<128>(p, g, q, k, v, out, lse, delta, dout, dq, dk, dv, parts, stream);
}

}  // namespace win
}  // namespace monarch
