// window_token.cu -- window attention of few query rows a key head (single tokens,
// a handful of new tokens) against many keys, in an ordinary or a paged cache.
//
// The work is reading the visible keys and values once, so the keys of one
// (sequence, key head) are split over CTAs, each with its own running maximum, sum
// and weighted values, and joined:
//   M = max_s m_s,  O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s.
// Up to 8 parts form a thread-block cluster and join through distributed shared
// memory: one launch and no workspace.  More parts (few key heads, long caches) are
// several clusters, whose results a second kernel joins.  Every join adds the parts
// in their order, so results do not depend on which CTA came first.
// The rows of a key head (queries x heads of its group) form tiles of 16, the height
// of mma.m16n8k16: every key is read once for each such tile, so once for a group of up to
// 16 heads and one query, and up to four times at the 64 rows where other kernels take
// over (window_api.cu).  The split counts the
// visible keys only (the sinks, then the window), from each sequence's own length,
// so ragged batches and windows divide evenly.
//
// bfloat16: one warp loads 64-key tiles of keys and values into a ring of stages (TMA;
// behind a page table one copy a page, 128-byte swizzle), four warps take 16 keys of
// each tile through ldmatrix and mma.sync.  The ring keeps the bytes in flight that
// the memory's latency needs whatever the warps wait for; loading fragments straight
// from global memory to registers reached 4.1 TB/s instead.  (The products need a tenth of
// the legacy tensor rate here; tcgen05 would spend a 128-row tile on 16 rows.)
// float32: FMA pipes, tiles of 32 keys through shared memory.
#include "window_mma.cuh"
#include "window_tc.cuh"

#include <cooperative_groups.h>

namespace monarch {
namespace win {
namespace {

namespace cg = cooperative_groups;

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kTokWarps = 4;                       // of the arithmetic
constexpr int kTokThreads = kTokWarps * 32;        // float32; one loading warp more for bfloat16
constexpr int kMaxCluster = 8;

struct TokenArgs {
    WinProblem p;
    int row_tiles, splits;   // splits: parts of the keys, `clusters` times the cluster size
    int clusters;
    float *part;   // [B * Hkv * row_tiles][clusters][16][d + 2]: O, m, l (clusters > 1)
    int *status;
    long long limit;
};

// Where the rows of one key head lie: a contiguous cache, or behind the page table.
// A page index outside the pool is reported and its keys count as absent.
struct KeyPlace {
    const int32_t *table;
    int64_t page_stride, token;
    int shift, mask, pages;
    int *status;
    // offset of row j (elements), or -1
    __device__ __forceinline__ int64_t at(int j) const {
        if (!table) return (int64_t)j * token;
        const int pg = table[j >> shift];
        if (pg < 0 || pg >= pages) {
            record_status(status, MONARCH_ERR_INVALID_ARG);
            return -1;
        }
        return pg * page_stride + (int64_t)(j & mask) * token;
    }
};

__device__ __forceinline__ KeyPlace key_place(const WinProblem &p, int b, int64_t token,
                                              int64_t page_stride, int *status) {
    KeyPlace kp;
    kp.table = p.table ? p.table + b * p.table_stride : nullptr;
    kp.page_stride = page_stride;
    kp.token = token;
    kp.shift = p.page_shift;
    kp.mask = (1 << p.page_shift) - 1;
    kp.pages = p.num_pages;
    kp.status = status;
    return kp;
}

// The rows of one CTA: tile rt of 16 of the Nq * G rows (query i, head of the group g),
// row rr = i * G + g.
struct TokenUnit {
    int b, hk, rt, split;
    Sequence seq;
    KeyTiles kt;
    int g0, g1;   // groups of T keys of this split
    RowKeys any;  // the keys that some row of the tile sees lie in these intervals
    // whether some key of [j, j + n) is among them
    __device__ __forceinline__ bool meets(int j, int n) const {
        return j < any.hi && (j + n > any.lo || j < any.sink);
    }
};

template <int T>
__device__ __forceinline__ TokenUnit token_unit(const TokenArgs &a, const Sequence &seq) {
    const WinProblem &p = a.p;
    TokenUnit u;
    u.split = blockIdx.x;
    u.rt = blockIdx.y;
    u.b = blockIdx.z / p.Hkv;
    u.hk = blockIdx.z % p.Hkv;
    u.seq = seq;
    const int i0 = u.rt * 16 / p.G, i1 = min(p.Nq, (u.rt * 16 + 15) / p.G + 1);
    u.kt = key_tiles<T>(p, u.seq, i0, i1);
    const int64_t n = u.kt.count();
    int r0, r1;
    real_rows(p, u.seq, i0, i1, r0, r1);
    const RowKeys x = row_keys(p, u.seq, r0), y = row_keys(p, u.seq, r1 - 1);
    u.any = r0 < r1 ? RowKeys{x.lo, y.hi, y.sink} : RowKeys{0, 0, 0};
    u.g0 = (int)(n * u.split / a.splits);
    u.g1 = (int)(n * (u.split + 1) / a.splits);
    return u;
}

__device__ __forceinline__ void write_lse(const WinProblem &p, float *lse, int b, int h, int i,
                                          float m, float l) {
    if (lse)
        lse[((int64_t)b * p.H + h) * p.Nq + i] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ---------------------------------------------------------------- join in a cluster
// One CTA's part of a row tile in shared memory: row r at r * (d + 4), its maximum and
// sum (log2 units) behind the rows.
template <int D> struct Part {
    static constexpr int kPitch = D + 4;
    static constexpr int kFloats = 16 * kPitch + 32;
};

__device__ __forceinline__ void store4(float *p, float a, float b, float c, float d) {
    *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float a, float b, float c, float d) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(a, b), pack_bf16(c, d));
}

// Joins the parts of the cluster's CTAs (a CTA alone: its own) and writes the rows, or
// with several clusters their part to the workspace.  The CTAs share the elements out.
template <int D, typename T>
__device__ __forceinline__ void join_cluster(const TokenArgs &a, const TokenUnit &u, float *part,
                                             T *out, float *lse) {
    constexpr int kPitch = Part<D>::kPitch;
    const WinProblem &p = a.p;
    const int rows = min(16, p.Nq * p.G - u.rt * 16);
    const int parts = a.splits / a.clusters;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = parts > 1 ? (int)cluster.block_rank() : 0;
    if (parts > 1)
        cluster.sync();
    else
        __syncthreads();
    for (int at = rank * blockDim.x + threadIdx.x; at < rows * (D / 4); at += parts * blockDim.x) {
        const int r = at / (D / 4), c = at % (D / 4) * 4;
        if (c >= p.d) continue;
        const float *src[kMaxCluster];
        float m[kMaxCluster], mx = -INFINITY;
#pragma unroll
        for (int s = 0; s < kMaxCluster; s++) {
            if (s >= parts) break;
            src[s] = parts > 1 ? cluster.map_shared_rank(part, s) : part;
            m[s] = src[s][16 * kPitch + r];
            mx = fmaxf(mx, m[s]);
        }
        const float safe = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int s = 0; s < kMaxCluster; s++) {
            if (s >= parts) break;
            const float f = exp2f(m[s] - safe);
            const float4 x = *reinterpret_cast<const float4 *>(src[s] + r * kPitch + c);
            sum = fmaf(f, src[s][16 * kPitch + 16 + r], sum);
            acc.x = fmaf(f, x.x, acc.x);
            acc.y = fmaf(f, x.y, acc.y);
            acc.z = fmaf(f, x.z, acc.z);
            acc.w = fmaf(f, x.w, acc.w);
        }
        if (a.clusters > 1) {
            const int64_t unit = ((int64_t)blockIdx.z * a.row_tiles + u.rt) * a.clusters;
            float *dst = a.part + ((unit + u.split / parts) * 16 + r) * (p.d + 2);
            *reinterpret_cast<float2 *>(dst + c) = make_float2(acc.x, acc.y);
            *reinterpret_cast<float2 *>(dst + c + 2) = make_float2(acc.z, acc.w);
            if (c == 0) *reinterpret_cast<float2 *>(dst + p.d) = make_float2(mx, sum);
        } else {
            const int rr = u.rt * 16 + r, i = rr / p.G, h = u.hk * p.G + rr % p.G;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            store4(out + u.b * p.o.batch + h * p.o.head + i * p.o.token + c, acc.x * inv,
                   acc.y * inv, acc.z * inv, acc.w * inv);
            if (c == 0) write_lse(p, lse, u.b, h, i, mx, sum);
        }
    }
    if (parts > 1) cluster.sync();   // the others have read this CTA's part
}

// The CTA's part from those of its four warps, which lie behind it.
template <int D> __device__ __forceinline__ void join_warps(float *part, int rows) {
    constexpr int kPitch = Part<D>::kPitch, kFloats = Part<D>::kFloats;
    for (int at = threadIdx.x; at < rows * (D / 4); at += blockDim.x) {
        const int r = at / (D / 4), c = at % (D / 4) * 4;
        const float *src = part + kFloats;
        float mx = -INFINITY;
#pragma unroll
        for (int x = 0; x < kTokWarps; x++) mx = fmaxf(mx, src[x * kFloats + 16 * kPitch + r]);
        const float safe = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < kTokWarps; x++) {
            const float *s = src + x * kFloats;
            const float f = exp2f(s[16 * kPitch + r] - safe);
            const float4 y = *reinterpret_cast<const float4 *>(s + r * kPitch + c);
            sum = fmaf(f, s[16 * kPitch + 16 + r], sum);
            acc.x = fmaf(f, y.x, acc.x);
            acc.y = fmaf(f, y.y, acc.y);
            acc.z = fmaf(f, y.z, acc.z);
            acc.w = fmaf(f, y.w, acc.w);
        }
        *reinterpret_cast<float4 *>(part + r * kPitch + c) = acc;
        if (c == 0) part[16 * kPitch + r] = mx, part[16 * kPitch + 16 + r] = sum;
    }
}

// ---------------------------------------------------------------- bfloat16
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Ring of kStages tiles of 64 keys and values: 96 KB at d = 128, so two CTAs fit on an
// SM and keep up to 192 KB in flight.
template <int D> struct Ring {
    static constexpr int kStages = D == 128 ? 3 : 4;
    static constexpr uint32_t kPanelBytes = 64 * 128;               // 64 rows of 64 columns
    static constexpr uint32_t kHalf = (D / 64) * kPanelBytes;       // keys, then values
    static constexpr uint32_t kStage = 2 * kHalf;
    static constexpr uint32_t kBars = kStages * kStage;             // full, empty, good, abort
    static constexpr uint32_t kSmem = kBars + 128 + 1024;           // + slack to align the base
    // after the last tile the ring holds the four warps' parts and the CTA's
    static_assert(5 * Part<D>::kFloats * 4 <= kBars, "parts fit the ring");
};

template <int D>
__global__ void __launch_bounds__(kTokThreads + 32)
token_bf16_kernel(const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, TokenArgs a, int box,
                  const __nv_bfloat16 *q, __nv_bfloat16 *out, float *lse) {
    using R = Ring<D>;
    constexpr int NS = R::kStages, PN = D / 64;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = align1024(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + R::kBars);
    uint64_t *empty = full + NS;
    // [stage]: bit g: the page of the tile's keys 8 g .. 8 g + 7 exists
    volatile uint32_t *good = reinterpret_cast<volatile uint32_t *>(empty + NS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(empty + NS) + NS;
    const WinProblem &p = a.p;
    __shared__ TokenUnit shared_unit;
    TokenUnit u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = lane >> 2, t = lane & 3;
    const int rows = p.Nq * p.G;
    const WaitCtx w{a.limit, a.status, abort_flag};

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[D / 8][4];
#pragma unroll
    for (int x = 0; x < D / 8; x++)
#pragma unroll
        for (int c = 0; c < 4; c++) o[x][c] = 0.f;

    if (warp == kTokWarps) {
        // ---------------- loads; the first ones go out before the block meets.  The other
        // warps take the unit from this one, which reads the sequence once, and the barriers
        // are initialised by warp 0 meanwhile.
        Sequence seq{0, 0};
        if (lane == 0) seq = sequence(p, blockIdx.z / p.Hkv);
        seq.len = __shfl_sync(0xffffffffu, seq.len, 0);
        seq.start = __shfl_sync(0xffffffffu, seq.start, 0);
        u = token_unit<64>(a, seq);
        if (lane == 0) shared_unit = u;
        asm volatile("bar.sync 1, 64;" ::: "memory");
        int issued = 0;
        auto load = [&](int g) {
            const int st = issued % NS, j0 = u.kt.tile(g) * 64;
            uint8_t *dst = sm + st * R::kStage;
            if (p.table) {
                // one box of min(page, 64) keys a lane; pages that hold no visible key, or
                // are not in the pool, read zeros (a coordinate past the last page)
                const int jb = j0 + lane * box;
                const bool mine = lane * box < 64;
                int pg = p.num_pages;
                bool bad = false;
                if (mine && u.meets(jb, box)) {
                    pg = p.table[u.b * p.table_stride + (jb >> p.page_shift)];
                    bad = pg < 0 || pg >= p.num_pages;
                    if (bad) {
                        record_status(a.status, MONARCH_ERR_INVALID_ARG);
                        pg = p.num_pages;
                    }
                }
                uint32_t bits = __ballot_sync(0xffffffffu, bad), absent = 0;
                for (int x = 0; bits && x < 8; x++) absent |= ((bits >> (8 * x / box)) & 1) << x;
                if (lane == 0) {
                    good[st] = ~absent;
                    mbar_expect_tx(full + st, R::kStage);
                }
                __syncwarp();
                if (mine) {
                    const int row = jb & ((1 << p.page_shift) - 1);
                    uint8_t *at = dst + lane * box * 128;
                    for (int pn = 0; pn < PN; pn++) {
                        tma_load_4d(at + pn * R::kPanelBytes, &tmK, pn * 64, row, u.hk, pg, full + st);
                        tma_load_4d(at + R::kHalf + pn * R::kPanelBytes, &tmV, pn * 64, row, u.hk, pg,
                                    full + st);
                    }
                }
            } else if (lane == 0) {
                good[st] = ~0u;
                mbar_expect_tx(full + st, R::kStage);
                for (int pn = 0; pn < PN; pn++) {
                    tma_load_4d(dst + pn * R::kPanelBytes, &tmK, pn * 64, j0, u.hk, u.b, full + st);
                    tma_load_4d(dst + R::kHalf + pn * R::kPanelBytes, &tmV, pn * 64, j0, u.hk, u.b,
                                full + st);
                }
            }
            issued++;
        };
        int g = u.g0;
        for (; g < u.g1 && issued < NS; g++) load(g);
        __syncthreads();
        for (; g < u.g1; g++) {
            if (!wait_warp(empty + issued % NS, (issued / NS - 1) & 1, w)) break;
            load(g);
        }
        // every issued copy lands before the ring is used for the parts
        if (lane == 0)
            for (int it = max(0, issued - NS); it < issued; it++)
                wait_phase_cleanup(full + it % NS, (it / NS) & 1, kCleanupPolls);
    } else {
        if (warp == 0) {
            if (lane == 0) {
                prefetch_map(&tmK);
                prefetch_map(&tmV);
                for (int s = 0; s < NS; s++) {
                    mbar_init(full + s, 1);
                    mbar_init(empty + s, kTokWarps);
                }
                *abort_flag = 0;
                fence_mbar_init();
            }
            __syncwarp();
            asm volatile("bar.arrive 1, 64;" ::: "memory");
        }
        // ---------------- rows n and n + 8 of the tile (real or not); keys 16 warp .. + 15 of
        // each tile
        uint32_t qf[D / 16][4];
#pragma unroll
        for (int y = 0; y < 2; y++) {
            const int rr = blockIdx.y * 16 + n + 8 * y, i = rr / p.G;
            const __nv_bfloat16 *src = q + blockIdx.z / p.Hkv * p.q.batch +
                                       (blockIdx.z % p.Hkv * p.G + rr % p.G) * p.q.head +
                                       i * p.q.token + 2 * t;
#pragma unroll
            for (int x = 0; x < D / 16; x++)
#pragma unroll
                for (int c = 0; c < 2; c++)
                    qf[x][y + 2 * c] = rr < rows && x * 16 + c * 8 < p.d
                                           ? *reinterpret_cast<const uint32_t *>(src + x * 16 + c * 8)
                                           : 0u;
        }
        __syncthreads();
        u = shared_unit;
        RowKeys rk[2];   // (none for a row that is not real: its logits do not count)
#pragma unroll
        for (int y = 0; y < 2; y++) {
            const int rr = u.rt * 16 + n + 8 * y;
            rk[y] = rr < rows ? row_keys(p, u.seq, rr / p.G) : RowKeys{0, 0, 0};
        }
        // this lane's row of an 8 x 8 matrix: key r8 (+ 8) of the 16, 16-byte column c
        const int r8 = lane & 7, mi = lane >> 3;
        const uint32_t base = smem_u32(sm) + warp * 16 * 128;
        for (int g = u.g0; g < u.g1; g++) {
            const int it = g - u.g0, st = it % NS, j0 = u.kt.tile(g) * 64 + warp * 16;
            if (!wait_warp(full + st, (it / NS) & 1, w)) break;
            if (u.meets(j0, 16)) {
                const uint32_t kt = base + st * R::kStage, vt = kt + R::kHalf;
                const uint32_t bits = good[st] >> (2 * warp);
                float s[2][4];
#pragma unroll
                for (int x = 0; x < 2; x++) {
#pragma unroll
                    for (int c = 0; c < 4; c++) s[x][c] = 0.f;
#pragma unroll
                    for (int kk = 0; kk < D / 32; kk++) {
                        const int c = kk * 4 + mi;
                        uint32_t b[4];
                        ldmatrix4(b, kt + (c >> 3) * R::kPanelBytes + (8 * x + r8) * 128 +
                                         (((c & 7) ^ r8) << 4));
                        mma16816(s[x], qf[2 * kk], b[0], b[1]);
                        mma16816(s[x], qf[2 * kk + 1], b[2], b[3]);
                    }
                }
                // s[x][2 y + c]: row n + 8 y, key j0 + 8 x + 2 t + c
                float alpha[2];
                bool moved = false;
#pragma unroll
                for (int y = 0; y < 2; y++) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int x = 0; x < 2; x++)
#pragma unroll
                        for (int c = 0; c < 2; c++) {
                            float &z = s[x][2 * y + c];
                            const bool see = rk[y].sees(j0 + 8 * x + 2 * t + c) && ((bits >> x) & 1);
                            z = see ? z * p.scale_log2 : -INFINITY;
                            mx = fmaxf(mx, z);
                        }
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    mx = fmaxf(mx, m[y]);
                    const float safe = mx == -INFINITY ? 0.f : mx;
                    alpha[y] = fast_exp2(m[y] - safe);
                    moved |= mx > m[y];
                    m[y] = mx;
                    float sum = 0.f;
#pragma unroll
                    for (int x = 0; x < 2; x++)
#pragma unroll
                        for (int c = 0; c < 2; c++) {
                            float &z = s[x][2 * y + c];
                            z = fast_exp2(z - safe);
                            sum += z;
                        }
                    l[y] = l[y] * alpha[y] + sum;
                }
                if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                    for (int x = 0; x < D / 8; x++)
#pragma unroll
                        for (int c = 0; c < 4; c++) o[x][c] *= alpha[c >> 1];
                }
                const uint32_t pf[4] = {pack_bf16(s[0][0], s[0][1]), pack_bf16(s[0][2], s[0][3]),
                                        pack_bf16(s[1][0], s[1][1]), pack_bf16(s[1][2], s[1][3])};
                // values that no row sees may be NaN, and 0 * NaN is NaN: they count as 0
                const bool whole = u.any.sees(j0) && u.any.sees(j0 + 15) &&
                                   (j0 >= u.any.lo || j0 + 15 < u.any.sink);
                uint32_t keep[2] = {~0u, ~0u};
                if (!whole)
#pragma unroll
                    for (int x = 0; x < 2; x++) {
                        const int j = j0 + 8 * x + 2 * t;
                        keep[x] = (u.any.sees(j) ? 0xFFFFu : 0u) |
                                  (u.any.sees(j + 1) ? 0xFFFF0000u : 0u);
                    }
#pragma unroll
                for (int dd = 0; dd < D / 16; dd++) {
                    const int c = dd * 2 + (mi >> 1);
                    uint32_t b[4];
                    ldmatrix4_trans(b, vt + (c >> 3) * R::kPanelBytes +
                                           ((mi & 1) * 8 + r8) * 128 + (((c & 7) ^ r8) << 4));
                    mma16816(o[2 * dd], pf, b[0] & keep[0], b[1] & keep[1]);
                    mma16816(o[2 * dd + 1], pf, b[2] & keep[0], b[3] & keep[1]);
                }
            }
            mbar_arrive_warp(empty + st);
        }
    }

    // the four warps' parts, then the CTA's, in the ring's memory
    __syncthreads();
    constexpr int kPitch = Part<D>::kPitch, kFloats = Part<D>::kFloats;
    float *part = reinterpret_cast<float *>(sm);
    if (warp < kTokWarps) {
        float *mine = part + (1 + warp) * kFloats;
#pragma unroll
        for (int y = 0; y < 2; y++) {
            l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
            l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
            const int r = n + 8 * y;
            if (t == 0) {
                mine[16 * kPitch + r] = m[y];
                mine[16 * kPitch + 16 + r] = l[y];
            }
#pragma unroll
            for (int x = 0; x < D / 8; x++)
                *reinterpret_cast<float2 *>(mine + r * kPitch + x * 8 + 2 * t) =
                    make_float2(o[x][2 * y], o[x][2 * y + 1]);
        }
    }
    __syncthreads();
    join_warps<D>(part, min(16, rows - u.rt * 16));
    join_cluster<D>(a, u, part, out, lse);
}

// ---------------------------------------------------------------- float32
// 16 bytes to shared memory, asynchronously; zeros where `there` is false.
__device__ __forceinline__ void copy16(float *dst, const float *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}

// Tiles of 32 keys, the next one's copies behind this one's arithmetic; 8 keys a warp.  In
// the logits four lanes share a key, a quarter of the columns each, which stay in registers
// for all rows (at most R); in the output a lane has columns lane, lane + 32, ..., and a
// value serves all rows.  Each warp has its own maxima and sums; they join at the end.
// Bound by memory up to four rows (8 key heads of 32768 keys, d = 128: 70.6 us, 3.8 TB/s),
// then by the FMA pipes.  One tile at a time, its rows divided among the warps and a lane a
// key, took 128; 24 sequences of 6000 keys, 4 heads a key head 186 us instead of 101.
template <int D, int R>
__global__ void __launch_bounds__(kTokThreads)
token_f32_kernel(TokenArgs a, const float *q, const float *k, const float *v, float *out,
                 float *lse) {
    constexpr int P = D + 4, C = D / 32, kTile = 32 * P + 32 * D;
    extern __shared__ __align__(16) float buf[];   // two tiles of keys and values, q, sp
    __shared__ RowKeys row_range[R];
    float *sq = buf + 2 * kTile;
    const WinProblem &p = a.p;
    __shared__ Sequence shared_seq;
    Sequence seq = first_threads_sequence(p, blockIdx.z / p.Hkv);
    share_sequence(seq, &shared_seq);
    const TokenUnit u = token_unit<32>(a, seq);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, key = lane & 7, quarter = lane >> 3;
    float *sp = sq + 16 * D + warp * R * 8;   // the warp's probabilities, [row][8]
    const int rows = min(R, p.Nq * p.G - u.rt * 16);
    const float *kb = k + u.hk * p.k.head + (p.table ? 0 : u.b * p.k.batch);
    const float *vb = v + u.hk * p.v.head + (p.table ? 0 : u.b * p.v.batch);
    const KeyPlace kp = key_place(p, u.b, p.k.token, p.k.batch, a.status);
    const KeyPlace vp = key_place(p, u.b, p.v.token, p.v.batch, a.status);
    for (int x = threadIdx.x; x < rows * D / 4; x += kTokThreads) {
        const int r = x / (D / 4), c = x % (D / 4) * 4, rr = u.rt * 16 + r;
        *reinterpret_cast<float4 *>(sq + r * D + c) = *reinterpret_cast<const float4 *>(
            q + u.b * p.q.batch + (u.hk * p.G + rr % p.G) * p.q.head + (rr / p.G) * p.q.token + c);
    }
    if (threadIdx.x < rows) row_range[threadIdx.x] = row_keys(p, u.seq, (u.rt * 16 + threadIdx.x) / p.G);
    float m[R], l[R], o[R][C];
#pragma unroll
    for (int r = 0; r < R; r++) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < C; c++) o[r][c] = 0.f;
    }
    // tile g to its buffer, asynchronously; keys that no row sees, or whose page does not
    // exist, become zeros
    auto load = [&](int g) {
        const int j0 = u.kt.tile(g) * 32;
        float *sk = buf + (g & 1) * kTile, *sv = sk + 32 * P;
        for (int x = threadIdx.x; x < 32 * D / 4; x += kTokThreads) {
            const int r = x / (D / 4), c = x % (D / 4) * 4, j = j0 + r;
            int64_t ka = -1, va = -1;
            if (u.any.sees(j)) ka = kp.at(j), va = vp.at(j);
            copy16(sk + r * P + c, kb + (ka >= 0 ? ka + c : 0), ka >= 0);
            copy16(sv + r * D + c, vb + (va >= 0 ? va + c : 0), va >= 0);
        }
    };
    if (u.g0 < u.g1) load(u.g0);
    copies_commit();
    for (int g = u.g0; g < u.g1; g++) {
        const int j0 = u.kt.tile(g) * 32;
        const float *sk = buf + (g & 1) * kTile, *sv = sk + 32 * P;
        __syncthreads();   // the other buffer's last readers are done
        if (g + 1 < u.g1) load(g + 1);
        copies_commit();
        copies_wait<1>();
        __syncthreads();
        const int j = j0 + warp * 8 + key;
        const bool there = u.any.sees(j) && kp.at(j) >= 0;
        float4 kr[D / 16];
        const float *kp4 = sk + (warp * 8 + key) * P + quarter * (D / 4);
#pragma unroll
        for (int c = 0; c < D / 16; c++) kr[c] = *reinterpret_cast<const float4 *>(kp4 + 4 * c);
#pragma unroll
        for (int r = 0; r < R; r++) {
            if (r >= rows) break;   // the same for the whole CTA
            const float *qr = sq + r * D + quarter * (D / 4);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int c = 0; c < D / 16; c++) {
                const float4 y = *reinterpret_cast<const float4 *>(qr + 4 * c);
                acc.x = fmaf(y.x, kr[c].x, acc.x);
                acc.y = fmaf(y.y, kr[c].y, acc.y);
                acc.z = fmaf(y.z, kr[c].z, acc.z);
                acc.w = fmaf(y.w, kr[c].w, acc.w);
            }
            float z = (acc.x + acc.y) + (acc.z + acc.w);
            z += __shfl_xor_sync(0xffffffffu, z, 8);
            z += __shfl_xor_sync(0xffffffffu, z, 16);
            z = there && row_range[r].sees(j) ? z * p.scale_log2 : -INFINITY;
            float mx = z;
#pragma unroll
            for (int s = 4; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
            mx = fmaxf(mx, m[r]);
            const float safe = mx == -INFINITY ? 0.f : mx;
            const float alpha = exp2f(m[r] - safe), e = exp2f(z - safe);
            m[r] = mx;
            l[r] = l[r] * alpha + e;   // of this lane's key
#pragma unroll
            for (int c = 0; c < C; c++) o[r][c] *= alpha;
            if (quarter == 0) sp[r * 8 + key] = e;
        }
        __syncwarp();
#pragma unroll
        for (int jj = 0; jj < 8; jj += 4) {
            float vr[4][C];
#pragma unroll
            for (int x = 0; x < 4; x++)
#pragma unroll
                for (int c = 0; c < C; c++) vr[x][c] = sv[(warp * 8 + jj + x) * D + c * 32 + lane];
#pragma unroll
            for (int r = 0; r < R; r++) {
                if (r >= rows) break;
                const float4 w = *reinterpret_cast<const float4 *>(sp + r * 8 + jj);
#pragma unroll
                for (int c = 0; c < C; c++)
                    o[r][c] = fmaf(w.w, vr[3][c], fmaf(w.z, vr[2][c], fmaf(w.y, vr[1][c],
                                                                        fmaf(w.x, vr[0][c], o[r][c]))));
            }
        }
    }
    // the warps' parts, then the CTA's, over the tiles (every warp is done with them, and no
    // copy is under way)
    copies_wait<0>();
    __syncthreads();
    constexpr int kPitch = Part<D>::kPitch;
    static_assert(5 * Part<D>::kFloats <= 2 * kTile, "the parts fit the tiles");
    float *part = buf, *mine = part + (1 + warp) * Part<D>::kFloats;
#pragma unroll
    for (int r = 0; r < R; r++) {
        if (r >= rows) break;
        float sum = l[r];
#pragma unroll
        for (int s = 4; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
#pragma unroll
        for (int c = 0; c < C; c++) mine[r * kPitch + c * 32 + lane] = o[r][c];
        if (lane == 0) mine[16 * kPitch + r] = m[r], mine[16 * kPitch + 16 + r] = sum;
    }
    __syncthreads();
    join_warps<D>(part, rows);
    join_cluster<D>(a, u, part, out, lse);
}

// ---------------------------------------------------------------- join of clusters
// One warp a row (query, head).
template <typename T>
__global__ void __launch_bounds__(256) token_join_kernel(TokenArgs a, T *out, float *lse) {
    const WinProblem &p = a.p;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, rows = p.Nq * p.G;
    if (row >= (int64_t)p.B * p.Hkv * rows) return;
    const int rr = (int)(row % rows);
    const int64_t bh = row / rows;
    const int b = (int)(bh / p.Hkv), hk = (int)(bh % p.Hkv);
    const int d2 = p.d + 2;
    const float *part =
        a.part + ((bh * a.row_tiles + rr / 16) * a.clusters * 16 + rr % 16) * (int64_t)d2;
    const int64_t step = 16 * (int64_t)d2;
    float mx = -INFINITY;
    for (int s = lane; s < a.clusters; s += 32) mx = fmaxf(mx, part[s * step + p.d]);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    const float safe = mx == -INFINITY ? 0.f : mx;
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
#pragma unroll 4
    for (int s = 0; s < a.clusters; s++) {
        const float *src = part + s * step;
        const float f = exp2f(src[p.d] - safe);
        sum = fmaf(f, src[p.d + 1], sum);
#pragma unroll
        for (int c = 0; c < 4; c++)
            if (c * 32 < p.d) acc[c] = fmaf(f, src[c * 32 + lane], acc[c]);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int i = rr / p.G, h = hk * p.G + rr % p.G;
    T *dst = out + b * p.o.batch + h * p.o.head + i * p.o.token;
#pragma unroll
    for (int c = 0; c < 4; c++)
        if (c * 32 < p.d) dst[c * 32 + lane] = from_f32<T>(acc[c] * inv);
    if (lane == 0) write_lse(p, lse, b, h, i, mx, sum);
}

template <typename T>
cudaError_t join(const TokenArgs &a, T *out, float *lse, cudaStream_t stream) {
    const int64_t rows = (int64_t)a.p.B * a.p.H * a.p.Nq;
    token_join_kernel<T><<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(a, out, lse);
    return cudaGetLastError();
}

}  // namespace

// Parts of the visible keys.  More parts fill the SMs and even out ragged lengths; each
// costs a prologue and a join, and parts beyond the clusters that fit on the device at once
// (kFit: 72 of four CTAs where 71 fit take two rounds) another round.  Up to 8 parts are one
// cluster, more are clusters of 8.
//
// Taken is the number with the least estimated time, in microseconds: rounds (two thirds of
// them counted by what they hold, as lengths may be ragged) of tiles at the rate of the
// latency of a CTA's copies or of the SM's share of the memory, 4 for a CTA's prologue and
// join, 2.5 and more for the join of clusters.  Against as many as make three CTAs an SM,
// bfloat16: one sequence of 4000 keys, 12 heads 22.7 -> 14.8 us; 4 x 2000 keys, 8 key heads
// 24.6 -> 13.8; 24 x 6000 keys, 4 key heads of 64 46.9 -> 32.3; four of 131072 keys 252 -> 242.
// kFit, latency and share are the bfloat16 kernels' on 148 SMs.  A float32 tile has half the keys
// and the same bytes, and the float32 kernels use the same numbers although more of their
// CTAs fit on an SM: for them the estimate is a rule of thumb.  Keys are counted by what the
// tensors hold, as the lengths are on the device.
int parts_of(int64_t units, double tiles, int d) {
    static constexpr int kFit[2][8] = {{444, 222, 142, 104, 82, 71, 56, 48},   // d = 32, 64
                                       {296, 148, 93, 71, 56, 45, 37, 33}};    // d = 128
    const int *fit = kFit[d == 128];
    const double latency = d == 128 ? 1.16 : 0.87, share = d == 128 ? 0.73 : 0.36;
    int best = 1;
    double least = 1e30;
    for (int parts = 1; parts <= 512 && (parts == 1 || tiles >= 2 * parts);
         parts = parts < 8 ? parts + 1 : 2 * parts) {
        const int size = parts < kMaxCluster ? parts : kMaxCluster, groups = parts / size;
        const int64_t clusters = units * groups, room = fit[size - 1];
        const double held = max(1.0, (double)clusters / room);
        const double rounds = ((double)((clusters + room - 1) / room) + 2 * held) / 3;
        const int64_t per_sm = (min(clusters, room) * size + 147) / 148;
        const double time = rounds * (tiles / parts * max(latency, per_sm * share) + 4) +
                            (groups > 1 ? 2.5 + 0.1 * groups : 0);
        if (time < least) least = time, best = parts;
    }
    return best;
}

TokenPlan token_plan(const WinProblem &p, monarch_dtype dtype) {
    TokenPlan t;
    t.row_tiles = (p.Nq * p.G + 15) / 16;
    const int64_t units = (int64_t)p.B * p.Hkv * t.row_tiles;
    const int64_t most = most_keys(p, p.Nq);
    // (a tile of 64 bfloat16 or 32 float32 keys)
    const int64_t parts = parts_of(units, most / (dtype == MONARCH_BF16 ? 64.0 : 32.0), p.d);
    t.clusters = (int)((parts + kMaxCluster - 1) / kMaxCluster);
    t.splits = (int)((parts + t.clusters - 1) / t.clusters) * t.clusters;
    t.bytes = t.clusters > 1 ? (size_t)units * t.clusters * 16 * (p.d + 2) * sizeof(float) : 0;
    return t;
}

namespace {

// A launch of grid.x / parts clusters of `parts` CTAs.
template <typename... Params, typename... Args>
cudaError_t launch_parts(void (*kernel)(Params...), const TokenArgs &a, const dim3 &grid, int threads,
                         uint32_t smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = a.splits / a.clusters;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D>
cudaError_t launch_f32(const TokenArgs &a, const dim3 &grid, const void *q, const void *k,
                       const void *v, void *out, float *lse, cudaStream_t stream) {
    const bool few = a.p.Nq * a.p.G <= 4;
    const auto kernel = few ? token_f32_kernel<D, 4> : token_f32_kernel<D, 16>;
    const uint32_t smem = (2 * (32 * (D + 4) + 32 * D) + 16 * D + kTokWarps * (few ? 4 : 16) * 8) * 4;
    const cudaError_t e = tcs::set_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    return launch_parts(kernel, a, grid, kTokThreads, smem, stream, a, (const float *)q,
                        (const float *)k, (const float *)v, (float *)out, lse);
}

template <int D>
cudaError_t launch_bf16(const TokenArgs &a, const dim3 &grid, const void *q, const void *k,
                        const void *v, void *out, float *lse, cudaStream_t stream) {
    const WinProblem &p = a.p;
    const int page = 1 << p.page_shift, box = p.table ? min(page, 64) : 64;
    const int tokens = p.table ? page : p.Nk, batches = p.table ? p.num_pages : p.B;
    CUtensorMap mk, mv;
    if (!map_tokens(&mk, k, p.k, batches, p.Hkv, tokens, p.d, (uint32_t)box) ||
        !map_tokens(&mv, v, p.v, batches, p.Hkv, tokens, p.d, (uint32_t)box))
        return cudaErrorInvalidValue;
    cudaError_t e = tcs::set_smem(token_bf16_kernel<D>, Ring<D>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_parts(token_bf16_kernel<D>, a, grid, kTokThreads + 32, Ring<D>::kSmem, stream, mk,
                        mv, a, box, (const __nv_bfloat16 *)q, (__nv_bfloat16 *)out, lse);
}

}  // namespace

cudaError_t token_forward(const WinProblem &p, monarch_dtype dtype, const TokenPlan &plan,
                          const void *q, const void *k, const void *v, void *out, float *lse,
                          void *workspace, int *status, long long limit, cudaStream_t stream) {
    const TokenArgs a{p, plan.row_tiles, plan.splits, plan.clusters, (float *)workspace, status, limit};
    const dim3 grid(plan.splits, plan.row_tiles, p.B * p.Hkv);
    cudaError_t e;
    if (dtype == MONARCH_F32)
        e = p.d == 32   ? launch_f32<32>(a, grid, q, k, v, out, lse, stream)
            : p.d == 64 ? launch_f32<64>(a, grid, q, k, v, out, lse, stream)
                        : launch_f32<128>(a, grid, q, k, v, out, lse, stream);
    else
        e = p.d == 128 ? launch_bf16<128>(a, grid, q, k, v, out, lse, stream)
                       : launch_bf16<64>(a, grid, q, k, v, out, lse, stream);
    if (e != cudaSuccess || plan.clusters == 1) return e;
    return dtype == MONARCH_F32 ? join(a, (float *)out, lse, stream)
                                : join(a, (__nv_bfloat16 *)out, lse, stream);
}

}  // namespace win
}  // namespace monarch
