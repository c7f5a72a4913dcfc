// window_token.cu -- window attention of few query rows a key head (single tokens,
// a handful of new tokens) against many keys, in an ordinary or a paged cache.
//
// The work is reading the visible keys and values once, so the keys of one
// (sequence, key head) are split over CTAs, each with its own running maximum, sum
// and weighted values, and a second kernel joins the parts:
//   M = max_s m_s,  O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s.
// The rows of a key head (queries x heads of its group) form tiles of 16, the height
// of mma.m16n8k16: every key is read once for all of them.  The split counts the
// visible keys only (the sinks, then the window), from each sequence's own length,
// so ragged batches and windows divide evenly.
//
// bfloat16: each warp takes groups of 16 keys; keys and values go from global
// memory straight to the fragments.  The head dimension of the first product and the
// columns of the second are permuted so that each lane's 16-byte loads are whole
// fragments: lane (n, t) = (lane / 4, lane % 4) reads elements 32 kb + 8 t .. + 7 of
// key n, four fragment registers of two K-steps, and elements 8 n .. + 7 (+ 64 h) of
// the value rows 2 t and 2 t + 1, which byte permutes pair up along the keys.
// float32: FMA pipes, tiles of 32 keys through shared memory, one lane a key.
#include "tc_primitives.cuh"
#include "window_common.cuh"

namespace monarch {
namespace win {
namespace {

using tc::fast_exp2;
using tc::pack_bf16;

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kTokWarps = 4;
constexpr int kTokThreads = kTokWarps * 32;

struct TokenArgs {
    WinProblem p;
    int row_tiles, splits;
    float *part;   // [B * Hkv * row_tiles][splits][16][d + 2]: O, m, l (splits > 1)
    int *status;
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
__device__ __forceinline__ TokenUnit token_unit(const TokenArgs &a) {
    const WinProblem &p = a.p;
    TokenUnit u;
    u.split = blockIdx.x;
    u.rt = blockIdx.y;
    u.b = blockIdx.z / p.Hkv;
    u.hk = blockIdx.z % p.Hkv;
    u.seq = sequence(p, u.b);
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

// Row rr's part (16 rows of d values, then m and l) or, with one split, its output.
__device__ __forceinline__ float *part_row(const TokenArgs &a, const TokenUnit &u, int r) {
    const int64_t unit = ((int64_t)blockIdx.z * a.row_tiles + u.rt) * a.splits + u.split;
    return a.part + (unit * 16 + r) * (a.p.d + 2);
}

template <typename T>
__device__ __forceinline__ void write_lse(const WinProblem &p, float *lse, int b, int h, int i,
                                          float m, float l) {
    if (lse)
        lse[((int64_t)b * p.H + h) * p.Nq + i] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ---------------------------------------------------------------- bfloat16
__device__ __forceinline__ uint4 load16(const __nv_bfloat16 *p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}
__device__ __forceinline__ uint2 load8(const __nv_bfloat16 *p) {
    uint2 r;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                 : "=r"(r.x), "=r"(r.y)
                 : "l"(p));
    return r;
}

// c += a b: a 16 x 16 (row), b 16 x 8 (column), bfloat16 with float32 sums.
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(kTokThreads)
token_bf16_kernel(TokenArgs a, const __nv_bfloat16 *q, const __nv_bfloat16 *k,
                  const __nv_bfloat16 *v, __nv_bfloat16 *out, float *lse) {
    constexpr int KB = D / 32;                // 32-element blocks of the head dimension
    constexpr int E = D >= 64 ? 8 : 4;        // value elements a lane reads at once
    constexpr int VH = D / (8 * E);           // such reads a row
    constexpr int VW = E / 2;                 // registers of one
    __shared__ float so[kTokWarps][16][D + 4];
    __shared__ float sml[kTokWarps][16][2];
    const WinProblem &p = a.p;
    const TokenUnit u = token_unit<16>(a);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = lane >> 2, t = lane & 3;
    const int rows = p.Nq * p.G;
    const __nv_bfloat16 *kb = k + u.hk * p.k.head + (p.table ? 0 : u.b * p.k.batch);
    const __nv_bfloat16 *vb = v + u.hk * p.v.head + (p.table ? 0 : u.b * p.v.batch);
    const KeyPlace kp = key_place(p, u.b, p.k.token, p.k.batch, a.status);
    const KeyPlace vp = key_place(p, u.b, p.v.token, p.v.batch, a.status);

    uint4 qf[2][KB];
    RowKeys rk[2];
#pragma unroll
    for (int x = 0; x < 2; x++) {
        const int rr = u.rt * 16 + n + 8 * x;
        rk[x] = RowKeys{0, 0, 0};
        const bool real = rr < rows;
        const int i = rr / p.G, h = u.hk * p.G + rr % p.G;
        if (real) rk[x] = row_keys(p, u.seq, i);
#pragma unroll
        for (int c = 0; c < KB; c++) {
            qf[x][c] = make_uint4(0, 0, 0, 0);
            if (real && rk[x].hi > 0)
                qf[x][c] = load16(q + u.b * p.q.batch + h * p.q.head + i * p.q.token + c * 32 + t * 8);
        }
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[VH][E][4];
#pragma unroll
    for (int x = 0; x < VH; x++)
#pragma unroll
        for (int e = 0; e < E; e++)
#pragma unroll
            for (int c = 0; c < 4; c++) o[x][e][c] = 0.f;

    uint4 kf[2][KB];
    uint32_t vf[2][2][VH][VW];   // [8-key tile][key 2t or 2t + 1]
    bool there[2];               // the tile's page exists (load_k)
    auto load_k = [&](int g) {
        const int j0 = u.kt.tile(g) * 16;
#pragma unroll
        for (int x = 0; x < 2; x++) {
            const int j = j0 + 8 * x + n;
            // (pages hold at least 8 keys: the table has an entry for all 8 or none)
            const int64_t at = u.meets(j0 + 8 * x, 8) ? kp.at(j) : -1;
            there[x] = at >= 0;
#pragma unroll
            for (int c = 0; c < KB; c++) {
                kf[x][c] = make_uint4(0, 0, 0, 0);
                if (at >= 0 && j < u.seq.len) kf[x][c] = load16(kb + at + c * 32 + t * 8);
            }
        }
    };
    auto load_v = [&](int g) {
        const int j0 = u.kt.tile(g) * 16;
#pragma unroll
        for (int x = 0; x < 2; x++) {
            const int j = j0 + 8 * x + 2 * t;
            const int64_t at = u.meets(j0 + 8 * x, 8) ? vp.at(j) : -1;
#pragma unroll
            for (int y = 0; y < 2; y++)   // a value that no row sees is not read: 0 * NaN is NaN
#pragma unroll
                for (int c = 0; c < VH; c++) {
                    uint32_t *r = vf[x][y][c];
                    const __nv_bfloat16 *src = vb + at + y * p.v.token + c * 64 + n * E;
                    const bool read = at >= 0 && u.any.sees(j + y);
                    if (E == 8) {
                        const uint4 w = read ? load16(src) : make_uint4(0, 0, 0, 0);
                        r[0] = w.x, r[1] = w.y, r[VW - 2] = w.z, r[VW - 1] = w.w;
                    } else {
                        const uint2 w = read ? load8(src) : make_uint2(0, 0);
                        r[0] = w.x, r[1] = w.y;
                    }
                }
        }
    };

    int g = u.g0 + warp;
    if (g < u.g1) {
        load_k(g);
        load_v(g);
    }
    for (; g < u.g1; g += kTokWarps) {
        const int j0 = u.kt.tile(g) * 16;
        const bool next = g + kTokWarps < u.g1;
        float s[2][4];
#pragma unroll
        for (int x = 0; x < 2; x++) {
#pragma unroll
            for (int c = 0; c < 4; c++) s[x][c] = 0.f;
#pragma unroll
            for (int c = 0; c < KB; c++) {
                mma16816(s[x], qf[0][c].x, qf[1][c].x, qf[0][c].y, qf[1][c].y, kf[x][c].x, kf[x][c].y);
                mma16816(s[x], qf[0][c].z, qf[1][c].z, qf[0][c].w, qf[1][c].w, kf[x][c].z, kf[x][c].w);
            }
        }
        const bool th0 = there[0], th1 = there[1];
        if (next) load_k(g + kTokWarps);
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
                    const bool see = rk[y].sees(j0 + 8 * x + 2 * t + c) && (x ? th1 : th0);
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
            for (int x = 0; x < VH; x++)
#pragma unroll
                for (int e = 0; e < E; e++)
#pragma unroll
                    for (int c = 0; c < 4; c++) o[x][e][c] *= alpha[c >> 1];
        }
        const uint32_t p0 = pack_bf16(s[0][0], s[0][1]), p1 = pack_bf16(s[0][2], s[0][3]);
        const uint32_t p2 = pack_bf16(s[1][0], s[1][1]), p3 = pack_bf16(s[1][2], s[1][3]);
#pragma unroll
        for (int x = 0; x < VH; x++)
#pragma unroll
            for (int w = 0; w < VW; w++) {
                // elements 2w and 2w + 1 of the two keys of each 8-key tile
                const uint32_t a0 = vf[0][0][x][w], a1 = vf[0][1][x][w];
                const uint32_t b0 = vf[1][0][x][w], b1 = vf[1][1][x][w];
                mma16816(o[x][2 * w], p0, p1, p2, p3, __byte_perm(a0, a1, 0x5410),
                         __byte_perm(b0, b1, 0x5410));
                mma16816(o[x][2 * w + 1], p0, p1, p2, p3, __byte_perm(a0, a1, 0x7632),
                         __byte_perm(b0, b1, 0x7632));
            }
        if (next) load_v(g + kTokWarps);
    }

    // the warps' parts meet in shared memory.  o[x][e][2 y + c] is row n + 8 y, column
    // 64 x + (2 t + c) E + e.
#pragma unroll
    for (int y = 0; y < 2; y++) {
        l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
        l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
        const int r = n + 8 * y;
        if (t == 0) {
            sml[warp][r][0] = m[y];
            sml[warp][r][1] = l[y];
        }
#pragma unroll
        for (int x = 0; x < VH; x++)
#pragma unroll
            for (int c = 0; c < 2; c++)
#pragma unroll
                for (int e = 0; e < E; e += 4)
                    *reinterpret_cast<float4 *>(&so[warp][r][64 * x + (2 * t + c) * E + e]) =
                        make_float4(o[x][e][2 * y + c], o[x][e + 1][2 * y + c],
                                    o[x][e + 2][2 * y + c], o[x][e + 3][2 * y + c]);
    }
    __syncthreads();
    for (int at = threadIdx.x; at < 16 * (D / 4); at += kTokThreads) {
        const int r = at / (D / 4), c = at % (D / 4) * 4;
        const int rr = u.rt * 16 + r;
        if (rr >= rows) continue;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kTokWarps; w++) mx = fmaxf(mx, sml[w][r][0]);
        const float safe = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kTokWarps; w++) {
            const float f = fast_exp2(sml[w][r][0] - safe);
            const float4 x = *reinterpret_cast<const float4 *>(&so[w][r][c]);
            sum += f * sml[w][r][1];
            acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
        }
        if (a.splits > 1) {
            float *dst = part_row(a, u, r);
            *reinterpret_cast<float2 *>(dst + c) = make_float2(acc.x, acc.y);
            *reinterpret_cast<float2 *>(dst + c + 2) = make_float2(acc.z, acc.w);
            if (c == 0) *reinterpret_cast<float2 *>(dst + D) = make_float2(mx, sum);
        } else {
            const int i = rr / p.G, h = u.hk * p.G + rr % p.G;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            *reinterpret_cast<uint2 *>(out + u.b * p.o.batch + h * p.o.head + i * p.o.token + c) =
                make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
            if (c == 0) write_lse<float>(p, lse, u.b, h, i, mx, sum);
        }
    }
}

// ---------------------------------------------------------------- float32
// Warp w owns rows w, w + 4, w + 8, w + 12 of the tile; lane = key in the logits and
// column (mod 32) in the output.
template <int D>
__global__ void __launch_bounds__(kTokThreads)
token_f32_kernel(TokenArgs a, const float *q, const float *k, const float *v, float *out,
                 float *lse) {
    constexpr int P = D + 4;
    __shared__ __align__(16) float sq[16 * D];
    __shared__ __align__(16) float sk[32 * P];
    __shared__ __align__(16) float sv[32 * D];
    const WinProblem &p = a.p;
    const TokenUnit u = token_unit<32>(a);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = p.Nq * p.G;
    const float *kb = k + u.hk * p.k.head + (p.table ? 0 : u.b * p.k.batch);
    const float *vb = v + u.hk * p.v.head + (p.table ? 0 : u.b * p.v.batch);
    const KeyPlace kp = key_place(p, u.b, p.k.token, p.k.batch, a.status);
    const KeyPlace vp = key_place(p, u.b, p.v.token, p.v.batch, a.status);
    for (int x = threadIdx.x; x < 16 * D / 4; x += kTokThreads) {
        const int r = x / (D / 4), c = x % (D / 4) * 4, rr = u.rt * 16 + r;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (rr < rows)
            y = *reinterpret_cast<const float4 *>(q + u.b * p.q.batch +
                                                  (u.hk * p.G + rr % p.G) * p.q.head +
                                                  (rr / p.G) * p.q.token + c);
        *reinterpret_cast<float4 *>(sq + r * D + c) = y;
    }
    RowKeys rk[4];
    float m[4], l[4], o[4][D / 32];
#pragma unroll
    for (int x = 0; x < 4; x++) {
        const int rr = u.rt * 16 + warp + 4 * x;
        rk[x] = RowKeys{0, 0, 0};
        if (rr < rows) rk[x] = row_keys(p, u.seq, rr / p.G);
        m[x] = -INFINITY;
        l[x] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 32; c++) o[x][c] = 0.f;
    }
    for (int g = u.g0; g < u.g1; g++) {
        const int j0 = u.kt.tile(g) * 32;
        __syncthreads();
        for (int x = threadIdx.x; x < 32 * D / 4; x += kTokThreads) {
            const int r = x / (D / 4), c = x % (D / 4) * 4, j = j0 + r;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f), z = y;
            if (u.any.sees(j)) {
                const int64_t ka = kp.at(j), va = vp.at(j);
                if (ka >= 0) y = *reinterpret_cast<const float4 *>(kb + ka + c);
                if (va >= 0) z = *reinterpret_cast<const float4 *>(vb + va + c);
            }
            *reinterpret_cast<float4 *>(sk + r * P + c) = y;
            *reinterpret_cast<float4 *>(sv + r * D + c) = z;
        }
        __syncthreads();
        const int j = j0 + lane;
        const bool there = u.any.sees(j) && kp.at(j) >= 0;
#pragma unroll
        for (int x = 0; x < 4; x++) {
            if (u.rt * 16 + warp + 4 * x >= rows) continue;   // the same for the whole warp
            const float *qr = sq + (warp + 4 * x) * D, *kr = sk + lane * P;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int c = 0; c < D; c += 4) {
                const float4 qa = *reinterpret_cast<const float4 *>(qr + c);
                const float4 ka = *reinterpret_cast<const float4 *>(kr + c);
                acc.x = fmaf(qa.x, ka.x, acc.x);
                acc.y = fmaf(qa.y, ka.y, acc.y);
                acc.z = fmaf(qa.z, ka.z, acc.z);
                acc.w = fmaf(qa.w, ka.w, acc.w);
            }
            const float z = there && rk[x].sees(j)
                                ? ((acc.x + acc.y) + (acc.z + acc.w)) * p.scale_log2
                                : -INFINITY;
            float mx = z;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
            mx = fmaxf(mx, m[x]);
            const float safe = mx == -INFINITY ? 0.f : mx;
            const float alpha = exp2f(m[x] - safe), e = exp2f(z - safe);
            m[x] = mx;
            l[x] = l[x] * alpha + e;
#pragma unroll
            for (int c = 0; c < D / 32; c++) o[x][c] *= alpha;
#pragma unroll 4
            for (int jj = 0; jj < 32; jj++) {
                const float w = __shfl_sync(0xffffffffu, e, jj);
#pragma unroll
                for (int c = 0; c < D / 32; c++)
                    o[x][c] = fmaf(w, sv[jj * D + c * 32 + lane], o[x][c]);
            }
        }
    }
#pragma unroll
    for (int x = 0; x < 4; x++) {
        const int r = warp + 4 * x, rr = u.rt * 16 + r;
        if (rr >= rows) continue;
        float sum = l[x];
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        if (a.splits > 1) {
            float *dst = part_row(a, u, r);
#pragma unroll
            for (int c = 0; c < D / 32; c++) dst[c * 32 + lane] = o[x][c];
            if (lane == 0) dst[D] = m[x], dst[D + 1] = sum;
        } else {
            const int i = rr / p.G, h = u.hk * p.G + rr % p.G;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            float *dst = out + u.b * p.o.batch + h * p.o.head + i * p.o.token;
#pragma unroll
            for (int c = 0; c < D / 32; c++) dst[c * 32 + lane] = o[x][c] * inv;
            if (lane == 0) write_lse<float>(p, lse, u.b, h, i, m[x], sum);
        }
    }
}

// ---------------------------------------------------------------- join
// One warp a row (query, head): the parts of its splits in order, so the result does
// not depend on which CTA came first.
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
        a.part + ((bh * a.row_tiles + rr / 16) * a.splits * 16 + rr % 16) * (int64_t)d2;
    const int64_t step = 16 * (int64_t)d2;
    float mx = -INFINITY;
    for (int s = lane; s < a.splits; s += 32) mx = fmaxf(mx, part[s * step + p.d]);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    const float safe = mx == -INFINITY ? 0.f : mx;
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
    for (int s = 0; s < a.splits; s++) {
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
    if (lane == 0) write_lse<T>(p, lse, b, h, i, mx, sum);
}

template <typename T>
cudaError_t join(const TokenArgs &a, T *out, float *lse, cudaStream_t stream) {
    const int64_t rows = (int64_t)a.p.B * a.p.H * a.p.Nq;
    token_join_kernel<T><<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(a, out, lse);
    return cudaGetLastError();
}

}  // namespace

// Splits: enough CTAs for the 148 SMs several times over (the loads in flight of about
// eight warps an SM cover the memory's latency), and no part below four groups of keys
// a warp, where the join would cost more than the split saves.
TokenPlan token_plan(const WinProblem &p, monarch_dtype dtype) {
    TokenPlan t;
    t.row_tiles = (p.Nq * p.G + 15) / 16;
    const int64_t units = (int64_t)p.B * p.Hkv * t.row_tiles;
    // the most keys that one tile of rows can see
    int64_t most = p.Nk;
    if (p.left >= 0 && p.right >= 0) {
        const int64_t span = ((int64_t)p.left + p.right + 1) * p.frame + p.Nq + p.frame;
        most = min(most, span + min(p.sink_end, (int64_t)p.Nk));
    }
    const int64_t group = dtype == MONARCH_BF16 ? 64 : 32;   // keys of one step of a CTA
    const int64_t want = (148 * 8 + units - 1) / units;
    const int64_t room = max((int64_t)1, most / (group * 2));
    t.splits = (int)max((int64_t)1, min(min(want, room), (int64_t)1024));
    t.bytes = t.splits > 1 ? (size_t)units * t.splits * 16 * (p.d + 2) * sizeof(float) : 0;
    return t;
}

cudaError_t token_forward(const WinProblem &p, monarch_dtype dtype, const TokenPlan &plan,
                          const void *q, const void *k, const void *v, void *out, float *lse,
                          void *workspace, int *status, cudaStream_t stream) {
    TokenArgs a{p, plan.row_tiles, plan.splits, (float *)workspace, status};
    const dim3 grid(plan.splits, plan.row_tiles, p.B * p.Hkv);
    if (dtype == MONARCH_F32) {
        const float *qf = (const float *)q, *kf = (const float *)k, *vf = (const float *)v;
        float *of = (float *)out;
        if (p.d == 32)
            token_f32_kernel<32><<<grid, kTokThreads, 0, stream>>>(a, qf, kf, vf, of, lse);
        else if (p.d == 64)
            token_f32_kernel<64><<<grid, kTokThreads, 0, stream>>>(a, qf, kf, vf, of, lse);
        else
            token_f32_kernel<128><<<grid, kTokThreads, 0, stream>>>(a, qf, kf, vf, of, lse);
        cudaError_t e = cudaGetLastError();
        return e != cudaSuccess || plan.splits == 1 ? e : join<float>(a, of, lse, stream);
    }
    const __nv_bfloat16 *qb = (const __nv_bfloat16 *)q, *kb = (const __nv_bfloat16 *)k;
    const __nv_bfloat16 *vb = (const __nv_bfloat16 *)v;
    __nv_bfloat16 *ob = (__nv_bfloat16 *)out;
    if (p.d == 32)
        token_bf16_kernel<32><<<grid, kTokThreads, 0, stream>>>(a, qb, kb, vb, ob, lse);
    else if (p.d == 64)
        token_bf16_kernel<64><<<grid, kTokThreads, 0, stream>>>(a, qb, kb, vb, ob, lse);
    else
        token_bf16_kernel<128><<<grid, kTokThreads, 0, stream>>>(a, qb, kb, vb, ob, lse);
    cudaError_t e = cudaGetLastError();
    return e != cudaSuccess || plan.splits == 1 ? e : join<__nv_bfloat16>(a, ob, lse, stream);
}

}  // namespace win
}  // namespace monarch
