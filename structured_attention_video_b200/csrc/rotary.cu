// rotary.cu -- rotary positions of queries and keys, one axis or up to three
// (frame, row, column), and their backward (the rotation by the negative angle).
//
//   (a, b) -> magnitude (a cos t - b sin t, a sin t + b cos t),
//   t = position(axis of the pair) * frequency(pair).
//
// Bound by memory: every element is read once and written once.  A thread keeps one
// 16-byte chunk of the head dimension (of both halves in the half layout) of one
// token, computes its sines and cosines once, and walks the heads of q and k with
// several loads in flight.
//
// Angles.  The frequency in turns per position becomes a 64-bit binary fraction, so
// position * frequency mod 1 is one wrapping integer product, exact up to
// position * 2^-64 and the 2^-53 of the given frequency: far positions lose nothing.
// The top bits give the quarter turn, and the rest (at most an eighth of a turn to
// either side) keeps 24 significant bits in float32.
#include "rotary.cuh"

namespace monarch {
namespace rot {
namespace {

constexpr int kThreads = 256;

// 16 bytes of a row: as they are, and as floats.
template <typename T> struct Chunk;
template <> struct Chunk<float> {
    static constexpr int n = 4;
    __device__ static __forceinline__ void floats(const uint4 &v, float (&x)[4]) {
        x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
    }
    __device__ static __forceinline__ uint4 bits(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
};
template <> struct Chunk<__nv_bfloat16> {
    static constexpr int n = 8;
    __device__ static __forceinline__ void floats(const uint4 &v, float (&x)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ static __forceinline__ uint4 bits(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// cos and sin of pair `i` at the token's positions.
__device__ __forceinline__ void turn(const RotaryProblem &p, const int64_t (&pos)[3], int i,
                                     float &c, float &s) {
    const int axis = (i >= p.end[0]) + (i >= p.end[1]);
    double f = p.freqs[i] * 0.15915494309189533577;   // 1 / (2 pi)
    f -= floor(f);
    const uint64_t step = (uint64_t)(f * 18446744073709551616.0);
    const int64_t at = axis == 0 ? pos[0] : axis == 1 ? pos[1] : pos[2];
    const uint32_t phase = (uint32_t)(((uint64_t)at * step) >> 32);
    const uint32_t quarter = (phase + (1u << 29)) >> 30;
    const int rest = (int)(phase - (quarter << 30));    // an eighth of a turn to either side
    float sr, cr;
    sincospif((float)rest * 4.656612873077393e-10f, &sr, &cr);   // 2^-31: half turns
    c = quarter & 1 ? -sr : cr;
    s = quarter & 1 ? cr : sr;
    if (quarter & 2) c = -c, s = -s;
    c *= p.magnitude;
    s *= p.inverse ? -p.magnitude : p.magnitude;
}

__device__ __forceinline__ void token_position(const RotaryProblem &p, int b, int n,
                                               int64_t (&pos)[3]) {
    if (p.positions) {
        const int32_t *at = p.positions + b * p.pos_batch + n * p.pos_token;
        pos[0] = at[0];
        pos[1] = p.axes > 1 ? at[1] : 0;
        pos[2] = p.axes > 2 ? at[2] : 0;
        return;
    }
    const int64_t first = p.starts ? (int64_t)p.starts[b] : p.start;
    if (p.gh > 0) {
        const int hw = p.gh * p.gw;
        pos[0] = first + n / hw;
        pos[1] = n % hw / p.gw;
        pos[2] = n % p.gw;
    } else {
        pos[0] = first + n;
        pos[1] = pos[2] = 0;
    }
}

// HALF: pairs (i, i + pairs), chunks of both halves in one thread; else pairs
// (2 i, 2 i + 1) inside a chunk.  Items of a token: the rotated chunks, then the
// chunks behind the rotated part, which are copied (or, in place, left alone).  A block has
// `tokens` whole tokens.  The heads go in batches whose loads are issued together, the
// first batch's before the sines and cosines are computed.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads)
rotary_kernel(RotaryProblem p, int items, int rotated, int tokens, const T *q, const T *k, T *qo,
              T *ko) {
    constexpr int V = Chunk<T>::n, U = HALF ? 3 : 4, P = HALF ? V : V / 2;
    const int t = (int)threadIdx.x / items, item = (int)threadIdx.x - t * items;
    const unsigned tok = blockIdx.x * tokens + t;
    if (t >= tokens || tok >= (unsigned)p.B * p.N) return;
    const int b = tok / (unsigned)p.N, n = tok - b * p.N;
    const bool copy = item >= rotated;
    const int x0 = copy && HALF ? 2 * p.pairs + (item - rotated) * V : item * V;

    // heads [h0, h1) of q's and then k's
    const int heads = p.H + p.Hkv;
    const int h0 = blockIdx.y * p.heads_per_block, h1 = min(heads, h0 + p.heads_per_block);
    const int64_t iq = b * p.q.batch + n * p.q.token + x0, ik = b * p.k.batch + n * p.k.token + x0;
    const int64_t oq = b * p.qo.batch + n * p.qo.token + x0,
                  ok = b * p.ko.batch + n * p.ko.token + x0;
    auto source = [&](int h) {
        return h < p.H ? q + iq + h * p.q.head : k + ik + (h - p.H) * p.k.head;
    };
    auto target = [&](int h) {
        return h < p.H ? qo + oq + h * p.qo.head : ko + ok + (h - p.H) * p.ko.head;
    };
    uint4 a[U], c[HALF ? U : 1];
    auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (h + u >= h1) break;
            const T *src = source(h + u);
            a[u] = __ldcs(reinterpret_cast<const uint4 *>(src));
            if (HALF && !copy) c[u] = __ldcs(reinterpret_cast<const uint4 *>(src + p.pairs));
        }
    };
    load(h0);

    float cs[P], sn[P];
#pragma unroll
    for (int i = 0; i < P; i++) cs[i] = 1.f, sn[i] = 0.f;
    if (!copy) {
        int64_t pos[3];
        token_position(p, b, n, pos);
#pragma unroll
        for (int i = 0; i < P; i++) {
            const int pair = HALF ? x0 + i : x0 / 2 + i;
            if (pair < p.pairs) turn(p, pos, pair, cs[i], sn[i]);
        }
    }
    // pairs of an interleaved chunk that turn; the words behind them stay as they are
    const int turning = HALF || copy ? P : min(P, p.pairs - x0 / 2);
    for (int h = h0; h < h1; h += U) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (h + u >= h1) break;
            T *dst = target(h + u);
            if (copy) {
                if (dst != source(h + u)) __stcs(reinterpret_cast<uint4 *>(dst), a[u]);
                continue;
            }
            float x[V], r[V];
            Chunk<T>::floats(a[u], x);
            if (HALF) {
                float y[V], s[V];
                Chunk<T>::floats(c[u], y);
#pragma unroll
                for (int i = 0; i < V; i++) {
                    r[i] = x[i] * cs[HALF ? i : 0] - y[i] * sn[HALF ? i : 0];
                    s[i] = x[i] * sn[HALF ? i : 0] + y[i] * cs[HALF ? i : 0];
                }
                __stcs(reinterpret_cast<uint4 *>(dst + p.pairs), Chunk<T>::bits(s));
            } else {
#pragma unroll
                for (int i = 0; i < V / 2; i++) {
                    r[2 * i] = x[2 * i] * cs[i] - x[2 * i + 1] * sn[i];
                    r[2 * i + 1] = x[2 * i] * sn[i] + x[2 * i + 1] * cs[i];
                }
            }
            uint4 bits = Chunk<T>::bits(r);
            if (turning < P) {   // (word w holds part of pair w P / 4)
                if (turning <= 0) bits.x = a[u].x;
                if (turning <= P / 4) bits.y = a[u].y;
                if (turning <= P / 2) bits.z = a[u].z;
                if (turning <= 3 * P / 4) bits.w = a[u].w;
            }
            __stcs(reinterpret_cast<uint4 *>(dst), bits);
        }
        if (h + U < h1) load(h + U);
    }
}

// The half layout where a chunk would cross the halves (pairs not a multiple of the
// chunk): one pair, or one copied element, a thread.
template <typename T>
__global__ void __launch_bounds__(kThreads)
rotary_half_pairs_kernel(RotaryProblem p, const T *q, const T *k, T *qo, T *ko) {
    const int items = p.d - p.pairs;
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (id >= (int64_t)p.B * p.N * items) return;
    const int item = (int)(id % items);
    const int64_t tok = id / items;
    const int n = (int)(tok % p.N), b = (int)(tok / p.N);
    const bool copy = item >= p.pairs;
    const int x0 = copy ? item + p.pairs : item;
    float c = 1.f, s = 0.f;
    if (!copy) {
        int64_t pos[3];
        token_position(p, b, n, pos);
        turn(p, pos, item, c, s);
    }
    const int heads = p.H + p.Hkv;
    const int h0 = blockIdx.y * p.heads_per_block, h1 = min(heads, h0 + p.heads_per_block);
    for (int hh = h0; hh < h1; hh++) {
        const bool isq = hh < p.H;
        const int h = isq ? hh : hh - p.H;
        const Strides &si = isq ? p.q : p.k, &so = isq ? p.qo : p.ko;
        const T *src = (isq ? q : k) + b * si.batch + h * si.head + n * si.token + x0;
        T *dst = (isq ? qo : ko) + b * so.batch + h * so.head + n * so.token + x0;
        const float x = to_f32(src[0]);
        if (copy) {
            dst[0] = src[0];
        } else {
            const float y = to_f32(src[p.pairs]);
            dst[0] = from_f32<T>(x * c - y * s);
            dst[p.pairs] = from_f32<T>(x * s + y * c);
        }
    }
}

template <typename T>
cudaError_t run(RotaryProblem p, const void *q, const void *k, void *qo, void *ko,
                cudaStream_t stream) {
    constexpr int V = Chunk<T>::n;
    const bool half = p.half, pairwise = half && p.pairs % V != 0;
    const int rotated = half ? p.pairs / V : (2 * p.pairs + V - 1) / V;
    const int items = pairwise ? p.d - p.pairs
                      : half   ? rotated + (p.d - 2 * p.pairs) / V
                               : p.d / V;
    // (an item is 16 bytes: at most 256 of them at d = 1024)
    const int tokens = pairwise ? 0 : kThreads / items;
    const int64_t all = (int64_t)p.B * p.N;
    const int64_t blocks =
        pairwise ? (all * items + kThreads - 1) / kThreads : (all + tokens - 1) / tokens;
    // few tokens: the heads spread over blocks as well, so that the loads of a short
    // call run side by side instead of one after another
    const int heads = p.H + p.Hkv;
    const int64_t want = (148 * 8 + blocks - 1) / blocks;
    const int groups = (int)(want < heads ? want : heads);
    p.heads_per_block = (heads + groups - 1) / groups;
    const dim3 grid((unsigned)blocks, (heads + p.heads_per_block - 1) / p.heads_per_block);
    const T *qq = (const T *)q, *kk = (const T *)k;
    T *oq = (T *)qo, *ok = (T *)ko;
    if (pairwise)
        rotary_half_pairs_kernel<T><<<grid, kThreads, 0, stream>>>(p, qq, kk, oq, ok);
    else if (half)
        rotary_kernel<T, true><<<grid, kThreads, 0, stream>>>(p, items, rotated, tokens, qq, kk, oq, ok);
    else
        rotary_kernel<T, false><<<grid, kThreads, 0, stream>>>(p, items, rotated, tokens, qq, kk, oq, ok);
    return cudaGetLastError();
}

}  // namespace

cudaError_t rotary_forward(const RotaryProblem &p, monarch_dtype dtype, const void *q,
                           const void *k, void *qo, void *ko, cudaStream_t stream) {
    return dtype == MONARCH_F32 ? run<float>(p, q, k, qo, ko, stream)
                                : run<__nv_bfloat16>(p, q, k, qo, ko, stream);
}

}  // namespace rot
}  // namespace monarch
