// window_tc.cuh -- what the tensor-core forward (window_sm100.cu) and backward
// (window_bwd_sm100.cu) of the window attention share.
#pragma once

#include "monarch_tc_shared.cuh"
#include "window_common.cuh"

namespace monarch {
namespace win {

using namespace tc;
using tcs::align1024;
using tcs::kCleanupPolls;
using tcs::kMaxSmem;
using tcs::kPanel;
using tcs::wait_warp;

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(e));
    return e != 0;
}

__device__ __forceinline__ void mma_one(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_one_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                           uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// D = A B^T over a head of HD elements: A a 128-row tile, B of BROWS rows, both K-major
// 128-byte swizzled panels of 64 columns (a K-step of 16 is 32 bytes inside a panel).
template <int HD, int BROWS>
__device__ __forceinline__ void mma_head(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc) {
#pragma unroll
    for (int k = 0; k < HD / 16; k++)
        mma_one(d_tmem, a + (k >> 2) * (kPanel >> 4) + (k & 3) * 2,
                b + (k >> 2) * (BROWS * 128 >> 4) + (k & 3) * 2, idesc, k > 0);
}

// The same with A in tensor memory (bfloat16 pairs, 8 columns a K-step): shared memory
// then feeds B alone.
template <int HD, int BROWS>
__device__ __forceinline__ void mma_head_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                            uint32_t idesc) {
#pragma unroll
    for (int k = 0; k < HD / 16; k++)
        mma_one_ts(d_tmem, a_tmem + 8 * k, b + (k >> 2) * (BROWS * 128 >> 4) + (k & 3) * 2, idesc,
                   k > 0);
}

// One row of HD bfloat16 elements (d of them real, the others zero) from global memory
// to this lane's row of tensor memory, as the A operand of mma_head_ts.
template <int HD>
__device__ __forceinline__ void row_to_tmem(uint32_t taddr, const __nv_bfloat16 *src, int d,
                                            bool real) {
#pragma unroll
    for (int c = 0; c < HD / 2; c += 32) {
        uint32_t r[32];
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const int x = 2 * c + 8 * e;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (real && x < d) v = *reinterpret_cast<const uint4 *>(src + x);
            r[4 * e] = v.x, r[4 * e + 1] = v.y, r[4 * e + 2] = v.z, r[4 * e + 3] = v.w;
        }
        tmem_st32(taddr + c, r);
    }
    tmem_wait_st();
}

// D (+)= A B over 64 keys or queries: A bfloat16 pairs in tensor memory (8 columns a
// K-step; the second half of A GAP columns behind the first), B an MN-major swizzled block
// (16 rows = 2 KB a K-step).
template <int GAP>
__device__ __forceinline__ void mma_block64(uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                            uint32_t idesc, uint32_t acc) {
#pragma unroll
    for (int k = 0; k < 4; k++)
        mma_one_ts(d_tmem, a_tmem + (k >> 1) * GAP + (k & 1) * 8, b + 128 * k, idesc,
                   k > 0 ? 1u : acc);
}

// Rows [first, last) of a tile of 64-column panels (128-byte rows, panel_bytes apart)
// become zero, by `threads` threads of index `i`.  A whole row is zeroed, so the
// swizzle does not matter.  The caller orders it before the products' reads.
__device__ __forceinline__ void zero_rows(uint8_t *tile, int first, int last, int panels,
                                          uint32_t panel_bytes, int i, int threads) {
    const int n = (last - first) * 8;
    for (int x = i; x < n * panels; x += threads) {
        const int pn = x / n, y = x % n;
        *reinterpret_cast<uint4 *>(tile + pn * panel_bytes + (first + (y >> 3)) * 128 +
                                   (y & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
}

// A [B][heads][tokens][d] tensor as a 4-D map (x, token, head, batch), box of 64
// columns (columns past d read zeros) by `rows` tokens (rows past the tensor read zeros).
inline bool map_tokens(CUtensorMap *m, const void *base, const Strides &s, int B, int heads,
                       int tokens, int d, uint32_t rows) {
    const uint64_t dims[4] = {(uint64_t)d, (uint64_t)tokens, (uint64_t)heads, (uint64_t)B};
    const uint64_t str[3] = {(uint64_t)s.token * 2, (uint64_t)s.head * 2, (uint64_t)s.batch * 2};
    const uint32_t box[4] = {64, rows, 1, 1};
    return tcs::make_map(m, base, 4, dims, str, box);
}

}  // namespace win
}  // namespace monarch
