// window_tc.cuh -- what the bfloat16 kernels of the window attention share: products on
// tensor memory (window_sm100.cu) and the tensor maps (window_sm100.cu, window_token.cu).
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
