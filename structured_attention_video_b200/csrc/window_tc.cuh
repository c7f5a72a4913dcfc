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

// Four K-steps (K = 64) of D (+)= A B^T, both operands one K-major 128-byte swizzled
// panel of 64 columns: K-step k starts 32 k bytes into the panel.
__device__ __forceinline__ void mma4_ss_k64(uint32_t d_tmem, uint64_t a, uint64_t b,
                                            uint32_t idesc, uint32_t acc0) {
    asm volatile(
        "{\n\t.reg .pred e, p0;\n\t"
        ".reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.and.b32 p0, %4, 0, e;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc0)
        : "memory");
}

// D = A B^T over a head of D elements: panels of 64 columns, 16 KB apart (128 rows each).
template <int D>
__device__ __forceinline__ void mma_ss_head(uint32_t d_tmem, uint64_t a, uint64_t b,
                                            uint32_t idesc) {
    if (D == 128)
        mma8_ss_k128(d_tmem, a, b, idesc, 0u);
    else
        mma4_ss_k64(d_tmem, a, b, idesc, 0u);
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
