// window_common.cuh -- exact softmax attention over a window of frames and the
// first frames (sinks): problem description, mask arithmetic and the interfaces
// of its kernel families.
//
//   O_i = sum_j P_ij v_j,  P_ij = exp(scale q_i.k_j - lse_i),
//   lse_i = log sum_j exp(scale q_i.k_j),  j over the keys that query i sees.
//
// The mask of one query row is two intervals of keys: [lo, hi) and [0, sink) cut
// at hi.  lo and hi do not decrease with the query's position, so a tile of query
// rows meets two runs of key tiles and a tile of keys one run of query rows.
#pragma once

#include "monarch_common.cuh"

#include <algorithm>

namespace monarch {
namespace win {

struct Strides {
    int64_t batch, head, token;   // in elements; the head dimension has stride 1
};

// Everything a kernel needs to know about one call.
struct WinProblem {
    int B, H, Hkv, G;             // G = H / Hkv query heads share a key head
    int Nq, Nk, d;
    int frame, left, right;       // tokens per frame; frames seen before and after, -1: all
    int64_t sink_end;             // keys [0, sink_end) stay visible behind the window
    float scale, scale_log2;      // scale, scale * log2(e)
    const int32_t *lengths;       // [B] or null (Nk)
    const int32_t *starts;        // [B] or null
    int start;                    // of every sequence when starts is null
    int newest;                   // starts null: the last query is the newest key
    // behind a page table (one query a sequence): key j of sequence b is row
    // j % page of page table[b * table_stride + j / page]; k.batch and v.batch are then
    // the distances between pages
    const int32_t *table;
    int64_t table_stride;
    int page_shift, num_pages;
    Strides q, k, v, o;
};

// One sequence: its keys and the position of its first query.
struct Sequence {
    int len;
    int64_t start;
};

__device__ __forceinline__ Sequence sequence(const WinProblem &p, int b) {
    Sequence s;
    const int n = p.lengths ? p.lengths[b] : p.Nk;
    s.len = min(max(n, 0), p.Nk);
    s.start = p.starts ? (int64_t)p.starts[b] : p.newest ? (int64_t)s.len - p.Nq : (int64_t)p.start;
    return s;
}

// The sequence of a whole CTA, read once: trip counts and barriers follow from it, so all
// threads must have the same one whatever happens to lengths and starts meanwhile.  The
// first thread reads it; the block meets in share_sequence, and what needs no sequence
// goes between the two.
__device__ __forceinline__ Sequence first_threads_sequence(const WinProblem &p, int b) {
    return threadIdx.x == 0 ? sequence(p, b) : Sequence{0, 0};
}
__device__ __forceinline__ void share_sequence(Sequence &s, Sequence *shared) {
    if (threadIdx.x == 0) *shared = s;
    __syncthreads();
    s = *shared;
}

// Keys of one query row: [lo, hi) and [0, sink), sink <= lo.
struct RowKeys {
    int lo, hi, sink;
    __device__ __forceinline__ bool sees(int j) const {
        return j < hi && (j >= lo || j < sink);
    }
};

// Row i of a sequence (position start + i); a row outside [0, len) sees nothing.
__device__ __forceinline__ RowKeys row_keys(const WinProblem &p, const Sequence &s, int64_t i) {
    RowKeys r{0, 0, 0};
    const int64_t pos = s.start + i;
    if (i < 0 || i >= p.Nq || pos < 0 || pos >= s.len) return r;
    const int64_t f = p.frame == 1 ? pos : (int64_t)((uint32_t)pos / (uint32_t)p.frame);
    int64_t hi = s.len, lo = 0;
    if (p.right >= 0) hi = min(hi, (f + p.right + 1) * p.frame);
    if (p.left >= 0) lo = min(max((f - p.left) * p.frame, (int64_t)0), hi);
    r.lo = (int)lo;
    r.hi = (int)hi;
    r.sink = (int)min(p.sink_end, lo);
    return r;
}

// The real rows among [i0, i1): first and one past the last (empty: first >= last).
__device__ __forceinline__ void real_rows(const WinProblem &p, const Sequence &s, int i0, int i1,
                                          int &first, int &last) {
    first = (int)max((int64_t)i0, min((int64_t)i1, -s.start));
    last = (int)min((int64_t)min(i1, p.Nq), max((int64_t)i0, s.len - s.start));
}

// Key tiles of T keys that query rows [i0, i1) meet: nA tiles from 0 (sinks), then nB
// tiles from tile `first`.
struct KeyTiles {
    int nA, nB, first;
    __device__ __forceinline__ int count() const { return nA + nB; }
    __device__ __forceinline__ int tile(int it) const { return it < nA ? it : first + it - nA; }
};

template <int T>
__device__ __forceinline__ KeyTiles key_tiles(const WinProblem &p, const Sequence &s, int i0,
                                              int i1) {
    int r0, r1;
    real_rows(p, s, i0, i1, r0, r1);
    KeyTiles t{0, 0, 0};
    if (r0 >= r1) return t;
    const RowKeys a = row_keys(p, s, r0), b = row_keys(p, s, r1 - 1);
    t.first = a.lo / T;
    const int end = (b.hi + T - 1) / T;
    // the sinks that the last row's window has passed (it has passed most of all)
    t.nA = min((b.sink + T - 1) / T, t.first);
    t.nB = max(0, end - t.first);
    return t;
}

// Query rows [first, last) that can see a key of [j0, j1).
__device__ __forceinline__ void query_rows(const WinProblem &p, const Sequence &s, int j0, int j1,
                                           int &first, int &last) {
    const int64_t jl = min(j1, s.len);   // one past the last real key
    if (j0 >= jl) {
        first = last = 0;
        return;
    }
    const int64_t f0 = j0 / p.frame, f1 = (jl - 1) / p.frame;
    int64_t lo = 0, hi = s.len;          // positions
    if (p.right >= 0) lo = max((int64_t)0, (f0 - p.right) * p.frame);
    if (p.left >= 0 && j0 >= p.sink_end) hi = min(hi, (f1 + p.left + 1) * p.frame);
    lo = max((int64_t)0, lo - s.start);
    hi = min((int64_t)p.Nq, hi - s.start);
    first = (int)min(lo, (int64_t)p.Nq);
    last = (int)max(hi, (int64_t)0);
}

// Groups of this thread's asynchronous copies (cp.async).
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest N groups of this thread's copies have landed.
template <int N> __device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The most keys that a tile of `rows` queries can meet, from the mask and the tensors' sizes
// (lengths are on the device); the most queries that a tile of keys can.
inline int64_t most_keys(const WinProblem &p, int64_t rows) {
    if (p.left < 0 || p.right < 0) return p.Nk;
    const int64_t span = ((int64_t)p.left + p.right + 1) * p.frame + rows + p.frame;
    return std::min<int64_t>(p.Nk, span + std::min<int64_t>(p.sink_end, p.Nk));
}
inline int64_t most_queries(const WinProblem &p, int64_t keys) {
    if (p.left < 0 || p.right < 0 || p.sink_end > 0) return p.Nq;
    return std::min<int64_t>(p.Nq, ((int64_t)p.left + p.right + 1) * p.frame + keys + p.frame);
}

// The gradients' tensors of a backward call.
struct WinGrads {
    Strides dout, dq, dk, dv;
};

// SIMT kernels, 32-bit arithmetic (window_simt.cu).  Workspace bytes, 0 where none are
// needed.
size_t simt_forward_bytes(const WinProblem &p);
cudaError_t simt_forward(const WinProblem &p, const float *q, const float *k, const float *v,
                         float *out, float *lse, void *workspace, cudaStream_t stream);
size_t simt_backward_bytes(const WinProblem &p);   // of `parts`
cudaError_t simt_backward(const WinProblem &p, const WinGrads &g, const float *q, const float *k,
                          const float *v, const float *out, const float *lse, float *delta,
                          const float *dout, float *dq, float *dk, float *dv, void *parts,
                          cudaStream_t stream);
// Few query rows a key head against many keys, split over the keys (window_token.cu).
struct TokenPlan {
    int row_tiles;   // tiles of 16 rows (query, head of the group) a key head
    int splits;      // parts of the visible keys
    int clusters;    // groups of parts that join inside a thread-block cluster
    size_t bytes;    // workspace: none for one cluster
};
TokenPlan token_plan(const WinProblem &p, monarch_dtype dtype);
cudaError_t token_forward(const WinProblem &p, monarch_dtype dtype, const TokenPlan &plan,
                          const void *q, const void *k, const void *v, void *out, float *lse,
                          void *workspace, int *status, long long limit, cudaStream_t stream);

// Tensor-core kernels, bfloat16 (window_sm100.cu; backward window_bwd_mma.cu).
size_t tc_forward_bytes(const WinProblem &p);   // workspace, 0 where none is needed
cudaError_t tc_forward(const WinProblem &p, const void *q, const void *k, const void *v, void *out,
                       float *lse, void *workspace, int *status, long long limit,
                       cudaStream_t stream);

size_t mma_backward_bytes(const WinProblem &p);   // of `parts`, 0 where none are needed
cudaError_t mma_backward(const WinProblem &p, const WinGrads &g, const void *q, const void *k,
                         const void *v, const void *out, const float *lse, float *delta,
                         const void *dout, void *dq, void *dk, void *dv, void *parts, int *status,
                         long long limit, cudaStream_t stream);

}  // namespace win
}  // namespace monarch
