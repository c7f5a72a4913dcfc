// window_api.cu -- the C ABI of the window attention, the paged attention and the
// rotary positions: argument validation, workspace sizing and dispatch.
#include "rotary.cuh"
#include "window_common.cuh"

#include <math.h>

namespace monarch {
namespace {

using win::WinGrads;
using win::WinProblem;

constexpr int kPathSimt = 0, kPathTensor = 1, kPathToken = 2;

bool aligned(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Strides in elements: positive, 16-byte multiples, and no byte offset past what the
// tensor maps (40 bits) and 64-bit addressing hold.
monarch_status check_strides(const monarch_strides &s, int64_t elements, int64_t size) {
    const int64_t all[3] = {s.batch, s.head, s.token};
    for (int64_t x : all) {
        if (x <= 0) return MONARCH_ERR_INVALID_ARG;
        if (x % elements) return MONARCH_ERR_ALIGN;
        if (x >= (1LL << 40) / size) return MONARCH_ERR_SHAPE;
    }
    return MONARCH_OK;
}

win::Strides to_win(const monarch_strides &s) { return {s.batch, s.head, s.token}; }
rot::Strides to_rot(const monarch_strides &s) { return {s.batch, s.head, s.token}; }

monarch_status validate_window(const monarch_window_desc *c, WinProblem *p) {
    if (!c) return MONARCH_ERR_INVALID_ARG;
    if (c->B < 1 || c->H < 1 || c->Hkv < 1 || c->Nq < 1 || c->Nk < 1 || c->d < 1 ||
        c->frame < 1 || c->left < -1 || c->right < -1 || c->sinks < 0)
        return MONARCH_ERR_INVALID_ARG;
    if (c->dtype != MONARCH_F32 && c->dtype != MONARCH_BF16) return MONARCH_ERR_INVALID_ARG;
    if (!(c->scale > 0.f) || !isfinite(c->scale)) return MONARCH_ERR_INVALID_ARG;
    if (c->d != 32 && c->d != 64 && c->d != 128) return MONARCH_ERR_UNSUPPORTED;
    if (c->H % c->Hkv) return MONARCH_ERR_SHAPE;
    if ((int64_t)c->B * c->H > 65535 || c->Nq > (1 << 30) || c->Nk > (1 << 30) ||
        (int64_t)c->B * c->H * c->Nq >= (1LL << 33) || (int64_t)c->B * c->Hkv * c->Nk >= (1LL << 33))
        return MONARCH_ERR_SHAPE;
    const int64_t size = c->dtype == MONARCH_BF16 ? 2 : 4;
    const monarch_strides *all[4] = {&c->q, &c->k, &c->v, &c->out};
    for (const monarch_strides *s : all) {
        const monarch_status st = check_strides(*s, 16 / size, size);
        if (st != MONARCH_OK) return st;
    }
    p->B = c->B;
    p->H = c->H;
    p->Hkv = c->Hkv;
    p->G = c->H / c->Hkv;
    p->Nq = c->Nq;
    p->Nk = c->Nk;
    p->d = c->d;
    p->frame = c->frame;
    p->left = c->left;
    p->right = c->right;
    p->sink_end = (int64_t)c->sinks * c->frame;
    p->scale = c->scale;
    p->scale_log2 = (float)((double)c->scale * 1.4426950408889634);
    p->lengths = c->lengths;
    p->starts = c->starts;
    p->newest = c->start == MONARCH_NEWEST;
    p->start = p->newest ? 0 : c->start;
    p->table = nullptr;
    p->table_stride = 0;
    p->page_shift = 0;
    p->num_pages = 0;
    p->q = to_win(c->q);
    p->k = to_win(c->k);
    p->v = to_win(c->v);
    p->o = to_win(c->out);
    return MONARCH_OK;
}

// Few query rows a key head leave the tensor-core tiles of 128 rows mostly empty and,
// with them, most SMs without work: up to 64 rows the token kernels run.  These / those, us,
// everything visible, bfloat16: 8 x 4096 keys, 8 key heads of 128 82 / 130 at 64 rows and
// 144 / 130 at 128; 2000 keys, 12 heads of 128 17 / 33 and 31 / 33; 16 x 1000 keys, 16 heads
// of 64 42 / 41 at 32 rows and 64 / 41 at 64 (many heads fill the SMs by themselves).
// float32: 8 x 4096 keys 840 / 1060 at 64 rows, 2000 keys 62 / 45 at 32.
int choose(const WinProblem &p, monarch_dtype dtype) {
    if ((int64_t)p.Nq * p.G <= 64) return kPathToken;
    return dtype == MONARCH_BF16 ? kPathTensor : kPathSimt;
}

size_t at_least_256(size_t n) { return n < 256 ? 256 : n; }

monarch_status status_of(cudaError_t e) { return e == cudaSuccess ? MONARCH_OK : MONARCH_ERR_CUDA; }

// A pointer field whose target (lengths, starts) must be 4-byte aligned.
bool aligned4(const void *p) { return aligned(p, 4); }

// In place means element by element: whether the strides that count are the same.
bool same_place(const monarch_rotary_desc *c, int heads, const monarch_strides &a,
                const monarch_strides &b) {
    return (c->B == 1 || a.batch == b.batch) && (heads == 1 || a.head == b.head) &&
           (c->N == 1 || a.token == b.token);
}

// delta_i of every query row, at the front of the backward's workspace.
size_t delta_bytes(const WinProblem &p) {
    return ((size_t)p.B * p.H * p.Nq * sizeof(float) + 255) & ~(size_t)255;
}

// A workspace for a call that needs `need` bytes (none: anything goes).
monarch_status check_workspace(size_t need, const void *workspace, size_t ws_bytes) {
    if (need == 0) return MONARCH_OK;
    if (!workspace) return MONARCH_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return MONARCH_ERR_ALIGN;
    return ws_bytes < at_least_256(need) ? MONARCH_ERR_NO_MEMORY : MONARCH_OK;
}

monarch_status run_token(const WinProblem &p, monarch_dtype dtype, const void *q, const void *k,
                         const void *v, void *out, float *lse, void *workspace, size_t ws_bytes,
                         cudaStream_t stream) {
    const win::TokenPlan plan = win::token_plan(p, dtype);
    const monarch_status ws = check_workspace(plan.bytes, workspace, ws_bytes);
    if (ws != MONARCH_OK) return ws;
    int *status = device_status_word();
    if (!status) return MONARCH_ERR_CUDA;
    return status_of(
        win::token_forward(p, dtype, plan, q, k, v, out, lse, workspace, status,
                           device_wait_limit(), stream));
}

// The page table's part of a paged call; p comes from validate_window.
monarch_status validate_paged(const monarch_window_desc *c, WinProblem *p) {
    if (!c) return MONARCH_ERR_INVALID_ARG;
    const monarch_status st = validate_window(c, p);
    if (st != MONARCH_OK) return st;
    if (c->Nq != 1) return MONARCH_ERR_SHAPE;
    p->newest = 1;
    p->start = 0;
    p->starts = nullptr;
    return MONARCH_OK;
}

}  // namespace
}  // namespace monarch

using namespace monarch;

extern "C" {

size_t monarch_window_attn_workspace_bytes(const monarch_window_desc *desc) {
    WinProblem p;
    if (validate_window(desc, &p) != MONARCH_OK) return 0;
    const int path = choose(p, desc->dtype);
    return at_least_256(path == kPathToken    ? win::token_plan(p, desc->dtype).bytes
                        : path == kPathTensor ? win::tc_forward_bytes(p)
                                              : win::simt_forward_bytes(p));
}

int monarch_window_attn_path(const monarch_window_desc *desc) {
    WinProblem p;
    if (validate_window(desc, &p) != MONARCH_OK) return -1;
    return choose(p, desc->dtype);
}

monarch_status monarch_window_attn_fwd_ws(const monarch_window_desc *desc, const void *q,
                                          const void *k, const void *v, void *out, float *lse,
                                          void *workspace, size_t ws_bytes,
                                          monarch_stream_t stream) {
    if (!q || !k || !v || !out) return MONARCH_ERR_INVALID_ARG;
    WinProblem p;
    const monarch_status st = validate_window(desc, &p);
    if (st != MONARCH_OK) return st;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
        !aligned4(lse) || !aligned4(p.lengths) || !aligned4(p.starts))
        return MONARCH_ERR_ALIGN;
    const int path = choose(p, desc->dtype);
    cudaStream_t s = (cudaStream_t)stream;
    if (path == kPathToken)
        return run_token(p, desc->dtype, q, k, v, out, lse, workspace, ws_bytes, s);
    const monarch_status ws = check_workspace(
        path == kPathSimt ? win::simt_forward_bytes(p) : win::tc_forward_bytes(p), workspace, ws_bytes);
    if (ws != MONARCH_OK) return ws;
    if (path == kPathSimt)
        return status_of(win::simt_forward(p, (const float *)q, (const float *)k, (const float *)v,
                                           (float *)out, lse, workspace, s));
    int *status = device_status_word();
    if (!status) return MONARCH_ERR_CUDA;
    return status_of(
        win::tc_forward(p, q, k, v, out, lse, workspace, status, device_wait_limit(), s));
}

size_t monarch_window_attn_bwd_workspace_bytes(const monarch_window_desc *desc) {
    WinProblem p;
    if (validate_window(desc, &p) != MONARCH_OK) return 0;
    return at_least_256(delta_bytes(p) +
                        (desc->dtype == MONARCH_BF16 ? win::mma_backward_bytes(p)
                                                     : win::simt_backward_bytes(p)));
}

monarch_status monarch_window_attn_bwd_ws(const monarch_window_desc *desc,
                                          const monarch_window_grads *grads, const void *q,
                                          const void *k, const void *v, const void *out,
                                          const float *lse, const void *dout, void *dq, void *dk,
                                          void *dv, void *workspace, size_t ws_bytes,
                                          monarch_stream_t stream) {
    if (!grads || !q || !k || !v || !out || !lse || !dout || !dq || !dk || !dv || !workspace)
        return MONARCH_ERR_INVALID_ARG;
    WinProblem p;
    monarch_status st = validate_window(desc, &p);
    if (st != MONARCH_OK) return st;
    const int64_t size = desc->dtype == MONARCH_BF16 ? 2 : 4;
    const monarch_strides *all[4] = {&grads->dout, &grads->dq, &grads->dk, &grads->dv};
    for (const monarch_strides *x : all) {
        st = check_strides(*x, 16 / size, size);
        if (st != MONARCH_OK) return st;
    }
    const void *ptrs[8] = {q, k, v, out, dout, dq, dk, dv};
    for (const void *x : ptrs)
        if (!aligned(x, 16)) return MONARCH_ERR_ALIGN;
    if (!aligned4(lse) || !aligned4(p.lengths) || !aligned4(p.starts) || !aligned(workspace, 256))
        return MONARCH_ERR_ALIGN;
    if (ws_bytes < monarch_window_attn_bwd_workspace_bytes(desc)) return MONARCH_ERR_NO_MEMORY;
    const WinGrads g{to_win(grads->dout), to_win(grads->dq), to_win(grads->dk), to_win(grads->dv)};
    cudaStream_t s = (cudaStream_t)stream;
    float *delta = (float *)workspace;
    void *parts = (char *)workspace + delta_bytes(p);
    if (desc->dtype == MONARCH_F32)
        return status_of(win::simt_backward(p, g, (const float *)q, (const float *)k,
                                            (const float *)v, (const float *)out, lse, delta,
                                            (const float *)dout, (float *)dq, (float *)dk,
                                            (float *)dv, parts, s));
    int *status = device_status_word();
    if (!status) return MONARCH_ERR_CUDA;
    return status_of(win::mma_backward(p, g, q, k, v, out, lse, delta, dout, dq, dk, dv, parts,
                                       status, device_wait_limit(), s));
}

size_t monarch_paged_attn_workspace_bytes(const monarch_window_desc *desc) {
    WinProblem p;
    if (validate_paged(desc, &p) != MONARCH_OK) return 0;
    return at_least_256(win::token_plan(p, desc->dtype).bytes);
}

monarch_status monarch_paged_attn_ws(const monarch_window_desc *desc, const void *q,
                                     const void *k_pages, const void *v_pages,
                                     const int32_t *page_table, int64_t table_stride,
                                     int32_t page_size, int32_t num_pages, void *out, float *lse,
                                     void *workspace, size_t ws_bytes, monarch_stream_t stream) {
    if (!q || !k_pages || !v_pages || !page_table || !out)
        return MONARCH_ERR_INVALID_ARG;
    WinProblem p;
    const monarch_status st = validate_paged(desc, &p);
    if (st != MONARCH_OK) return st;
    if (!p.lengths || num_pages < 1) return MONARCH_ERR_INVALID_ARG;
    if (page_size < 8 || page_size > 65536 || (page_size & (page_size - 1)))
        return MONARCH_ERR_UNSUPPORTED;
    if (p.Nk % page_size || (p.B > 1 && table_stride < p.Nk / page_size)) return MONARCH_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) ||
        !aligned4(page_table) || !aligned4(lse) || !aligned4(p.lengths))
        return MONARCH_ERR_ALIGN;
    p.table = page_table;
    p.table_stride = table_stride;
    p.page_shift = 0;
    while ((1 << p.page_shift) < page_size) p.page_shift++;
    p.num_pages = num_pages;
    return run_token(p, desc->dtype, q, k_pages, v_pages, out, lse, workspace, ws_bytes,
                     (cudaStream_t)stream);
}

monarch_status monarch_rotary(const monarch_rotary_desc *c, const void *q, const void *k,
                              const double *freqs, void *q_out, void *k_out,
                              monarch_stream_t stream) {
    if (!c || !q || !q_out || !freqs) return MONARCH_ERR_INVALID_ARG;
    if (c->B < 1 || c->N < 1 || c->H < 1 || c->Hkv < 0 || c->d < 1 || c->pairs < 1 ||
        c->axes < 1 || c->axes > 3 || (c->half & ~1) || (c->inverse & ~1) || c->grid_h < 0 ||
        c->grid_w < 0)
        return MONARCH_ERR_INVALID_ARG;
    if (c->dtype != MONARCH_F32 && c->dtype != MONARCH_BF16) return MONARCH_ERR_INVALID_ARG;
    if (!isfinite(c->magnitude)) return MONARCH_ERR_INVALID_ARG;
    if (c->Hkv > 0 ? (!k || !k_out) : (k || k_out)) return MONARCH_ERR_INVALID_ARG;
    const int64_t size = c->dtype == MONARCH_BF16 ? 2 : 4, chunk = 16 / size;
    if (c->d > 1024 || c->d % chunk) return MONARCH_ERR_UNSUPPORTED;
    if (2 * (int64_t)c->pairs > c->d || c->N > (1 << 30)) return MONARCH_ERR_SHAPE;
    // token indexes in 32 bits; blocks of the launch: one thread an element of a token at most
    if ((int64_t)c->B * c->N >= (1LL << 31) || (int64_t)c->B * c->N * c->d >= (1LL << 38) ||
        c->H > 32767 || c->Hkv > 32767)
        return MONARCH_ERR_SHAPE;
    int64_t sum = 0;
    for (int i = 0; i < c->axes; i++) {
        if (c->pairs_of_axis[i] < 0) return MONARCH_ERR_INVALID_ARG;
        sum += c->pairs_of_axis[i];
    }
    if (sum != c->pairs) return MONARCH_ERR_SHAPE;
    // one way to get positions: given, along one axis, or on a grid with three
    if (c->positions) {
        if (c->grid_h || c->grid_w || c->starts || c->start) return MONARCH_ERR_INVALID_ARG;
        if (c->pos_batch < 0 || c->pos_token < 0) return MONARCH_ERR_INVALID_ARG;
    } else if (c->axes == 1 ? (c->grid_h || c->grid_w)
                            : (c->axes != 3 || c->grid_h < 1 || c->grid_w < 1)) {
        return MONARCH_ERR_INVALID_ARG;
    } else if (c->axes == 3 && (int64_t)c->grid_h * c->grid_w > (1 << 30)) {
        return MONARCH_ERR_SHAPE;
    }
    const monarch_strides *all[4] = {&c->q, &c->q_out, &c->k, &c->k_out};
    for (int i = 0; i < (c->Hkv ? 4 : 2); i++) {
        const monarch_status st = check_strides(*all[i], chunk, size);
        if (st != MONARCH_OK) return st;
    }
    if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(k_out, 16) ||
        !aligned(freqs, 8) || !aligned4(c->starts) || !aligned4(c->positions))
        return MONARCH_ERR_ALIGN;
    // a thread reads what it writes and nothing else: an output in another place of an input,
    // or two outputs in one place, would hold whatever block came last
    if ((q_out == q && !same_place(c, c->H, c->q, c->q_out)) ||
        (c->Hkv && ((k_out == k && !same_place(c, c->Hkv, c->k, c->k_out)) || q_out == k ||
                    k_out == q || q_out == k_out)))
        return MONARCH_ERR_INVALID_ARG;
    rot::RotaryProblem p;
    p.B = c->B;
    p.N = c->N;
    p.H = c->H;
    p.Hkv = c->Hkv;
    p.d = c->d;
    p.pairs = c->pairs;
    p.axes = c->axes;
    p.end[0] = c->pairs_of_axis[0];
    p.end[1] = c->axes > 1 ? p.end[0] + c->pairs_of_axis[1] : c->pairs;
    p.half = c->half;
    p.inverse = c->inverse;
    p.magnitude = c->magnitude;
    p.gh = c->grid_h;
    p.gw = c->grid_w;
    p.start = c->start;
    p.starts = c->starts;
    p.positions = c->positions;
    p.pos_batch = c->pos_batch;
    p.pos_token = c->pos_token;
    p.freqs = freqs;
    p.heads_per_block = 1;
    p.q = to_rot(c->q);
    p.k = to_rot(c->k);
    p.qo = to_rot(c->q_out);
    p.ko = to_rot(c->k_out);
    return status_of(rot::rotary_forward(p, c->dtype, q, k, q_out, k_out, (cudaStream_t)stream));
}

monarch_status monarch_rotary_frequencies(int pairs, double base, monarch_rotary_scaling scaling,
                                          double factor, double original, double beta_fast,
                                          double beta_slow, double *freqs, double *magnitude) {
    if (!freqs || pairs < 1 || !(base > 1.0) || !isfinite(base)) return MONARCH_ERR_INVALID_ARG;
    if (scaling < MONARCH_ROTARY_PLAIN || scaling > MONARCH_ROTARY_YARN)
        return MONARCH_ERR_INVALID_ARG;
    if (scaling != MONARCH_ROTARY_PLAIN && (!(factor >= 1.0) || !isfinite(factor)))
        return MONARCH_ERR_INVALID_ARG;
    if (scaling == MONARCH_ROTARY_YARN &&
        (!(original > 0.0) || !(beta_slow > 0.0) || !(beta_fast > beta_slow) ||
         !isfinite(original) || !isfinite(beta_fast)))
        return MONARCH_ERR_INVALID_ARG;
    if (magnitude) *magnitude = scaling == MONARCH_ROTARY_YARN ? 0.1 * log(factor) + 1.0 : 1.0;
    if (scaling == MONARCH_ROTARY_NTK && pairs > 1)
        base *= pow(factor, (double)pairs / (pairs - 1));
    // pair i turns original * base^(-i/pairs) / (2 pi) times in the trained length;
    // the index at which that is beta
    const double two_pi = 6.283185307179586476925;
    auto index_of = [&](double beta) {
        return pairs * log(original / (beta * two_pi)) / log(base);
    };
    double low = 0, high = 0;
    if (scaling == MONARCH_ROTARY_YARN) {
        low = fmax(0.0, floor(index_of(beta_fast)));
        high = fmin(2.0 * pairs - 1.0, ceil(index_of(beta_slow)));
        if (high <= low) high = low + 0.001;
    }
    for (int i = 0; i < pairs; i++) {
        const double f = pow(base, -(double)i / pairs);
        if (scaling == MONARCH_ROTARY_LINEAR) {
            freqs[i] = f / factor;
        } else if (scaling == MONARCH_ROTARY_YARN) {
            double blend = (i - low) / (high - low);
            blend = fmin(1.0, fmax(0.0, blend));
            freqs[i] = f * (1.0 - blend) + f / factor * blend;
        } else {
            freqs[i] = f;
        }
    }
    return MONARCH_OK;
}

}  // extern "C"
