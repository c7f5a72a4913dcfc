// torch_binding.cpp -- argument checks and marshalling of the window attention, the paged
// attention and the rotary positions: torch tensors onto the C ABI of monarch_attn.h.
//
// A CPython module (monarch_torch) that reads shapes, strides and pointers from the
// tensors' C++ objects.  A short call takes 5.0 us of host time, 3.3 of it the launch; with
// the same checks in Python and ctypes it took 11.5, more than its kernels take on the
// GPU.  Python passes every argument by position; window.py and positions.py hold the
// public signatures.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <array>
#include <cmath>
#include <string>

#include "../../include/monarch_attn.h"

namespace {

using at::Tensor;

PyObject *g_status_error = nullptr;   // MonarchError(status, where)

[[noreturn]] void refuse(const std::string &why) { C10_THROW_ERROR(ValueError, why); }
[[noreturn]] void wrong_type(const std::string &why) { C10_THROW_ERROR(TypeError, why); }

// ---------------------------------------------------------------- arguments
// The positional arguments of a call, taken in order.
struct Args {
    PyObject *const *at;
    Py_ssize_t left;
    PyObject *next() {
        if (left-- <= 0) wrong_type("too few arguments");
        return *at++;
    }
    void end() const {
        if (left != 0) wrong_type("too many arguments");
    }
};

const Tensor &tensor(PyObject *x, const char *name) {
    if (!THPVariable_Check(x)) wrong_type(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(x);
}
bool given(PyObject *x) { return x != Py_None; }

int64_t integer(PyObject *x, const char *name) {
    PyObject *index = PyNumber_Index(x);
    if (!index) {
        PyErr_Clear();
        refuse(std::string(name) + " must be an integer");
    }
    int overflow = 0;
    const int64_t n = PyLong_AsLongLongAndOverflow(index, &overflow);
    Py_DECREF(index);
    if (overflow) refuse(std::string(name) + " out of range");
    return n;
}
int32_t narrow(int64_t n, const char *name) {
    if (n < INT32_MIN || n > INT32_MAX) refuse(std::string(name) + " out of range");
    return (int32_t)n;
}
int32_t int32(PyObject *x, const char *name) { return narrow(integer(x, name), name); }

float real(PyObject *x, const char *name) {
    const double r = PyFloat_AsDouble(x);
    if (r == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(name) + " must be a number");
    }
    return (float)r;
}

// A tuple or list of `least` to `most` integers.
int integers(PyObject *x, int least, int most, int32_t *out, const char *name) {
    if (!PyTuple_Check(x) && !PyList_Check(x)) refuse(std::string(name) + " must be a tuple");
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(x);
    if (n < least || n > most) refuse(std::string(name) + " has the wrong number of entries");
    for (Py_ssize_t i = 0; i < n; i++) out[i] = int32(PySequence_Fast_GET_ITEM(x, i), name);
    return (int)n;
}

bool flag(PyObject *x) {
    const int r = PyObject_IsTrue(x);
    if (r < 0) throw python_error();
    return r != 0;
}

bool is_word(PyObject *x, const char *word) {
    return PyUnicode_Check(x) && PyUnicode_CompareWithASCIIString(x, word) == 0;
}
bool is_bnhd(PyObject *layout) {
    if (is_word(layout, "bhnd")) return false;
    if (!is_word(layout, "bnhd")) refuse("layout must be one of ['bhnd', 'bnhd']");
    return true;
}

// ---------------------------------------------------------------- tensors
void same_device(int dev, const Tensor &t) {
    if (!t.is_cuda() || t.get_device() != dev) refuse("all tensors must be on the same CUDA device");
}
int index_of(const Tensor &t) {
    if (!t.is_cuda()) refuse("all tensors must be on the same CUDA device");
    return (int)t.get_device();
}
monarch_dtype dtype_of(const Tensor &t) {
    if (t.scalar_type() == at::kBFloat16) return MONARCH_BF16;
    if (t.scalar_type() != at::kFloat) refuse("dtype must be float32 or bfloat16");
    return MONARCH_F32;
}
// t is on the first tensor's device and has its type.
void alike(const Tensor &first, const Tensor &t) {
    same_device((int)first.get_device(), t);
    if (t.scalar_type() != first.scalar_type()) refuse("all tensors must share one dtype");
}

// (batch, head, token) strides of a 4-D tensor; a dimension of size 1 gets a stride that
// the library accepts, whatever torch says (it is never used).
monarch_strides strides4(const Tensor &t, bool bnhd) {
    const auto n = t.sizes(), s = t.strides();
    if (s[3] != 1) refuse("tensors must have stride 1 along the head dimension");
    int64_t x[3];
    for (int i = 0; i < 3; i++) x[i] = n[i] == 1 ? n[3] : s[i];
    return bnhd ? monarch_strides{x[0], x[2], x[1]} : monarch_strides{x[0], x[1], x[2]};
}
// The same of [B, H, d], one token.
monarch_strides strides3(const Tensor &t) {
    const auto n = t.sizes(), s = t.strides();
    if (s[2] != 1) refuse("tensors must have stride 1 along the head dimension");
    return {n[0] == 1 ? n[2] : s[0], n[1] == 1 ? n[2] : s[1], n[2]};
}

const int32_t *index_pointer(PyObject *x, const char *name, int64_t B, int dev) {
    const Tensor &t = tensor(x, name);
    if (t.scalar_type() != at::kInt || !t.is_cuda() || t.get_device() != dev || t.dim() != 1 ||
        t.size(0) != B || !t.is_contiguous())
        refuse(std::string(name) +
               " must be a contiguous int32 tensor of [B] on the inputs' device");
    return t.const_data_ptr<int32_t>();
}

// Memory of `need` bytes where a call needs more than none (256; 0: the call itself says
// what is wrong): the caller's, if it is large enough, or new.
struct Workspace {
    Tensor owner;
    void *ptr = nullptr;
    size_t bytes = 0;
    Workspace(size_t need, PyObject *mine, const Tensor &like) {
        if (need <= 256) return;
        if (given(mine)) {
            const Tensor &w = tensor(mine, "workspace");
            if (!w.is_cuda() || w.get_device() != like.get_device() || !w.is_contiguous())
                refuse("workspace must be contiguous and on the inputs' device");
            if ((size_t)w.nbytes() >= need) owner = w;
        }
        if (!owner.defined()) owner = at::empty({(int64_t)need}, like.options().dtype(at::kByte));
        ptr = owner.data_ptr();
        bytes = owner.nbytes();
    }
};

// The tensors' device, current for the rest of a call (workspace sizes depend on it too).
c10::Device on(int dev) { return c10::Device(c10::kCUDA, (c10::DeviceIndex)dev); }

// call(stream) on the device's current stream.
template <typename Call> void launch(int dev, const char *where, const Call &call) {
    const monarch_status status =
        call((monarch_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
    if (status == MONARCH_OK) return;
    PyObject *e = PyObject_CallFunction(g_status_error, "is", (int)status, where);
    if (e) {
        PyErr_SetObject((PyObject *)Py_TYPE(e), e);
        Py_DECREF(e);
    }
    throw python_error();
}

// A new tensor, or the caller's own object.
PyObject *result(const Tensor &t, PyObject *mine) {
    if (!mine || !given(mine)) return THPVariable_Wrap(t);
    Py_INCREF(mine);
    return mine;
}
PyObject *results(PyObject *a, PyObject *b, PyObject *c = nullptr) {
    PyObject *t = a && b ? PyTuple_New(c ? 3 : 2) : nullptr;
    if (!t) {
        Py_XDECREF(a);
        Py_XDECREF(b);
        Py_XDECREF(c);
        return nullptr;
    }
    PyTuple_SET_ITEM(t, 0, a);
    PyTuple_SET_ITEM(t, 1, b);
    if (c) PyTuple_SET_ITEM(t, 2, c);
    return t;
}
PyObject *none() { Py_RETURN_NONE; }

// ---------------------------------------------------------------- window attention
// The mask's part of a description.
void read_mask(monarch_window_desc *d, PyObject *window, PyObject *sinks, PyObject *frame) {
    int32_t w[2];
    integers(window, 2, 2, w, "window");
    d->left = w[0];
    d->right = w[1];
    d->sinks = int32(sinks, "sinks");
    d->frame = int32(frame, "frame");
}
void read_scale(monarch_window_desc *d, PyObject *scale) {
    d->scale = given(scale) ? real(scale, "scale") : d->d > 0 ? (float)(1 / std::sqrt((double)d->d)) : 0.f;
}

// q, k, v, window, sinks, frame, lengths, starts, scale, layout of every window call.
struct WindowCall {
    const Tensor &q, &k, &v;
    monarch_window_desc desc = {};
    bool bnhd;
    int dev;
    explicit WindowCall(Args &a)
        : q(tensor(a.next(), "q")), k(tensor(a.next(), "k")), v(tensor(a.next(), "v")) {
        PyObject *window = a.next(), *sinks = a.next(), *frame = a.next(), *lengths = a.next(),
                 *starts = a.next(), *scale = a.next();
        bnhd = is_bnhd(a.next());
        if (q.dim() != 4 || k.dim() != 4 || k.sizes() != v.sizes())
            refuse("expected 4-D tensors, k and v alike");
        dev = index_of(q);
        desc.dtype = dtype_of(q);
        alike(q, k);
        alike(q, v);
        if (k.size(0) != q.size(0) || k.size(3) != q.size(3))
            refuse("q, k and v must share batch and head dimension");
        const int heads = bnhd ? 2 : 1, tokens = 3 - heads;
        desc.B = narrow(q.size(0), "batch");
        desc.H = narrow(q.size(heads), "heads");
        desc.Hkv = narrow(k.size(heads), "heads");
        desc.Nq = narrow(q.size(tokens), "tokens");
        desc.Nk = narrow(k.size(tokens), "tokens");
        desc.d = narrow(q.size(3), "head dimension");
        read_mask(&desc, window, sinks, frame);
        read_scale(&desc, scale);
        if (!given(starts)) {
            desc.start = MONARCH_NEWEST;
        } else if (THPVariable_Check(starts)) {
            desc.starts = index_pointer(starts, "starts", desc.B, dev);
        } else {
            desc.start = int32(starts, "starts");
            if (desc.start == MONARCH_NEWEST) refuse("starts out of range");
        }
        if (given(lengths)) desc.lengths = index_pointer(lengths, "lengths", desc.B, dev);
        desc.q = strides4(q, bnhd);
        desc.k = strides4(k, bnhd);
        desc.v = strides4(v, bnhd);
    }
    void read_out(const Tensor &out) {
        if (out.sizes() != q.sizes()) refuse("out must have q's shape");
        alike(q, out);
        desc.out = strides4(out, bnhd);
    }
    Tensor new_lse() const {
        return at::empty({desc.B, desc.H, desc.Nq}, q.options().dtype(at::kFloat));
    }
};

// (..., out, return_lse, workspace) -> out or (out, lse)
PyObject *window_attention(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a{args, n};
    WindowCall c(a);
    PyObject *mine = a.next();
    const bool with_lse = flag(a.next());
    PyObject *workspace = a.next();
    a.end();
    const Tensor out = given(mine) ? tensor(mine, "out") : at::empty_like(c.q);
    c.read_out(out);
    if (given(mine) && (out.data_ptr() == c.q.data_ptr() || out.data_ptr() == c.k.data_ptr() ||
                        out.data_ptr() == c.v.data_ptr()))
        refuse("out must not be an input");
    const Tensor lse = with_lse ? c.new_lse() : Tensor();
    const c10::cuda::CUDAGuard guard(on(c.dev));
    const Workspace ws(monarch_window_attn_workspace_bytes(&c.desc), workspace, c.q);
    launch(c.dev, "monarch_window_attn_fwd_ws", [&](monarch_stream_t s) {
        return monarch_window_attn_fwd_ws(&c.desc, c.q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(),
                                          out.data_ptr(), with_lse ? (float *)lse.data_ptr() : nullptr,
                                          ws.ptr, ws.bytes, s);
    });
    PyObject *o = result(out, mine);
    return with_lse ? results(o, THPVariable_Wrap(lse)) : o;
    END_HANDLE_TH_ERRORS
}

// (...) -> path
PyObject *window_attention_path(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a{args, n};
    WindowCall c(a);
    a.end();
    c.desc.out = c.desc.q;
    return PyLong_FromLong(monarch_window_attn_path(&c.desc));
    END_HANDLE_TH_ERRORS
}

// (..., out, lse, dout, workspace) -> (dq, dk, dv)
PyObject *window_attention_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a{args, n};
    WindowCall c(a);
    const Tensor &out = tensor(a.next(), "out"), &lse = tensor(a.next(), "lse"),
                 &dout = tensor(a.next(), "dout");
    PyObject *workspace = a.next();
    a.end();
    c.read_out(out);
    if (dout.sizes() != c.q.sizes()) refuse("dout must have q's shape");
    alike(c.q, dout);
    const std::array<int64_t, 3> rows = {c.desc.B, c.desc.H, c.desc.Nq};
    if (lse.scalar_type() != at::kFloat || lse.sizes() != at::IntArrayRef(rows) ||
        !lse.is_cuda() || lse.get_device() != c.dev || !lse.is_contiguous())
        refuse("lse must be the forward's contiguous float32 [B, H, Nq]");
    const Tensor dq = at::empty_like(c.q), dk = at::empty_like(c.k), dv = at::empty_like(c.v);
    const monarch_window_grads grads = {strides4(dout, c.bnhd), strides4(dq, c.bnhd),
                                        strides4(dk, c.bnhd), strides4(dv, c.bnhd)};
    const c10::cuda::CUDAGuard guard(on(c.dev));
    // (always used: never "none")
    const Workspace ws(std::max<size_t>(257, monarch_window_attn_bwd_workspace_bytes(&c.desc)),
                       workspace, c.q);
    launch(c.dev, "monarch_window_attn_bwd_ws", [&](monarch_stream_t s) {
        return monarch_window_attn_bwd_ws(&c.desc, &grads, c.q.data_ptr(), c.k.data_ptr(),
                                          c.v.data_ptr(), out.data_ptr(), (float *)lse.data_ptr(),
                                          dout.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                          dv.data_ptr(), ws.ptr, ws.bytes, s);
    });
    return results(THPVariable_Wrap(dq), THPVariable_Wrap(dk), THPVariable_Wrap(dv));
    END_HANDLE_TH_ERRORS
}

// (q, k_pages, v_pages, page_table, lengths, window, sinks, frame, scale, layout, out,
// return_lse, workspace) -> out or (out, lse)
PyObject *paged_attention(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a{args, n};
    const Tensor &q = tensor(a.next(), "q"), &k = tensor(a.next(), "k_pages"),
                 &v = tensor(a.next(), "v_pages"), &table = tensor(a.next(), "page_table");
    PyObject *lengths = a.next(), *window = a.next(), *sinks = a.next(), *frame = a.next(),
             *scale = a.next();
    const bool bnhd = is_bnhd(a.next());
    PyObject *mine = a.next();
    const bool with_lse = flag(a.next());
    PyObject *workspace = a.next();
    a.end();
    if (q.dim() != 3 || k.dim() != 4 || k.sizes() != v.sizes())
        refuse("expected q [B, H, d] and 4-D pools of pages, k and v alike");
    const int dev = index_of(q);
    monarch_window_desc desc = {};
    desc.dtype = dtype_of(q);
    alike(q, k);
    alike(q, v);
    const int heads = bnhd ? 2 : 1, tokens = 3 - heads;
    if (k.size(3) != q.size(2)) refuse("the pages must have q's head dimension");
    desc.B = narrow(q.size(0), "batch");
    if (table.scalar_type() != at::kInt || !table.is_cuda() || table.get_device() != dev ||
        table.dim() != 2 || table.size(0) != desc.B || table.stride(1) != 1)
        refuse("page_table must be int32 [B, width] on the inputs' device");
    const int64_t width = table.size(1), page = k.size(tokens);
    if (width < 1 || width > (1 << 30) || page < 1 || page > (1 << 30) || width * page > (1 << 30))
        refuse("page table of " + std::to_string(width) + " pages of " + std::to_string(page) +
               " keys: out of range");
    desc.H = narrow(q.size(1), "heads");
    desc.Hkv = narrow(k.size(heads), "heads");
    desc.Nq = 1;
    desc.Nk = (int32_t)(width * page);
    desc.d = narrow(q.size(2), "head dimension");
    read_mask(&desc, window, sinks, frame);
    read_scale(&desc, scale);
    desc.start = MONARCH_NEWEST;
    desc.lengths = index_pointer(lengths, "lengths", desc.B, dev);
    desc.q = strides3(q);
    desc.k = strides4(k, bnhd);
    desc.v = strides4(v, bnhd);
    const Tensor out = given(mine) ? tensor(mine, "out") : at::empty_like(q);
    if (out.sizes() != q.sizes()) refuse("out must have q's shape");
    alike(q, out);
    if (given(mine) && out.data_ptr() == q.data_ptr()) refuse("out must not be an input");
    desc.out = strides3(out);
    const Tensor lse =
        with_lse ? at::empty({desc.B, desc.H, 1}, q.options().dtype(at::kFloat)) : Tensor();
    const c10::cuda::CUDAGuard guard(on(dev));
    const Workspace ws(monarch_paged_attn_workspace_bytes(&desc), workspace, q);
    launch(dev, "monarch_paged_attn_ws", [&](monarch_stream_t s) {
        return monarch_paged_attn_ws(&desc, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                     (const int32_t *)table.data_ptr(),
                                     desc.B > 1 ? table.stride(0) : width, (int32_t)page,
                                     narrow(k.size(0), "pages"), out.data_ptr(),
                                     with_lse ? (float *)lse.data_ptr() : nullptr, ws.ptr, ws.bytes,
                                     s);
    });
    PyObject *o = result(out, mine);
    return with_lse ? results(o, THPVariable_Wrap(lse)) : o;
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- rotary positions
// (q, k, freqs, dims, style, grid, positions, start, magnitude, layout, out, inverse) ->
// (q_out, k_out)
PyObject *rotary(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a{args, n};
    const Tensor &q = tensor(a.next(), "q");
    PyObject *k_arg = a.next();
    const Tensor k = given(k_arg) ? tensor(k_arg, "k") : Tensor();
    const Tensor &freqs = tensor(a.next(), "freqs");
    PyObject *dims = a.next(), *style = a.next(), *grid = a.next(), *positions = a.next(),
             *start = a.next(), *magnitude = a.next();
    const bool bnhd = is_bnhd(a.next());
    PyObject *outs = a.next();
    monarch_rotary_desc desc = {};
    desc.inverse = flag(a.next());
    a.end();
    desc.half = is_word(style, "half");
    if (!desc.half && !is_word(style, "interleaved"))
        refuse("style must be one of ['interleaved', 'half']");
    if (q.dim() != 4 || (k.defined() && k.dim() != 4)) refuse("expected 4-D tensors");
    const int dev = index_of(q);
    desc.dtype = dtype_of(q);
    const int heads = bnhd ? 2 : 1, tokens = 3 - heads;
    desc.B = narrow(q.size(0), "batch");
    desc.H = narrow(q.size(heads), "heads");
    desc.N = narrow(q.size(tokens), "tokens");
    desc.d = narrow(q.size(3), "head dimension");
    if (k.defined()) {
        alike(q, k);
        if (k.size(0) != q.size(0) || k.size(tokens) != q.size(tokens) || k.size(3) != q.size(3))
            refuse("q and k must share batch, tokens and head dimension");
        desc.Hkv = narrow(k.size(heads), "heads");
    }
    if (freqs.scalar_type() != at::kDouble || freqs.dim() != 1 || !freqs.is_cuda() ||
        freqs.get_device() != dev || !freqs.is_contiguous())
        refuse("freqs must be a contiguous float64 vector on the inputs' device");
    desc.pairs = narrow(freqs.size(0), "frequencies");
    desc.axes = 1;
    desc.pairs_of_axis[0] = desc.pairs;
    if (given(dims)) {
        int32_t widths[3] = {0, 0, 0};
        desc.axes = integers(dims, 1, 3, widths, "dims");
        int64_t sum = 0;
        for (int i = 0; i < 3; i++) {
            if (widths[i] < 0 || widths[i] % 2) sum = -1;
            if (sum >= 0) sum += widths[i];
            desc.pairs_of_axis[i] = widths[i] / 2;
        }
        if (sum != 2 * (int64_t)desc.pairs)
            refuse("dims must be 1 to 3 even widths that sum to twice the frequencies");
    }
    if (given(grid)) {
        int32_t g[3];
        integers(grid, 3, 3, g, "grid");
        if (g[0] < 1 || g[1] < 1 || g[2] < 1 || (int64_t)g[1] * g[2] > INT32_MAX ||
            (int64_t)g[0] * g[1] * g[2] != desc.N)
            refuse("N = " + std::to_string(desc.N) + " is not frames * rows * columns of the grid");
        if (given(positions)) refuse("give grid or positions, not both");
        desc.grid_h = g[1];
        desc.grid_w = g[2];
    }
    if (given(positions)) {
        // [N] or [B, N], several axes last
        const Tensor &p = tensor(positions, "positions");
        const int rank = desc.axes > 1 ? 2 : 1, batch = (int)p.dim() - rank;
        if (p.scalar_type() != at::kInt || !p.is_cuda() || p.get_device() != dev ||
            (batch != 0 && batch != 1) || p.size(batch) != desc.N ||
            (rank == 2 && (p.size(batch + 1) != desc.axes || p.stride(batch + 1) != 1)) ||
            (batch == 1 && p.size(0) != 1 && p.size(0) != desc.B))
            refuse("positions must be int32 [N] or [B, N], with several axes a last dimension of "
                   "them, on the inputs' device");
        desc.positions = p.const_data_ptr<int32_t>();
        desc.pos_batch = batch == 1 && p.size(0) > 1 ? p.stride(0) : 0;
        desc.pos_token = desc.N > 1 ? p.stride(batch) : 0;
    }
    if (THPVariable_Check(start))
        desc.starts = index_pointer(start, "start", desc.B, dev);
    else
        desc.start = int32(start, "start");
    desc.magnitude = real(magnitude, "magnitude");

    PyObject *q_mine = Py_None, *k_mine = Py_None;
    if (given(outs)) {
        if ((!PyTuple_Check(outs) && !PyList_Check(outs)) || PySequence_Fast_GET_SIZE(outs) != 2)
            refuse("out must be (q_out, k_out)");
        q_mine = PySequence_Fast_GET_ITEM(outs, 0);
        k_mine = PySequence_Fast_GET_ITEM(outs, 1);
        if (given(k_mine) != k.defined())
            refuse("out must be (q_out, k_out), k_out None exactly when k is");
    }
    const Tensor qo = given(q_mine) ? tensor(q_mine, "q_out") : at::empty_like(q);
    const Tensor ko = !k.defined() ? Tensor() : given(k_mine) ? tensor(k_mine, "k_out") : at::empty_like(k);
    if (qo.sizes() != q.sizes() || (k.defined() && ko.sizes() != k.sizes()))
        refuse("outputs must have the inputs' shapes");
    alike(q, qo);
    desc.q = strides4(q, bnhd);
    desc.q_out = strides4(qo, bnhd);
    if (k.defined()) {
        alike(q, ko);
        desc.k = strides4(k, bnhd);
        desc.k_out = strides4(ko, bnhd);
    }
    const c10::cuda::CUDAGuard guard(on(dev));
    launch(dev, "monarch_rotary", [&](monarch_stream_t s) {
        return monarch_rotary(&desc, q.data_ptr(), k.defined() ? k.data_ptr() : nullptr,
                              (const double *)freqs.data_ptr(), qo.data_ptr(),
                              k.defined() ? ko.data_ptr() : nullptr, s);
    });
    return results(result(qo, q_mine), k.defined() ? result(ko, k_mine) : none());
    END_HANDLE_TH_ERRORS
}

// The exception class of refused calls.
PyObject *set_status_error(PyObject *, PyObject *cls) {
    Py_INCREF(cls);
    Py_XSETREF(g_status_error, cls);
    Py_RETURN_NONE;
}

#define ENTRY(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(window_attention),
                         ENTRY(window_attention_path),
                         ENTRY(window_attention_backward),
                         ENTRY(paged_attention),
                         ENTRY(rotary),
                         {"set_status_error", set_status_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "monarch_torch", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_monarch_torch() { return PyModule_Create(&module); }
