// tensors.cpp -- the calls of the attention operators, and of those around a
// block, with torch tensors: sizes, types, strides and devices are checked here
// and addresses handed to the C calls of ar.h.  Argument marshalling only.
//
// Read from Python, the attributes of a call's eight or more tensors took
// 12-20 us, several times what the kernels of a decode step run; here a call
// with nothing to launch takes 0.3 us, the C call's own checks among them.
//
// Every function takes its arguments by position, the stream last (None: the
// current stream of the tensors' device), and returns the C call's status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <exception>
#include <initializer_list>
#include <string>

#include "ar.h"

namespace {

struct PythonError {};  // the Python error is set

// torch's function of that name, looked up when the module is loaded: a static
// that is set at its first use waits for another thread's setting of it with the
// interpreter's lock held, which that thread may need.
PyObject *current_stream;

[[noreturn]] void fail(PyObject *type, const char *format, ...) {
    va_list args;
    va_start(args, format);
    PyErr_FormatV(type, format, args);
    va_end(args);
    throw PythonError();
}

using at::ScalarType;
constexpr int64_t kAny = -1;

const char *name_of(ScalarType t) {
    switch (t) {
        case ScalarType::BFloat16: return "torch.bfloat16, torch.int16 or torch.uint16";
        case ScalarType::Float: return "torch.float32";
        case ScalarType::Long: return "torch.int64";
        case ScalarType::Int: return "torch.int32";
        default: return "torch.uint8";
    }
}

// The arguments of one call: every tensor is checked as it is taken.
class Args {
  public:
    Args(PyObject *const *args, Py_ssize_t given, Py_ssize_t wanted) : args_(args), last_(wanted - 1) {
        if (given != wanted) fail(PyExc_TypeError, "%zd arguments expected, got %zd", wanted, given);
    }

    // A tensor of that type and shape (kAny: any size).
    const at::Tensor &tensor(const char *what, ScalarType type, std::initializer_list<int64_t> shape, bool contiguous = true) {
        return fitting(next(what), what, type, shape, contiguous);
    }

    const at::Tensor &fitting(const at::Tensor &t, const char *what, ScalarType type, std::initializer_list<int64_t> shape, bool contiguous) {
        const ScalarType have = t.scalar_type();
        const bool bf16 = type == ScalarType::BFloat16 && (have == ScalarType::Short || have == ScalarType::UInt16);
        if (have != type && !bf16) fail(PyExc_ValueError, "%s: %s expected, got %s", what, name_of(type), at::toString(have));
        bool fits = t.dim() == (int64_t)shape.size();
        for (int64_t d = 0; fits && d < t.dim(); ++d)
            fits = shape.begin()[d] == kAny || shape.begin()[d] == t.size(d);
        if (!fits) {
            const std::string want = text(shape.begin(), shape.size()), got = text(t.sizes().data(), t.dim());
            fail(PyExc_ValueError, "%s: shape (%s) expected, got (%s)", what, want.c_str(), got.c_str());
        }
        if (contiguous && !t.is_contiguous()) fail(PyExc_ValueError, "%s: the tensor must be contiguous", what);
        return t;
    }

    // (tokens, heads, channels) of bf16 with contiguous channels.
    const at::Tensor &rows(const char *what, int64_t tokens, int64_t heads, int64_t dim) {
        const at::Tensor &t = tensor(what, ScalarType::BFloat16, {tokens, heads, dim}, false);
        if (t.size(2) > 1 && t.stride(2) != 1) fail(PyExc_ValueError, "%s: channels must be contiguous", what);
        return t;
    }

    // Whether the next argument is None, which is taken then.
    bool none() { return args_[at_] == Py_None ? (++at_, true) : false; }

    // (tokens, channels) of bf16 with contiguous channels.
    ar_rows plane(const char *what, int64_t tokens, int64_t dim) { return as_plane(fitting(next(what), what, ScalarType::BFloat16, {tokens, dim}, false), what); }

    // (dim) for all tokens, or (tokens, dim).
    ar_rows gate(const char *what, int64_t tokens, int64_t dim) {
        const at::Tensor &t = next(what);
        if (t.dim() == 1) return ar_rows{fitting(t, what, ScalarType::BFloat16, {dim}, true).data_ptr(), 0, 0};
        ar_rows r = as_plane(fitting(t, what, ScalarType::BFloat16, {tokens, dim}, false), what);
        if (tokens <= 1) r.token_stride = dim;
        else if (r.token_stride == 0)
            fail(PyExc_ValueError, "%s: one gate for all tokens is a tensor of shape (%lld)", what, (long long)dim);
        return r;
    }

    // One tensor (tokens, dim), or a sequence of up to AR_MAX_P of them with one stride.
    int planes(const char *what, int64_t tokens, int64_t dim, ar_ptrs *to, int64_t *stride) {
        PyObject *o = args_[at_];
        if (THPVariable_Check(o)) {
            const ar_rows r = plane(what, tokens, dim);
            to->p[0] = r.p, *stride = r.token_stride;
            return 1;
        }
        ++at_;
        if (!PyList_Check(o) && !PyTuple_Check(o))
            fail(PyExc_TypeError, "%s: expected CUDA tensors, got %s", what, Py_TYPE(o)->tp_name);
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(o);
        if (n < 1 || n > AR_MAX_P) fail(PyExc_ValueError, "%s: 1 to %d tensors expected, got %zd", what, AR_MAX_P, n);
        for (Py_ssize_t i = 0; i < n; ++i) {
            const ar_rows r = as_plane(fitting(take(PySequence_Fast_GET_ITEM(o, i), what), what, ScalarType::BFloat16, {tokens, dim}, false), what);
            if (i == 0) *stride = r.token_stride;
            else if (tokens > 1 && r.token_stride != *stride) fail(PyExc_ValueError, "%s: tensors of one stride expected", what);
            to->p[i] = r.p;
        }
        return (int)n;
    }

    // At least so many bytes, of any type.
    const at::Tensor &bytes(const char *what, int64_t least) {
        const at::Tensor &t = next(what);
        const int64_t have = t.numel() * (int64_t)t.element_size();
        if (!t.is_contiguous()) fail(PyExc_ValueError, "%s: the tensor must be contiguous", what);
        if (have < least)
            fail(PyExc_ValueError, "%s: %lld bytes, the call touches %lld", what, (long long)have, (long long)least);
        return t;
    }

    // The argument so many places on, a tensor of that many dimensions; it is not taken.
    const at::Tensor &peek(int on, const char *what, int64_t dims) {
        const at::Tensor &t = take(args_[at_ + on], what);
        if (t.dim() != dims) fail(PyExc_ValueError, "%s: %lld dimensions expected, got %lld", what, (long long)dims, (long long)t.dim());
        return t;
    }

    int64_t integer() {
        const long long v = PyLong_AsLongLong(args_[at_++]);
        if (v == -1 && PyErr_Occurred()) throw PythonError();
        return v;
    }

    // An integer that a C int argument takes.
    int small() {
        const int64_t v = integer();
        if (v != (int)v) fail(PyExc_OverflowError, "%lld does not fit an int", (long long)v);
        return (int)v;
    }

    double number() {
        const double v = PyFloat_AsDouble(args_[at_++]);
        if (v == -1.0 && PyErr_Occurred()) throw PythonError();
        return v;
    }

    double number_or(double otherwise) { return args_[at_] == Py_None ? (++at_, otherwise) : number(); }

    // The stream, the last argument, and the check that it and all tensors are
    // on one GPU, which is the current one until this object goes: kernels are
    // launched on the current device, whatever their stream.
    void *stream() {
        if (!device_.is_cuda()) fail(PyExc_TypeError, "expected CUDA tensors, got tensors on %s", device_.str().c_str());
        guard_.reset_device(device_);
        PyObject *s = args_[last_], *owned = nullptr;
        if (s == Py_None) {
            PyObject *index = PyLong_FromLong(device_.index());
            s = owned = index ? PyObject_CallOneArg(current_stream, index) : nullptr;
            Py_XDECREF(index);
        } else if (!PyLong_Check(s)) {
            PyObject *index = PyObject_GetAttrString(s, "device_index");
            const long at = index ? PyLong_AsLong(index) : -1;
            Py_XDECREF(index);
            if (at == -1 && PyErr_Occurred()) throw PythonError();
            if (at != device_.index()) fail(PyExc_ValueError, "stream: on cuda:%ld, tensors on %s", at, device_.str().c_str());
            s = owned = PyObject_GetAttrString(s, "cuda_stream");
        }
        if (!s) throw PythonError();
        void *p = PyLong_AsVoidPtr(s);
        Py_XDECREF(owned);
        if (!p && PyErr_Occurred()) throw PythonError();
        return p;
    }

  private:
    static ar_rows as_plane(const at::Tensor &t, const char *what) {
        if (t.size(1) > 1 && t.stride(1) != 1) fail(PyExc_ValueError, "%s: channels must be contiguous", what);
        return ar_rows{t.numel() ? t.data_ptr() : nullptr, t.stride(0), 0};
    }

    const at::Tensor &next(const char *what) { return take(args_[at_++], what); }

    const at::Tensor &take(PyObject *o, const char *what) {
        if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s: expected a CUDA tensor, got %s", what, Py_TYPE(o)->tp_name);
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!seen_) device_ = t.device(), seen_ = true;
        else if (t.device() != device_)
            fail(PyExc_ValueError, "%s: on %s, others on %s", what, t.device().str().c_str(), device_.str().c_str());
        // nothing is recorded for autograd, and nothing is lost without a word
        if (t.requires_grad() && c10::GradMode::is_enabled())
            fail(PyExc_ValueError, "%s: requires a gradient, which this call does not record: call it under torch.no_grad()", what);
        return t;
    }

    static std::string text(const int64_t *n, size_t count) {
        std::string s;
        for (size_t i = 0; i < count; ++i) s += (i ? ", " : "") + (n[i] == kAny ? std::string("any") : std::to_string(n[i]));
        return s;
    }

    PyObject *const *args_;
    Py_ssize_t last_;
    int at_ = 0;
    bool seen_ = false;
    at::Device device_{at::kCPU};
    c10::OptionalDeviceGuard guard_;
};

ar_rows as_rows(const at::Tensor &t) {
    return ar_rows{t.numel() ? t.data_ptr() : nullptr, t.stride(0), t.stride(1)};
}

// Sizes that the C calls take as int: what does not fit is beyond their
// limits, and refused there.
int as_int(int64_t v) { return v > 0x7FFFFFFF ? 0x7FFFFFFF : (int)v; }

// What both directions of the head norms take after the gradients.
struct NormArgs {
    ar_rows q, k;
    void *qw, *kw, *cs, *pos;
    int64_t tokens, heads, kv_heads, dim, rotated, table;

    explicit NormArgs(Args &a) {
        const at::Tensor &tq = a.rows("q", kAny, kAny, kAny);
        tokens = tq.size(0), heads = tq.size(1), dim = tq.size(2);
        const at::Tensor &tk = a.rows("k", tokens, kAny, dim);
        kv_heads = tk.size(1);
        q = as_rows(tq), k = as_rows(tk);
        qw = a.tensor("q_weight", ScalarType::BFloat16, {dim}).data_ptr();
        kw = a.tensor("k_weight", ScalarType::BFloat16, {dim}).data_ptr();
        const at::Tensor &tc = a.tensor("cos_sin", ScalarType::Float, {kAny, kAny});
        cs = tc.data_ptr(), table = tc.size(0), rotated = tc.size(1);
        pos = a.tensor("positions", ScalarType::Long, {tokens}).data_ptr();
    }
};

int qk_norm_rope(Args &a) {
    const NormArgs n(a);
    const ar_rows qo = as_rows(a.rows("q_out", n.tokens, n.heads, n.dim));
    const ar_rows ko = as_rows(a.rows("k_out", n.tokens, n.kv_heads, n.dim));
    const float eps = (float)a.number();
    const int interleaved = a.small();
    return ar_qk_norm_rope(n.q, n.k, n.qw, n.kw, n.cs, n.pos, qo, ko, n.tokens, as_int(n.heads), as_int(n.kv_heads), as_int(n.dim),
                           as_int(n.rotated), n.table, eps, interleaved, a.stream());
}

int qk_norm_rope_bwd(Args &a) {
    const NormArgs n(a);
    const ar_rows gq = as_rows(a.rows("q_grad", n.tokens, n.heads, n.dim));
    const ar_rows gk = as_rows(a.rows("k_grad", n.tokens, n.kv_heads, n.dim));
    const ar_rows dq = as_rows(a.rows("dq", n.tokens, n.heads, n.dim));
    const ar_rows dk = as_rows(a.rows("dk", n.tokens, n.kv_heads, n.dim));
    void *dqw = a.tensor("dq_weight", ScalarType::Float, {n.dim}).data_ptr();
    void *dkw = a.tensor("dk_weight", ScalarType::Float, {n.dim}).data_ptr();
    const int64_t least = ar_qk_norm_rope_bwd_workspace(n.tokens, as_int(n.heads), as_int(n.kv_heads), as_int(n.dim));
    if (least < 0) return (int)least;
    void *ws = a.bytes("workspace", least).data_ptr();
    const float eps = (float)a.number();
    const int interleaved = a.small();
    return ar_qk_norm_rope_bwd(gq, gk, n.q, n.k, n.qw, n.kw, n.cs, n.pos, dq, dk, dqw, dkw, ws, n.tokens, as_int(n.heads),
                               as_int(n.kv_heads), as_int(n.dim), as_int(n.rotated), n.table, eps, interleaved, a.stream());
}

// k, v, slots, cache, page_size.
template <bool READ>
int kv4(Args &a) {
    const at::Tensor &k = a.rows(READ ? "k_out" : "k", kAny, kAny, kAny);
    const int64_t tokens = k.size(0), heads = k.size(1), dim = k.size(2);
    const ar_rows v = as_rows(a.rows(READ ? "v_out" : "v", tokens, heads, dim));
    void *slots = a.tensor("slots", ScalarType::Long, {tokens}).data_ptr();
    const at::Tensor &cache = a.tensor("cache", ScalarType::Byte, {kAny, heads, kAny, 34 * dim});
    const int page = a.small();
    if (cache.size(2) != page / 32)
        fail(PyExc_ValueError, "cache: shape (any, heads, page_size / 32, 34 dim) expected, got %lld tiles in a page of %d",
             (long long)cache.size(2), page);
    if (READ)
        return ar_kv4_read(cache.data_ptr(), slots, as_rows(k), v, tokens, as_int(heads), as_int(dim), cache.size(0), page, a.stream());
    return ar_kv4_write(as_rows(k), v, slots, cache.data_ptr(), tokens, as_int(heads), as_int(dim), cache.size(0), page, a.stream());
}

// q, out, lse, cache, page_table, q_start, kv_len, workspace, page_size,
// kv_heads, max_q, max_kv, window, scale (None: 1 / sqrt(dim)).
int kv4_attention(Args &a) {
    const at::Tensor &q = a.rows("q", kAny, kAny, kAny);
    const int64_t tokens = q.size(0), heads = q.size(1), dim = q.size(2);
    const ar_rows out = as_rows(a.rows("out", tokens, heads, dim));
    void *lse = a.tensor("lse", ScalarType::Float, {tokens, heads}).data_ptr();
    const at::Tensor &cache = a.tensor("cache", ScalarType::Byte, {kAny, kAny, kAny, 34 * dim});
    const at::Tensor &table = a.tensor("page_table", ScalarType::Int, {kAny, kAny}, false);
    const int64_t batch = table.size(0), per = table.size(1);
    if (per > 1 && table.stride(1) != 1) fail(PyExc_ValueError, "page_table: a sequence's entries must be contiguous");
    void *start = a.tensor("q_start", ScalarType::Int, {batch + 1}).data_ptr();
    void *len = a.tensor("kv_len", ScalarType::Int, {batch}).data_ptr();
    const at::Tensor &ws = a.bytes("workspace", 0);
    const int page = a.small(), kv_heads = a.small();
    const int64_t max_q = a.integer(), max_kv = a.integer(), window = a.integer();
    const float scale = (float)a.number_or(1.0 / std::sqrt((double)dim));
    if (cache.size(1) != kv_heads || cache.size(2) != page / 32)
        fail(PyExc_ValueError, "cache: shape (any, kv_heads, page_size / 32, 34 dim) expected, got %lld heads and %lld tiles in a page",
             (long long)cache.size(1), (long long)cache.size(2));
    const int64_t least = ar_kv4_attention_workspace(batch, tokens, max_q, max_kv, as_int(heads), kv_heads, as_int(dim));
    if (least < 0) return (int)least;
    if (ws.numel() * (int64_t)ws.element_size() < least)
        fail(PyExc_ValueError, "workspace: %lld bytes, the call touches %lld", (long long)(ws.numel() * ws.element_size()), (long long)least);
    return ar_kv4_attention(as_rows(q), cache.data_ptr(), table.data_ptr(), table.stride(0), start, len, out, lse, ws.data_ptr(), tokens,
                            batch, as_int(heads), kv_heads, as_int(dim), cache.size(0), page, per, max_q, max_kv, window, scale, a.stream());
}

// parts, x, h, z, post_weight, gate, pre_weight, residual_scale, eps.
int block_norm(Args &a) {
    const at::Tensor &like = a.peek(1, "x", 2);
    const int64_t tokens = like.size(0), dim = like.size(1);
    ar_ptrs parts = {};
    int64_t stride = 0;
    const int count = a.planes("parts", tokens, dim, &parts, &stride);
    const ar_rows x = a.plane("x", tokens, dim), h = a.plane("h", tokens, dim);
    const bool has_z = !a.none();
    const ar_rows z = has_z ? a.plane("z", tokens, dim) : ar_rows{};
    void *post = a.none() ? nullptr : a.tensor("post_weight", ScalarType::BFloat16, {dim}).data_ptr();
    const ar_rows gate = a.none() ? ar_rows{} : a.gate("gate", tokens, dim);
    void *pre = a.none() ? nullptr : a.tensor("pre_weight", ScalarType::BFloat16, {dim}).data_ptr();
    if (has_z != (pre != nullptr)) fail(PyExc_ValueError, "z and pre_weight are given together or not at all");
    const float scale = (float)a.number(), eps = (float)a.number();
    return ar_block_norm(parts, stride, count, x, post, gate, pre, h, z, tokens, as_int(dim), scale, eps, a.stream());
}

// h_grad, z_grad, y, x, dx, dy, workspace, post_weight, gate, pre_weight,
// gate_grad, post_grad, pre_grad, residual_scale, eps.
int block_norm_bwd(Args &a) {
    const at::Tensor &like = a.peek(3, "x", 2);
    const int64_t tokens = like.size(0), dim = like.size(1);
    const ar_rows dh = a.none() ? ar_rows{} : a.plane("h_grad", tokens, dim);
    const bool has_dz = !a.none();
    const ar_rows dz = has_dz ? a.plane("z_grad", tokens, dim) : ar_rows{};
    const ar_rows y = a.plane("y", tokens, dim), x = a.plane("x", tokens, dim);
    const ar_rows dx = a.plane("dx", tokens, dim), dy = a.plane("dy", tokens, dim);
    const int64_t least = ar_block_norm_bwd_workspace(tokens, as_int(dim));
    if (least < 0) return (int)least;
    void *ws = a.bytes("workspace", least).data_ptr();
    void *post = a.none() ? nullptr : a.tensor("post_weight", ScalarType::BFloat16, {dim}).data_ptr();
    const bool has_gate = !a.none();  // the address of a gate of no tokens is null, too
    const ar_rows gate = has_gate ? a.gate("gate", tokens, dim) : ar_rows{};
    void *pre = a.none() ? nullptr : a.tensor("pre_weight", ScalarType::BFloat16, {dim}).data_ptr();
    if (has_dz != (pre != nullptr)) fail(PyExc_ValueError, "z_grad and pre_weight are given together or not at all");
    ar_rows dgate = {};
    if (!a.none()) {
        if (!has_gate) fail(PyExc_ValueError, "gate_grad: there is no gate");
        if (gate.token_stride) dgate = a.plane("gate_grad", tokens, dim);
        else dgate.p = a.tensor("gate_grad", ScalarType::Float, {dim}).data_ptr();
    }
    void *dpost = a.none() ? nullptr : a.tensor("post_grad", ScalarType::Float, {dim}).data_ptr();
    void *dpre = a.none() ? nullptr : a.tensor("pre_grad", ScalarType::Float, {dim}).data_ptr();
    if (dpost && !post) fail(PyExc_ValueError, "post_grad: there is no post_weight");
    if (dpre && !pre) fail(PyExc_ValueError, "pre_grad: there is no pre_weight");
    const float scale = (float)a.number(), eps = (float)a.number();
    return ar_block_norm_bwd(dh, dz, y, x, post, gate, pre, dx, dy, dgate, dpost, dpre, ws, tokens, as_int(dim), scale, eps, a.stream());
}

// Tiles and bytes of a packed matrix (n_out, n_in); 0 where the C call refuses it.
struct Packed {
    int64_t tiles, bytes;
    Packed(int64_t n_out, int64_t n_in) {
        const int64_t one = ar_w4_bytes(1, n_in);
        bytes = one < 0 ? 0 : one;
        tiles = (n_out + 15) / 16;
    }
};

// w, packed.
template <bool BACK>
int w4_pack(Args &a) {
    const at::Tensor &w = a.peek(0, "w", 2);
    const int64_t n_out = w.size(0), n_in = w.size(1);
    const ar_rows r = a.plane("w", n_out, n_in);
    const Packed size(n_out, n_in);
    if (!size.bytes) return AR_EINVAL;
    void *packed = a.tensor("packed", ScalarType::Byte, {size.tiles, size.bytes}).data_ptr();
    if (BACK) return ar_w4_unpack(packed, r.p, r.token_stride, n_out, n_in, a.stream());
    return ar_w4_pack(r.p, r.token_stride, packed, n_out, n_in, a.stream());
}

// x, packed, out.
int w4_linear(Args &a) {
    const at::Tensor &x = a.peek(0, "x", 2), &out = a.peek(2, "out", 2);
    const int64_t tokens = x.size(0), n_in = x.size(1), n_out = out.size(1);
    const ar_rows rx = a.plane("x", tokens, n_in);
    const Packed size(n_out, n_in);
    if (!size.bytes) return AR_EINVAL;
    void *packed = a.tensor("packed", ScalarType::Byte, {size.tiles, size.bytes}).data_ptr();
    const ar_rows ro = a.plane("out", tokens, n_out);
    return ar_w4_linear(rx, packed, ro, tokens, n_out, n_in, a.stream());
}

// x, router, gate_up, down, out, choice, weight, workspace, scale.
int w4_experts(Args &a) {
    const at::Tensor &tx = a.peek(0, "x", 2), &tr = a.peek(1, "router", 2), &tg = a.peek(2, "gate_up", 3), &tc = a.peek(5, "choice", 2);
    const int64_t tokens = tx.size(0), hidden = tx.size(1), experts = tr.size(0), inner = 8 * tg.size(1), top_k = tc.size(1);
    const ar_rows x = a.plane("x", tokens, hidden);
    void *router = a.tensor("router", ScalarType::BFloat16, {experts, hidden}).data_ptr();
    const Packed up(2 * inner, hidden), down(hidden, inner);
    const int64_t least = ar_w4_experts_workspace(tokens, hidden, inner, as_int(experts), as_int(top_k));
    if (!up.bytes || !down.bytes || least < 0) return AR_EINVAL;
    void *pu = a.tensor("gate_up", ScalarType::Byte, {experts, up.tiles, up.bytes}).data_ptr();
    void *pd = a.tensor("down", ScalarType::Byte, {experts, down.tiles, down.bytes}).data_ptr();
    const ar_rows out = a.plane("out", tokens, hidden);
    void *choice = a.tensor("choice", ScalarType::Int, {tokens, top_k}).data_ptr();
    void *weight = a.tensor("weight", ScalarType::Float, {tokens, top_k}).data_ptr();
    void *ws = a.bytes("workspace", least).data_ptr();
    const float scale = (float)a.number();
    return ar_w4_experts(x, router, pu, pd, out, choice, weight, ws, tokens, hidden, inner, as_int(experts), as_int(top_k), scale, a.stream());
}

template <int (*CALL)(Args &), int COUNT>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t given) {
    try {
        Args a(args, given, COUNT);
        return PyLong_FromLong(CALL(a));
    } catch (const PythonError &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

template <int (*CALL)(Args &), int COUNT>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<CALL, COUNT>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<qk_norm_rope, 11>("qk_norm_rope"),
    method<qk_norm_rope_bwd, 16>("qk_norm_rope_bwd"),
    method<kv4<false>, 6>("kv4_write"),
    method<kv4<true>, 6>("kv4_read"),
    method<kv4_attention, 15>("kv4_attention"),
    method<block_norm, 10>("block_norm"),
    method<block_norm_bwd, 16>("block_norm_bwd"),
    method<w4_pack<false>, 3>("w4_pack"),
    method<w4_pack<true>, 3>("w4_unpack"),
    method<w4_linear, 4>("w4_linear"),
    method<w4_experts, 10>("w4_experts"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "ar_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit_ar_tensors(void) {
    PyObject *torch = PyImport_ImportModule("torch._C");
    current_stream = torch ? PyObject_GetAttrString(torch, "_cuda_getCurrentRawStream") : nullptr;
    Py_XDECREF(torch);
    return current_stream ? PyModule_Create(&module) : nullptr;
}
