// bind.cpp -- the block operators' way from PyTorch tensors to the C ABI
// (include/moe.h): one call checks every tensor's type, shape, device and
// pitch, fills in the argument structures and calls the library.
//
// Why not in Python: a norm of one token takes 4 us on the device, and looking
// at its 11 tensors from Python took longer than that (11.4 us a call, now 6.6;
// a router's call of 128 tokens 4.8, now 2.8).
//
// Functions take the library function's address, the config's, the operator's
// device index (-1: CPU) and the stream's handle, then tensors (None where
// absent), and return the library's code.  They keep nothing between calls.
#include <Python.h>
#include <c10/core/GradMode.h>
#include <c10/core/impl/DeviceGuardImplInterface.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <algorithm>
#include <limits>
#include <sstream>

#include "moe.h"

namespace {

struct PythonError {};   // the interpreter's error is set

[[noreturn]] void fail(PyObject *type, const std::string &what) {
    PyErr_SetString(type, what.c_str());
    throw PythonError{};
}

int64_t number(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
}
template <class P>
P address(PyObject *o) {
    if (o == Py_None) return nullptr;
    void *v = PyLong_AsVoidPtr(o);
    if (!v && PyErr_Occurred()) throw PythonError{};
    return reinterpret_cast<P>(v);
}

at::ScalarType type_of(int dtype) { return dtype == MOE_DTYPE_F32 ? at::kFloat : at::kBFloat16; }

// Arguments of one call, taken in order, with the device its tensors must be on.
struct Args {
    PyObject *const *at, *const *end;
    int index = -1;
    bool grad = false;   // an input requires a gradient

    Args(PyObject *const *args, Py_ssize_t n) : at(args), end(args + n) {}
    PyObject *next() {
        if (at == end) fail(PyExc_TypeError, "too few arguments");
        return *at++;
    }
    void done() const {
        if (at != end) fail(PyExc_TypeError, "too many arguments");
    }
    // The next tensor, or nullptr for None.
    const at::Tensor *tensor(const char *name) {
        PyObject *o = next();
        if (o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) fail(PyExc_TypeError, std::string(name) + " must be a tensor");
        return &THPVariable_Unpack(o);
    }
    [[noreturn]] void refuse(const at::Tensor &t, const char *name, at::ScalarType dt, int64_t rows, int64_t cols, const char *what) {
        std::ostringstream s;
        s << name << " must be a " << dt << " tensor of shape [";
        if (rows >= 0) s << rows << ", ";
        s << cols << "] " << what << ", got " << t.scalar_type() << " " << t.sizes() << " with strides " << t.strides() << " on "
          << t.device();
        fail(PyExc_ValueError, s.str());
    }
    void check(const at::Tensor &t, const char *name, at::ScalarType dt, int64_t rows, int64_t cols) {
        const bool shape = rows < 0 ? t.dim() == 1 && t.size(0) == cols : t.dim() == 2 && t.size(0) == rows && t.size(1) == cols;
        if (!shape || t.scalar_type() != dt || t.get_device() != index) refuse(t, name, dt, rows, cols, "on the operator's device");
    }
    void *pointer(const at::Tensor &t, bool out) {
        grad |= !out && t.requires_grad();
        return out ? t.mutable_data_ptr() : const_cast<void *>(t.const_data_ptr());
    }
    // Called by the forward passes, whose outputs know nothing of their inputs' graph.
    void tell_of_graph(const char *what) const {
        if (!grad || !c10::GradMode::is_enabled()) return;
        const std::string s = std::string(what) + " got an input that requires a gradient, but takes no part in autograd: its outputs "
                              "are cut from the graph. Call it under torch.no_grad(), and the operator's backward() for gradients.";
        if (PyErr_WarnEx(PyExc_UserWarning, s.c_str(), 1) < 0) throw PythonError{};
    }

    // A [rows, cols] tensor whose rows are contiguous.
    template <class P>
    void rows(const at::Tensor *t, const char *name, at::ScalarType dt, int64_t rows, int64_t cols, P *&ptr, int64_t &ld, bool out) {
        ptr = nullptr, ld = 0;
        if (!t) return;
        check(*t, name, dt, rows, cols);
        ld = cols;
        if (!t->is_contiguous()) {
            if ((t->stride(1) != 1 && cols > 1) || (rows > 1 && t->stride(0) < cols))
                refuse(*t, name, dt, rows, cols, "with contiguous rows that do not overlap");
            if (rows > 1) ld = t->stride(0);
        }
        ptr = static_cast<P *>(pointer(*t, out));
    }
    // A contiguous tensor; rows < 0: of one dimension.
    template <class P>
    void flat(const at::Tensor *t, const char *name, at::ScalarType dt, int64_t rows, int64_t cols, P *&ptr, bool out) {
        ptr = nullptr;
        if (!t) return;
        check(*t, name, dt, rows, cols);
        if (!t->is_contiguous()) refuse(*t, name, dt, rows, cols, "contiguous");
        ptr = static_cast<P *>(pointer(*t, out));
    }
};

// An output that the call needs.
const at::Tensor *needed(const at::Tensor *t, const char *name) {
    if (!t) fail(PyExc_ValueError, std::string("out lacks ") + name);
    return t;
}

int tokens(const at::Tensor *t, const char *name) {
    if (!t) fail(PyExc_ValueError, std::string(name) + " is missing");
    if (t->dim() != 2 || t->size(0) > std::numeric_limits<int>::max())
        fail(PyExc_ValueError, std::string(name) + " must have two dimensions, at most 2^31 - 1 rows");
    return (int)t->size(0);
}

// Library calls run without the interpreter's lock, and on a GPU's tensors alone.
template <class F>
int unlocked(const Args &a, F f) {
    if (a.index < 0) fail(PyExc_RuntimeError, "the operator was made for the CPU: it only checks its arguments");
    PyThreadState *state = PyEval_SaveThread();
    const int rc = f();
    PyEval_RestoreThread(state);
    return rc;
}

// No C++ exception passes into the interpreter.
template <int (*F)(Args &)>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    try {
        Args a(args, n);
        return PyLong_FromLong(F(a));
    } catch (const PythonError &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// fn, cfg, index, stream
template <class Fn, class Cfg>
struct Head {
    Fn fn;
    const Cfg *cfg;
    void *stream;
    explicit Head(Args &a) {
        fn = address<Fn>(a.next());
        cfg = address<const Cfg *>(a.next());
        a.index = (int)number(a.next());
        stream = address<void *>(a.next());
        if (!fn || !cfg) fail(PyExc_TypeError, "no function or config");
        // The library launches on the current device, and every device's default stream has the handle 0.
        if (a.index < 0) return;
        const int now = c10::impl::getDeviceGuardImpl(c10::DeviceType::CUDA)->getDevice().index();
        if (now == a.index) return;
        std::ostringstream s;
        s << "the operator is on cuda:" << a.index << " and the current device is cuda:" << now << ": call it under torch.cuda.device("
          << a.index << ")";
        fail(PyExc_RuntimeError, s.str());
    }
};

// ..., residual, y, w_post, gate, w_pre, h, n, codes, sf, rstd_post, rstd_pre
int norm_forward(Args &a) {
    const Head<decltype(&moe_norm_forward), moe_norm_config> c(a);
    const int64_t H = c.cfg->hidden;
    const at::ScalarType s = type_of(c.cfg->stream_dtype), w = type_of(c.cfg->param_dtype);
    moe_norm_io io{};
    const at::Tensor *residual = a.tensor("residual"), *y = a.tensor("y"), *w_post = a.tensor("w_post"), *gate = a.tensor("gate"),
                     *w_pre = a.tensor("w_pre"), *h = a.tensor("h"), *n = a.tensor("n"), *codes = a.tensor("codes"),
                     *sf = a.tensor("sf"), *rstd_post = a.tensor("rstd_post"), *rstd_pre = a.tensor("rstd_pre");
    a.done();
    const int T = tokens(residual, "residual");
    const bool channel = c.cfg->gate == MOE_GATE_CHANNEL, quant = w_pre && c.cfg->quant != MOE_QUANT_NONE;
    a.rows(residual, "residual", s, T, H, io.residual, io.ld_residual, false);
    a.rows(y, "y", s, T, H, io.y, io.ld_y, false);
    a.flat(w_post, "w_post", w, -1, H, io.w_post, false);
    a.flat(gate, "gate", w, -1, channel ? H : T, io.gate, false);
    a.flat(w_pre, "w_pre", w, -1, H, io.w_pre, false);
    if (y) a.rows(needed(h, "h"), "h", s, T, H, io.h, io.ld_h, true);
    if (w_pre) a.rows(quant ? n : needed(n, "n"), "n", s, T, H, io.n, io.ld_n, true);
    if (quant) {
        const bool f32 = c.cfg->quant == MOE_QUANT_FP8_128;
        a.flat(needed(codes, "codes"), "codes", at::kByte, T, H, io.codes, true);
        a.flat(needed(sf, "sf"), "sf", f32 ? at::kFloat : at::kByte, T, H / (f32 ? 128 : 32), io.sf, true);
    }
    if (y && w_post) a.flat(rstd_post, "rstd_post", at::kFloat, -1, T, io.rstd_post, true);
    if (w_pre) a.flat(rstd_pre, "rstd_pre", at::kFloat, -1, T, io.rstd_pre, true);
    a.tell_of_graph("BlockNorm.forward");
    return unlocked(a, [&] { return c.fn(c.cfg, T, &io, c.stream); });
}

// ..., h, dh, dn, y, w_post, gate, w_pre, rstd_post, rstd_pre, dresidual, dy, dw_post, dgate, dw_pre, workspace, address of its
// size's function
int norm_backward(Args &a) {
    const Head<decltype(&moe_norm_backward), moe_norm_config> c(a);
    const int64_t H = c.cfg->hidden;
    const at::ScalarType s = type_of(c.cfg->stream_dtype), w = type_of(c.cfg->param_dtype);
    moe_norm_grad_io io{};
    const at::Tensor *h = a.tensor("h"), *dh = a.tensor("dh"), *dn = a.tensor("dn"), *y = a.tensor("y"), *w_post = a.tensor("w_post"),
                     *gate = a.tensor("gate"), *w_pre = a.tensor("w_pre"), *rstd_post = a.tensor("rstd_post"),
                     *rstd_pre = a.tensor("rstd_pre"), *dresidual = a.tensor("dresidual"), *dy = a.tensor("dy"),
                     *dw_post = a.tensor("dw_post"), *dgate = a.tensor("dgate"), *dw_pre = a.tensor("dw_pre");
    const at::Tensor *work = needed(a.tensor("workspace"), "workspace");
    const auto ws_bytes = address<decltype(&moe_norm_workspace_bytes)>(a.next());
    a.done();
    const int T = tokens(h, "h");
    void *ws;
    a.flat(work, "workspace", at::kByte, -1, std::max<int64_t>(work->numel(), (int64_t)ws_bytes(c.cfg, T)), ws, true);
    const int64_t gates = c.cfg->gate == MOE_GATE_CHANNEL ? H : T;
    a.rows(h, "h", s, T, H, io.h, io.ld_h, false);
    a.rows(dh, "dh", s, T, H, io.dh, io.ld_dh, false);
    a.rows(dn, "dn", s, T, H, io.dn, io.ld_dn, false);
    a.rows(y, "y", s, T, H, io.y, io.ld_y, false);
    a.flat(w_post, "w_post", w, -1, H, io.w_post, false);
    a.flat(gate, "gate", w, -1, gates, io.gate, false);
    a.flat(w_pre, "w_pre", w, -1, H, io.w_pre, false);
    if (w_post) a.flat(rstd_post, "rstd_post", at::kFloat, -1, T, io.rstd_post, false);
    if (w_pre) a.flat(rstd_pre, "rstd_pre", at::kFloat, -1, T, io.rstd_pre, false);
    a.rows(needed(dresidual, "dresidual"), "dresidual", s, T, H, io.dresidual, io.ld_dresidual, true);
    if (y) a.rows(needed(dy, "dy"), "dy", s, T, H, io.dy, io.ld_dy, true);
    if (w_post) a.flat(needed(dw_post, "dw_post"), "dw_post", at::kFloat, -1, H, io.dw_post, true);
    if (gate) a.flat(needed(dgate, "dgate"), "dgate", at::kFloat, -1, gates, io.dgate, true);
    if (w_pre) a.flat(needed(dw_pre, "dw_pre"), "dw_pre", at::kFloat, -1, H, io.dw_pre, true);
    return unlocked(a, [&] { return c.fn(c.cfg, T, &io, ws, c.stream); });
}

// seq_offsets, loss, counts, prob_mean, tokens, and (max_tokens, max_seqs, workspace address) that `T` tokens must fit
void losses(Args &a, int T, int E, bool write, moe_balance_io &io, void *&ws) {
    const at::Tensor *off = a.tensor("seq_offsets"), *loss = a.tensor("loss"), *counts = a.tensor("counts"),
                     *mean = a.tensor("prob_mean"), *tok = a.tensor("tokens");
    const int64_t max_tokens = number(a.next()), max_seqs = number(a.next());
    ws = address<void *>(a.next());
    if (off && (off->dim() != 1 || off->size(0) < 1 || off->size(0) > MOE_MAX_SEQS + 1))
        fail(PyExc_ValueError, "seq_offsets must be an int32 tensor of shape [sequences + 1]");
    const int64_t S = off ? off->size(0) - 1 : 1;
    if (write && (T > max_tokens || S > max_seqs)) {
        std::ostringstream s;
        s << T << " tokens in " << S << " sequences: the router was made for losses of " << max_tokens << " tokens in " << max_seqs;
        fail(PyExc_ValueError, s.str());
    }
    io.num_seqs = (int)S;
    a.flat(off, "seq_offsets", at::kInt, -1, S + 1, io.seq_offsets, false);
    a.flat(needed(loss, "loss"), "loss", at::kFloat, -1, 3, io.loss, write);
    a.flat(needed(counts, "counts"), "counts", at::kInt, S, E, io.counts, write);
    a.flat(needed(mean, "prob_mean"), "prob_mean", at::kFloat, S, E, io.prob_mean, write);
    a.flat(needed(tok, "tokens"), "tokens", at::kInt, -1, S + 2, io.seq_tokens, write);
}

// ..., logits, bias, topk_idx, topk_weights[, losses]
int router_forward(Args &a) {
    const Head<decltype(&moe_router_forward), moe_router_config> c(a);
    const int E = c.cfg->num_experts, k = c.cfg->topk;
    const at::Tensor *logits = a.tensor("logits"), *bias = a.tensor("bias"), *idx = a.tensor("topk_idx"),
                     *weights = a.tensor("topk_weights");
    const int T = tokens(logits, "logits");
    const void *l;
    const float *b;
    int32_t *i;
    float *w;
    int64_t ld;
    a.rows(logits, "logits", type_of(c.cfg->logits_dtype), T, E, l, ld, false);
    a.flat(bias, "bias", at::kFloat, -1, E, b, false);
    a.flat(needed(idx, "topk_idx"), "topk_idx", at::kInt, T, k, i, true);
    a.flat(needed(weights, "topk_weights"), "topk_weights", at::kFloat, T, k, w, true);
    moe_balance_io io{};
    void *ws = nullptr;
    const bool with_loss = a.at != a.end;
    if (with_loss) losses(a, T, E, true, io, ws);
    a.done();
    a.tell_of_graph("Router.forward");
    return unlocked(a, [&] { return c.fn(c.cfg, T, l, ld, b, i, w, with_loss ? &io : nullptr, ws, c.stream); });
}

// ..., logits, topk_idx, losses
int balance_loss(Args &a) {
    const Head<decltype(&moe_balance_loss), moe_router_config> c(a);
    const int E = c.cfg->num_experts;
    const at::Tensor *logits = a.tensor("logits"), *idx = a.tensor("topk_idx");
    const int T = tokens(logits, "logits");
    const void *l;
    const int32_t *i;
    int64_t ld;
    a.rows(logits, "logits", type_of(c.cfg->logits_dtype), T, E, l, ld, false);
    a.flat(needed(idx, "topk_idx"), "topk_idx", at::kInt, T, c.cfg->topk, i, false);
    moe_balance_io io{};
    void *ws;
    losses(a, T, E, true, io, ws);
    a.done();
    a.tell_of_graph("Router.balance_loss");
    return unlocked(a, [&] { return c.fn(c.cfg, T, l, ld, i, &io, ws, c.stream); });
}

// ..., logits, topk_idx, d_weights, d_logits[, d_loss, losses]
int router_backward(Args &a) {
    const Head<decltype(&moe_router_backward), moe_router_config> c(a);
    const int E = c.cfg->num_experts, k = c.cfg->topk;
    const at::Tensor *logits = a.tensor("logits"), *idx = a.tensor("topk_idx"), *weights = a.tensor("d_weights"),
                     *grad = a.tensor("d_logits");
    const int T = tokens(logits, "logits");
    const at::ScalarType s = type_of(c.cfg->logits_dtype);
    const void *l;
    const int32_t *i;
    const float *w, *dl = nullptr;
    void *g, *ws;
    int64_t ld, ld_g;
    a.rows(logits, "logits", s, T, E, l, ld, false);
    a.flat(idx, "topk_idx", at::kInt, T, k, i, false);
    a.flat(weights, "d_weights", at::kFloat, T, k, w, false);
    a.rows(needed(grad, "d_logits"), "d_logits", s, T, E, g, ld_g, true);
    moe_balance_io io{};
    const bool with_loss = a.at != a.end;
    if (with_loss) {
        const at::Tensor *d = a.tensor("d_loss");
        if (!d || d->numel() != 1 || d->scalar_type() != at::kFloat || d->get_device() != a.index)
            fail(PyExc_ValueError, "d_loss must be one f32 value on the operator's device");
        dl = static_cast<const float *>(d->const_data_ptr());
        losses(a, T, E, false, io, ws);
    }
    a.done();
    return unlocked(a, [&] { return c.fn(c.cfg, T, l, ld, i, w, with_loss ? &io : nullptr, dl, g, ld_g, c.stream); });
}

// ..., w, w_sf, store address
int linear_transform(Args &a) {
    const Head<decltype(&moe_fp4_linear_transform_weights), moe_fp4_linear_config> c(a);
    const int64_t N = c.cfg->out_features, K = c.cfg->in_features;
    const at::Tensor *w = a.tensor("w"), *w_sf = a.tensor("w_sf");
    void *store = address<void *>(a.next());
    a.done();
    const void *wp, *sp;
    a.flat(w, "w", at::kByte, N, K / 2, wp, false);
    a.flat(w_sf, "w_sf", at::kByte, N, K / 32, sp, false);
    return unlocked(a, [&] { return c.fn(c.cfg, wp, sp, store, c.stream); });
}

// ..., x, add, y, store address
int linear_forward(Args &a) {
    const Head<decltype(&moe_fp4_linear_forward), moe_fp4_linear_config> c(a);
    const int64_t n = c.cfg->act == MOE_ACT_SWIGLU ? c.cfg->out_features / 2 : c.cfg->out_features;
    const at::ScalarType o = type_of(c.cfg->out_dtype);
    const at::Tensor *x = a.tensor("x"), *add = a.tensor("add"), *y = a.tensor("y");
    const void *store = address<const void *>(a.next());
    a.done();
    const int T = tokens(x, "x");
    const void *xp, *ap;
    void *yp;
    int64_t ldx, lda, ldy;
    a.rows(x, "x", at::kBFloat16, T, c.cfg->in_features, xp, ldx, false);
    a.rows(add, "add", o, T, n, ap, lda, false);
    a.rows(needed(y, "y"), "y", o, T, n, yp, ldy, true);
    a.tell_of_graph("Fp4Linear.forward");
    return unlocked(a, [&] { return c.fn(c.cfg, T, xp, ldx, store, ap, lda, yp, ldy, c.stream); });
}

template <int (*F)(Args &)>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<norm_forward>("norm_forward"),         method<norm_backward>("norm_backward"),
                         method<router_forward>("router_forward"),     method<balance_loss>("balance_loss"),
                         method<router_backward>("router_backward"),   method<linear_transform>("linear_transform"),
                         method<linear_forward>("linear_forward"),     {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", "Tensors to the C ABI of the block operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
