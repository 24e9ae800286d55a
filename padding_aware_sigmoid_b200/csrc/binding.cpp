// Python entry points of the calls that are made once per token or layer
// (fwd_span, bwd_span, cache_append, fwd_paged): argument checks, outputs and the
// current stream in C++, then the C ABI of libsigattn.so (include/sigattn.h).
// A decoding step's kernels take a few microseconds, and the same checks in
// Python with a ctypes call of two dozen arguments took 13 to 17.  The C entry
// points are handed over by address (bind), so nothing here links to the
// library; PyTorch supplies tensors, device memory and streams only.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>
#include <string>

#include "../../include/sigattn.h"

namespace {

decltype(&sigattn_fwd_span) g_fwd_span;
decltype(&sigattn_bwd_span) g_bwd_span;
decltype(&sigattn_bwd_span_workspace_bytes) g_bwd_span_bytes;
decltype(&sigattn_cache_append) g_cache_append;
decltype(&sigattn_fwd_paged) g_fwd_paged;
decltype(&sigattn_fwd_paged_workspace_bytes) g_fwd_paged_bytes;
PyObject *g_check;    // raises for a status that is not OK

// A refusal, carried to the entry point, which raises it.
struct Refusal {
    PyObject *type;
    std::string what;
};
[[noreturn]] void refuse(const std::string &what) { throw Refusal{PyExc_ValueError, what}; }

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) throw Refusal{PyExc_TypeError, std::string(name) + " must be a tensor"};
    return THPVariable_Unpack(o);
}
const at::Tensor *optional_tensor(PyObject *o, const char *name) { return o == Py_None ? nullptr : &tensor(o, name); }

double number(PyObject *o, const char *name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refusal{PyExc_TypeError, std::string(name) + " must be a number"};
    }
    return v;
}

void *ptr(const at::Tensor *t) { return t == nullptr ? nullptr : t->data_ptr(); }
const int32_t *ints(const at::Tensor *t) { return static_cast<const int32_t *>(ptr(t)); }
const float *floats(const at::Tensor *t) { return static_cast<const float *>(ptr(t)); }

// Sizes reach the C ABI as int.
int narrow(int64_t v) {
    if (v > INT32_MAX) refuse("a size exceeds 2^31 - 1");
    return static_cast<int>(v);
}

sigattn_dtype dtype_of(const at::Tensor &t) {
    if (t.scalar_type() == at::kBFloat16) return SIGATTN_BF16;
    if (t.scalar_type() == at::kFloat) return SIGATTN_FP32;
    throw Refusal{PyExc_TypeError, std::string("sigattn takes bf16 or fp32 tensors, got ") + at::toString(t.scalar_type())};
}

// The query-side tensor of a call: [Z, L, H, D], contiguous, on a CUDA device.
struct Call {
    const at::Tensor &q;
    int Z, L, H, D, Hk = 0, device;
    explicit Call(const at::Tensor &t) : q(t) {
        if (q.dim() != 4) refuse("tensors must be [Z, L, H, D]");
        if (!q.is_cuda()) refuse("sigattn tensors must live on a CUDA device (no CPU fallback)");
        if (!q.is_contiguous()) refuse("tensors must be contiguous [Z, L, H, D]");
        Z = narrow(q.size(0));
        L = narrow(q.size(1));
        H = narrow(q.size(2));
        D = narrow(q.size(3));
        device = q.get_device();
        dtype_of(q);
    }
    void mine(const at::Tensor &t) const {
        if (t.scalar_type() != q.scalar_type() || t.get_device() != device || !t.is_cuda())
            refuse("all tensors must share dtype and device");
        if (!t.is_contiguous()) refuse("tensors must be contiguous");
    }
    // tensors [Z, L, Hk, D] of the key heads that the H query heads share
    void keys(std::initializer_list<const at::Tensor *> ts) {
        const at::Tensor &k = **ts.begin();
        for (const at::Tensor *t : ts) {
            if (t->dim() != 4 || t->sizes() != k.sizes() || t->size(0) != Z || t->size(1) != L || t->size(3) != D)
                refuse("k and v must be [Z, L, Hk, D] with the queries' Z, L and D");
            mine(*t);
        }
        share(k.size(2));
    }
    void share(int64_t heads) {
        Hk = narrow(heads);
        if (H > 0 && (Hk == 0 || H % Hk != 0))
            refuse(std::to_string(H) + " query heads cannot share " + std::to_string(Hk) + " key heads evenly");
    }
    void vector(const at::Tensor *t, at::ScalarType type, at::IntArrayRef shape, const char *name) const {
        if (t == nullptr) return;
        if (t->scalar_type() != type || t->sizes() != shape || t->get_device() != device || !t->is_cuda() ||
            !t->is_contiguous()) {
            std::string s;
            for (int64_t d : shape) s += (s.empty() ? "" : ", ") + std::to_string(d);
            refuse(std::string(name) + " must be a contiguous " + (type == at::kInt ? "int32" : "float32") + " [" + s +
                   "] tensor on the tensors' device");
        }
    }
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
        return at::detail::empty_cuda(shape, type, q.device(), std::nullopt);
    }
    // the caller's output, or a new one like `ref`
    at::Tensor output(PyObject *o, const at::Tensor &ref, const char *name) const {
        if (o == Py_None) return empty(ref.sizes(), ref.scalar_type());
        const at::Tensor &t = tensor(o, name);
        if (t.sizes() != ref.sizes() || t.scalar_type() != ref.scalar_type() || t.get_device() != device ||
            !t.is_cuda() || !t.is_contiguous())
            refuse("outputs and gradients must be contiguous, with the shape, dtype and device of the tensor they "
                   "belong to");
        return t;
    }
    // the caller's workspace, or one of `need` bytes held until the launch: its
    // memory goes back to the allocator of the current stream, in whose order it
    // may be used again
    at::Tensor workspace(PyObject *o, size_t need) const {
        if (o == Py_None) return need == 0 ? at::Tensor() : empty({static_cast<int64_t>(need)}, at::kByte);
        const at::Tensor &t = tensor(o, "workspace");
        if (t.get_device() != device || !t.is_cuda() || !t.is_contiguous())
            refuse("workspace must be a contiguous tensor on the tensors' device");
        return t;
    }
};
void *ws_ptr(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }
size_t ws_bytes(const at::Tensor &t) { return t.defined() ? t.nbytes() : 0; }

// Whether two contiguous tensors of one device share a byte.
bool overlap(const at::Tensor &a, const at::Tensor &b) {
    const char *x = static_cast<const char *>(a.data_ptr()), *y = static_cast<const char *>(b.data_ptr());
    return a.nbytes() > 0 && b.nbytes() > 0 && x < y + b.nbytes() && y < x + a.nbytes();
}

// Outputs that the caller gave must not lie over the inputs, which other blocks still
// read, or over one another.
void apart(std::initializer_list<const at::Tensor *> outs, std::initializer_list<const at::Tensor *> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const at::Tensor *i : ins)
            if (overlap(**o, *i)) refuse("outputs must not overlap inputs");
        for (auto u = outs.begin(); u != o; ++u)
            if (overlap(**o, **u)) refuse("outputs must not overlap one another");
    }
}

// bias: a number, or float32 [Z]; slopes: float32 [H] or None.
struct Score {
    float alpha, bias = 0.0f, cap;
    const float *bias_z = nullptr, *slopes;
    Score(const Call &c, PyObject *a, PyObject *b, PyObject *cp, PyObject *sl)
        : alpha(static_cast<float>(number(a, "alpha"))), cap(static_cast<float>(number(cp, "cap"))) {
        if (cap == 0.0f && number(cp, "cap") != 0.0) refuse("cap is too small for fp32 (0 stands for none)");
        if (THPVariable_Check(b)) {
            const at::Tensor &t = THPVariable_Unpack(b);
            c.vector(&t, at::kFloat, {c.Z}, "bias");
            bias_z = floats(&t);
        } else {
            bias = static_cast<float>(number(b, "bias"));
        }
        const at::Tensor *s = optional_tensor(sl, "slopes");
        c.vector(s, at::kFloat, {c.H}, "slopes");
        slopes = floats(s);
    }
};

// Calls entry point f of the library, the stream its last argument, with the
// tensors' device current and without the interpreter's lock; raises what it answers.
// The arguments are values by now: a refusal or an error of PyTorch's while they are
// formed must find the lock held.
template <typename F, typename... Args>
void run(const Call &c, const char *name, F *f, Args... args) {
    sigattn_status s;
    {
        std::optional<c10::cuda::CUDAGuard> guard;
        if (c10::cuda::current_device() != c.device) guard.emplace(static_cast<c10::DeviceIndex>(c.device));
        void *stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c.device)).stream();
        Py_BEGIN_ALLOW_THREADS;
        s = f(args..., stream);
        Py_END_ALLOW_THREADS;
    }
    if (s != SIGATTN_OK) {
        PyObject *r = PyObject_CallFunction(g_check, "is", static_cast<int>(s), name);
        Py_XDECREF(r);
        throw Refusal{nullptr, ""};    // the error is set
    }
}

// Calls an entry point's body and turns refusals and C++ errors into Python's.
template <typename F>
PyObject *guarded(Py_ssize_t given, Py_ssize_t wanted, F &&f) {
    if (given != wanted) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return f();
    } catch (const Refusal &r) {
        if (r.type != nullptr) PyErr_SetString(r.type, r.what.c_str());
    } catch (...) {
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// q, k, v, seqlens, alpha, bias, spans, cap, slopes, out
PyObject *fwd_span(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject * {
        Call c(tensor(a[0], "q"));
        const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &seqlens = tensor(a[3], "seqlens");
        c.keys({&k, &v});
        const at::Tensor *spans = optional_tensor(a[6], "spans");
        c.vector(&seqlens, at::kInt, {c.Z}, "seqlens");
        c.vector(spans, at::kInt, {c.Z, c.L, 2}, "spans");
        const Score s(c, a[4], a[5], a[7], a[8]);
        at::Tensor out = c.output(a[9], c.q, "out");
        if (a[9] != Py_None) apart({&out}, {&c.q, &k, &v});
        run(c, "sigattn_fwd_span", g_fwd_span, ptr(&c.q), ptr(&k), ptr(&v), ptr(&out), ints(&seqlens), ints(spans),
            c.Z, c.L, c.H, c.Hk, c.D, s.alpha, s.bias, s.bias_z, s.cap, s.slopes, dtype_of(c.q));
        return THPVariable_Wrap(std::move(out));
    });
}

// q, k, v, dout, seqlens, alpha, bias, spans, cap, slopes, dq, dk, dv, workspace
PyObject *bwd_span(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 14, [&]() -> PyObject * {
        Call c(tensor(a[0], "q"));
        const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &seqlens = tensor(a[4], "seqlens");
        c.keys({&k, &v});
        const at::Tensor dout = c.output(a[3], c.q, "dout");
        if (a[3] == Py_None) refuse("dout must be a tensor");
        const at::Tensor *spans = optional_tensor(a[7], "spans");
        c.vector(&seqlens, at::kInt, {c.Z}, "seqlens");
        c.vector(spans, at::kInt, {c.Z, c.L, 2}, "spans");
        const Score s(c, a[5], a[6], a[8], a[9]);
        at::Tensor dq = c.output(a[10], c.q, "dq"), dk = c.output(a[11], k, "dk"), dv = c.output(a[12], v, "dv");
        if (a[10] != Py_None || a[11] != Py_None || a[12] != Py_None) apart({&dq, &dk, &dv}, {&c.q, &k, &v, &dout});
        const sigattn_dtype dt = dtype_of(c.q);
        const at::Tensor ws = c.workspace(a[13], g_bwd_span_bytes(c.Z, c.L, dt));
        run(c, "sigattn_bwd_span", g_bwd_span, ptr(&c.q), ptr(&k), ptr(&v), ptr(&dout), ptr(&dq), ptr(&dk), ptr(&dv),
            ints(&seqlens), ints(spans), c.Z, c.L, c.H, c.Hk, c.D, s.alpha, s.bias, s.bias_z, s.cap, s.slopes,
            ws_ptr(ws), ws_bytes(ws), dt);
        return Py_BuildValue("(NNN)", THPVariable_Wrap(std::move(dq)), THPVariable_Wrap(std::move(dk)),
                             THPVariable_Wrap(std::move(dv)));
    });
}

// Cache pages [pages, page_size, Hk, D] beside a call's tensors; how many there are.
int check_pages(const Call &c, const at::Tensor &k, const at::Tensor &v) {
    if (k.dim() != 4 || k.size(3) != c.D || v.sizes() != k.sizes())
        refuse("k_pages and v_pages must be [pages, page_size, Hk, D]");
    for (const at::Tensor *t : {&k, &v})
        if (t->scalar_type() != c.q.scalar_type() || t->get_device() != c.device || !t->is_cuda() || !t->is_contiguous())
            refuse("k_pages and v_pages must be contiguous, with the tensors' dtype and device");
    const int64_t page = k.size(1);
    if (page != 16 && page != 32 && page != 64 && page != 128 && page != 256)
        refuse("page_size must be 16, 32, 64, 128 or 256, got " + std::to_string(page));
    return narrow(k.size(0));
}
int check_table(const Call &c, const at::Tensor &t) {
    if (t.dim() != 2) refuse("page_table must be a contiguous int32 [Z, max_pages] tensor");
    c.vector(&t, at::kInt, {c.Z, t.size(1)}, "page_table");
    return narrow(t.size(1));
}

// k, v, k_pages, v_pages, page_table, cache_lens, seqlens_new, inv_freq, interleaved, q, prefix_len, q_out, lens_out
PyObject *cache_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject * {
        const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
        const at::Tensor *q = optional_tensor(a[9], "q");
        Call c(q != nullptr ? *q : k);
        c.keys({&k, &v});
        const at::Tensor &kp = tensor(a[2], "k_pages"), &vp = tensor(a[3], "v_pages"), &table = tensor(a[4], "page_table");
        const at::Tensor &lens = tensor(a[5], "cache_lens"), &add = tensor(a[6], "seqlens_new");
        const int pages = check_pages(c, kp, vp);
        if (kp.size(2) != c.Hk) refuse("k_pages and v_pages must be [pages, page_size, Hk, D]");
        const int most = check_table(c, table);
        c.vector(&lens, at::kInt, {c.Z}, "cache_lens");
        c.vector(&add, at::kInt, {c.Z}, "seqlens_new");
        const at::Tensor *prefix = optional_tensor(a[10], "prefix_len"), *freq = optional_tensor(a[7], "inv_freq");
        c.vector(prefix, at::kInt, {1}, "prefix_len");
        int rot = 0;
        if (freq != nullptr) {
            c.vector(freq, at::kFloat, {freq->numel()}, "inv_freq");
            rot = narrow(2 * freq->numel());
            if (rot % 16 != 0 || rot > c.D)
                refuse("inv_freq must turn a multiple of 16 entries of a head, at most " + std::to_string(c.D) + ", got " +
                       std::to_string(rot));
        }
        const int interleaved = PyObject_IsTrue(a[8]);
        if (interleaved < 0) throw Refusal{nullptr, ""};
        at::Tensor out;
        if (q != nullptr) {
            out = c.output(a[11], *q, "q_out");
            if (overlap(out, k) || overlap(out, v) || (overlap(out, *q) && out.data_ptr() != q->data_ptr()))
                refuse("q_out must be q itself or overlap no input");
        }
        at::Tensor after = c.output(a[12], lens, "lens_out");
        // a sample's lengths are read by many warps, of which one writes the new one
        const bool itself = c.L == 1 && after.data_ptr() == lens.data_ptr();
        if ((overlap(after, lens) && !itself) || overlap(after, add) || (prefix != nullptr && overlap(after, *prefix)))
            refuse("lens_out must not overlap the lengths (it can be cache_lens itself for single tokens)");
        run(c, "sigattn_cache_append", g_cache_append, ptr(&k), ptr(&v), ptr(q), q != nullptr ? ptr(&out) : nullptr,
            ptr(&kp), ptr(&vp), ints(&table), ints(&lens), ints(&add), ints(prefix),
            static_cast<int32_t *>(ptr(&after)), c.Z, c.L, q != nullptr ? c.H : 0, c.Hk, c.D, pages,
            static_cast<int>(kp.size(1)), most, floats(freq), rot, interleaved, dtype_of(k));
        PyObject *first = q != nullptr ? THPVariable_Wrap(std::move(out)) : (Py_INCREF(Py_None), Py_None);
        return Py_BuildValue("(NN)", first, THPVariable_Wrap(std::move(after)));
    });
}

// q, k_pages, v_pages, page_table, seqlens_k, seqlens_q, alpha, bias, prefix_table, prefix_len, cap, slopes, out, workspace
PyObject *fwd_paged(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 14, [&]() -> PyObject * {
        Call c(tensor(a[0], "q"));
        const at::Tensor &kp = tensor(a[1], "k_pages"), &vp = tensor(a[2], "v_pages"), &table = tensor(a[3], "page_table");
        const at::Tensor &nk = tensor(a[4], "seqlens_k"), &nq = tensor(a[5], "seqlens_q");
        const int pages = check_pages(c, kp, vp);
        c.share(kp.size(2));
        const int most = check_table(c, table);
        c.vector(&nk, at::kInt, {c.Z}, "seqlens_k");
        c.vector(&nq, at::kInt, {c.Z}, "seqlens_q");
        const at::Tensor *pre = optional_tensor(a[8], "prefix_table"), *len = optional_tensor(a[9], "prefix_len");
        if ((pre == nullptr) != (len == nullptr)) refuse("prefix_table and prefix_len go together");
        int ahead = 0;
        if (pre != nullptr) {
            c.vector(pre, at::kInt, {pre->numel()}, "prefix_table");
            c.vector(len, at::kInt, {1}, "prefix_len");
            ahead = narrow(pre->numel());
        }
        const Score s(c, a[6], a[7], a[10], a[11]);
        at::Tensor out = c.output(a[12], c.q, "out");
        // over q itself: in bf16 the last kernel writes, when all have read; in fp32 each
        // row's block reads its queries first, and no other row's
        if (a[12] != Py_None && ((overlap(out, c.q) && out.data_ptr() != c.q.data_ptr()) || overlap(out, kp) || overlap(out, vp)))
            refuse("out must be q itself or overlap no input");
        const sigattn_dtype dt = dtype_of(c.q);
        const at::Tensor ws = c.workspace(a[13], g_fwd_paged_bytes(c.Z, c.L, c.H, c.Hk, c.D, dt));
        run(c, "sigattn_fwd_paged", g_fwd_paged, ptr(&c.q), ptr(&kp), ptr(&vp), ptr(&out), ints(&table), ints(&nk),
            ints(&nq), ints(pre), ints(len), c.Z, c.L, c.H, c.Hk, c.D, pages, static_cast<int>(kp.size(1)), most,
            ahead, s.alpha, s.bias, s.bias_z, s.cap, s.slopes, ws_ptr(ws), ws_bytes(ws), dt);
        return THPVariable_Wrap(std::move(out));
    });
}

// bind({name: address}, check)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 2, [&]() -> PyObject * {
        auto at = [&](const char *name) {
            PyObject *v = PyDict_GetItemString(a[0], name);
            void *p = v != nullptr ? PyLong_AsVoidPtr(v) : nullptr;
            if (p == nullptr) refuse(std::string("no address of ") + name);
            return p;
        };
        g_fwd_span = reinterpret_cast<decltype(g_fwd_span)>(at("sigattn_fwd_span"));
        g_bwd_span = reinterpret_cast<decltype(g_bwd_span)>(at("sigattn_bwd_span"));
        g_bwd_span_bytes = reinterpret_cast<decltype(g_bwd_span_bytes)>(at("sigattn_bwd_span_workspace_bytes"));
        g_cache_append = reinterpret_cast<decltype(g_cache_append)>(at("sigattn_cache_append"));
        g_fwd_paged = reinterpret_cast<decltype(g_fwd_paged)>(at("sigattn_fwd_paged"));
        g_fwd_paged_bytes = reinterpret_cast<decltype(g_fwd_paged_bytes)>(at("sigattn_fwd_paged_workspace_bytes"));
        Py_XDECREF(g_check);
        g_check = Py_NewRef(a[1]);
        Py_RETURN_NONE;
    });
}

#define CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {CALL(bind), CALL(fwd_span), CALL(bwd_span), CALL(cache_append), CALL(fwd_paged),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&g_module); }
