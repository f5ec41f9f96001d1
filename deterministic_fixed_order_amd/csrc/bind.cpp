// bind.cpp -- the ordinary call of a decode-step operator from Python, without
// the interpreter's share of it: reads the tensors, fills the public struct
// and calls the library (a Python call costs 4 to 7 us of reading ten tensors'
// types, shapes and strides, of which this needs less than 1).
//
// Only what it can take as it is: anything else (a wrong type, shape, device
// or layout, a missing argument) returns -1, and decode.py, whose checks are
// the same, says what is wrong.  So does whatever torch throws here (a tensor
// within a function transform has no address to give).  The library's functions
// come as addresses, so this links to neither the library nor HIP.

#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>

#include "detfold.h"

namespace {

struct Arg {
    const at::Tensor *t = nullptr;
    bool none = false;
    explicit Arg(PyObject *o)
    {
        none = o == Py_None;
        if (!none && THPVariable_Check(o))
            t = &THPVariable_Unpack(o);
    }
    // A tensor of this device, its last dimension contiguous.
    bool on(int64_t dev) const
    {
        return t && t->layout() == c10::kStrided && t->get_device() == dev && t->dim() > 0 &&
               (t->stride(-1) == 1 || t->size(-1) == 1);
    }
    // [n, heads, dim] (heads = 0: any)
    bool heads(int64_t dev, c10::ScalarType type, int64_t n, int64_t heads, int64_t dim) const
    {
        return on(dev) && t->scalar_type() == type && t->dim() == 3 && t->size(0) == n && t->size(2) == dim &&
               (heads == 0 || t->size(1) == heads);
    }
    // contiguous, of a shape
    bool plain(int64_t dev, c10::ScalarType type, c10::IntArrayRef shape) const
    {
        return t && t->layout() == c10::kStrided && t->get_device() == dev && t->scalar_type() == type && t->sizes() == shape &&
               t->is_contiguous();
    }
    template <typename T = void> const T *read() const { return t ? static_cast<const T *>(t->const_data_ptr()) : nullptr; }
    // For what is written: memory that the tensor shares with a lazy copy becomes its own.
    template <typename T = void> T *written() const { return t ? static_cast<T *>(t->mutable_data_ptr()) : nullptr; }
};

int type_of(c10::ScalarType t)
{
    return t == c10::kFloat ? DETFOLD_F32 : t == c10::kBFloat16 ? DETFOLD_BF16 : t == c10::kHalf ? DETFOLD_F16 : -1;
}

int cache_type_of(c10::ScalarType t) { return t == c10::kFloat8_e4m3fn ? DETFOLD_E4M3 : type_of(t); }

struct Numbers {
    bool ok = true;
    int64_t whole(PyObject *o)
    {
        const int64_t v = PyLong_Check(o) ? PyLong_AsLongLong(o) : (ok = false, 0);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return v;
    }
    void *address(PyObject *o)
    {
        void *p = PyLong_Check(o) ? PyLong_AsVoidPtr(o) : (ok = false, nullptr);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return p;
    }
};

PyObject *kDescribed, *kKeys, *kValues, *kKeyScale, *kValueScale;  // names of a PagedCache's attributes

struct Attr {  // one of these, held
    PyObject *o;
    Attr(PyObject *of, PyObject *name) : o(PyObject_GetAttr(of, name))
    {
        if (!o) {
            PyErr_Clear();
            o = Py_NewRef(Py_None);
        }
    }
    Attr(const Attr &) = delete;
    ~Attr() { Py_DECREF(o); }
};

// A PagedCache as it was described when it was made, with the addresses and
// strides that its tensors have now.
bool cache_of(PyObject *o, int64_t dev, bool written, detfold_paged_cache *c)
{
    const Attr described(o, kDescribed), ko(o, kKeys), vo(o, kValues);
    if (!PyBytes_Check(described.o) || PyBytes_GET_SIZE(described.o) != (Py_ssize_t)sizeof(*c))
        return false;
    std::memcpy(c, PyBytes_AS_STRING(described.o), sizeof(*c));
    const Arg k(ko.o), v(vo.o);
    for (const Arg *x : {&k, &v})
        if (!x->on(dev) || x->t->dim() != 4 || cache_type_of(x->t->scalar_type()) != c->type || x->t->size(0) != c->pages ||
            x->t->size(1) != c->page || x->t->size(2) != c->heads || x->t->size(3) != (x == &k ? c->dim : c->v_dim))
            return false;
    c->k = written ? k.written() : const_cast<void *>(k.read()), c->v = written ? v.written() : const_cast<void *>(v.read());
    c->k_page = k.t->stride(0), c->k_token = k.t->stride(1), c->k_head = k.t->stride(2);
    c->v_page = v.t->stride(0), c->v_token = v.t->stride(1), c->v_head = v.t->stride(2);
    for (const float **scale : {&c->k_scale, &c->v_scale})
        if (*scale) {
            const Attr so(o, scale == &c->k_scale ? kKeyScale : kValueScale);
            const Arg x(so.o);
            if (!x.plain(dev, c10::kFloat, {c->heads}))
                return false;
            *scale = x.read<float>();
        }
    return true;
}

// The library's call, without the interpreter's lock (which the arguments,
// evaluated before, still hold: what throws there needs it).
template <typename F, typename... A> int unlocked(F f, A... args)
{
    PyThreadState *const state = PyEval_SaveThread();
    const int rc = f(args...);
    PyEval_RestoreThread(state);
    return rc;
}

PyObject *not_taken() { return PyLong_FromLong(-1); }

typedef int (*AppendFn)(const detfold_paged_cache *, const detfold_append *, void *);
typedef int (*AttendFn)(const detfold_paged_cache *, const detfold_attend *, void *);
typedef int (*FoldFn)(void *, const void *, const float *, float *, int32_t, int32_t, int64_t, int64_t, int64_t, int64_t, void *);

// (function, cache, device, stream, k, v, slots, q, q_out, positions, cos, sin, pairs)
PyObject *append(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    detfold_paged_cache c;
    Numbers num;
    if (n != 13)
        return not_taken();
    const AppendFn f = (AppendFn)num.address(args[0]);
    const int64_t dev = num.whole(args[2]);
    if (!cache_of(args[1], dev, true, &c))
        return not_taken();
    void *stream = num.address(args[3]);
    const Arg k(args[4]), v(args[5]), slots(args[6]), q(args[7]), q_out(args[8]), positions(args[9]), cos(args[10]), sin(args[11]);
    if (!num.ok || !k.t || k.t->dim() != 3)
        return not_taken();
    const c10::ScalarType type = k.t->scalar_type();
    const int64_t tokens = k.t->size(0);
    detfold_append a = {};
    a.type = type_of(type);
    if (a.type < 0 || !k.heads(dev, type, tokens, c.heads, c.dim) || !v.heads(dev, type, tokens, c.heads, c.v_dim) ||
        !slots.plain(dev, c10::kLong, {tokens}))
        return not_taken();
    a.slots = slots.read<int64_t>();
    a.tokens = tokens;
    if (!q.none) {
        if (!q.heads(dev, type, tokens, 0, c.dim) || q.t->size(1) > INT32_MAX || !q_out.heads(dev, type, tokens, q.t->size(1), c.dim))
            return not_taken();
        a.q_out = q_out.written(), a.q = q.read();  // in this order: all may be one tensor's
        a.q_token = q.t->stride(0), a.q_head = q.t->stride(1);
        a.out_token = q_out.t->stride(0), a.out_head = q_out.t->stride(1);
        a.q_heads = (int32_t)q.t->size(1);
    } else if (!q_out.none) {
        return not_taken();
    }
    a.k = k.read(), a.k_token = k.t->stride(0), a.k_head = k.t->stride(1);
    a.v = v.read(), a.v_token = v.t->stride(0), a.v_head = v.t->stride(1);
    if (!cos.none) {
        if (!cos.t || cos.t->dim() != 2 || cos.t->size(1) > INT32_MAX / 2 || !cos.plain(dev, c10::kFloat, cos.t->sizes()) ||
            !sin.plain(dev, c10::kFloat, cos.t->sizes()) || !positions.plain(dev, c10::kLong, {tokens}))
            return not_taken();
        a.cos = cos.read<float>(), a.sin = sin.read<float>(), a.positions = positions.read<int64_t>();
        a.angles = cos.t->size(0);
        a.rot = (int32_t)(2 * cos.t->size(1));
    } else if (!sin.none || !positions.none) {
        return not_taken();
    }
    a.pairs = args[12] == Py_True ? 1 : 0;
    if (args[12] != Py_True && args[12] != Py_False)
        return not_taken();
    return PyLong_FromLong(unlocked(f, &c, &a, stream));
}

// (function, cache, device, stream, out, q, table, lens, scale, window, max_len, lse, workspace, split)
PyObject *attend(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    detfold_paged_cache c;
    Numbers num;
    if (n != 14)
        return not_taken();
    const AttendFn f = (AttendFn)num.address(args[0]);
    const int64_t dev = num.whole(args[2]);
    if (!cache_of(args[1], dev, false, &c))
        return not_taken();
    void *stream = num.address(args[3]);
    const Arg out(args[4]), q(args[5]), table(args[6]), lens(args[7]), lse(args[11]), workspace(args[12]);
    detfold_attend a = {};
    a.window = num.whole(args[9]), a.max_len = num.whole(args[10]);
    const int64_t split = num.whole(args[13]);
    if (!num.ok || !PyFloat_Check(args[8]) || split < 0 || split > INT32_MAX || !q.t || q.t->dim() != 3 || !out.t)
        return not_taken();
    const double scale = PyFloat_AS_DOUBLE(args[8]);
    a.scale = (float)scale;
    if (std::isfinite(scale) != std::isfinite(a.scale))
        return not_taken();
    const int64_t batch = q.t->size(0), q_heads = q.t->size(1);
    const c10::ScalarType type = q.t->scalar_type(), out_type = out.t->scalar_type();
    a.type = type_of(type), a.out_type = type_of(out_type);
    if (a.type < 0 || (out_type != type && out_type != c10::kFloat) || q_heads > INT32_MAX || !q.heads(dev, type, batch, 0, c.dim) ||
        !out.heads(dev, out_type, batch, q_heads, c.v_dim) || !lens.plain(dev, c10::kInt, {batch}))
        return not_taken();
    if (!table.on(dev) || table.t->scalar_type() != c10::kInt || table.t->dim() != 2 || table.t->size(0) != batch)
        return not_taken();
    if (!lse.none && !lse.plain(dev, c10::kFloat, {batch, q_heads}))
        return not_taken();
    if (!workspace.t || workspace.t->get_device() != dev || !workspace.t->is_contiguous())
        return not_taken();
    a.out = out.written(), a.out_row = out.t->stride(0), a.out_head = out.t->stride(1);
    a.q = q.read(), a.q_row = q.t->stride(0), a.q_head = q.t->stride(1);
    a.lse = lse.written<float>();
    a.table = table.read<int32_t>(), a.table_row = table.t->stride(0), a.table_width = table.t->size(1);
    a.lens = lens.read<int32_t>();
    a.workspace = workspace.written(), a.workspace_bytes = (int64_t)workspace.t->nbytes();
    a.batch = batch, a.q_heads = (int32_t)q_heads, a.split = (int32_t)split;
    return PyLong_FromLong(unlocked(f, &c, &a, stream));
}

// (function, device, stream, out, outs, lses, lse)
PyObject *fold(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    Numbers num;
    if (n != 7)
        return not_taken();
    const FoldFn f = (FoldFn)num.address(args[0]);
    const int64_t dev = num.whole(args[1]);
    void *stream = num.address(args[2]);
    const Arg out(args[3]), outs(args[4]), lses(args[5]), lse(args[6]);
    if (!num.ok || dev < 0 || !outs.on(dev) || outs.t->dim() < 2 || outs.t->size(0) < 1 || outs.t->size(0) > INT32_MAX)
        return not_taken();
    const at::Tensor &o = *outs.t;
    const c10::IntArrayRef shape = o.sizes(), one = shape.slice(1), rows_shape = one.slice(0, one.size() - 1);
    const int type = type_of(o.scalar_type());
    if (type < 0 || !out.plain(dev, o.scalar_type(), one) || !lses.t || lses.t->layout() != c10::kStrided || lses.t->get_device() != dev ||
        lses.t->scalar_type() != c10::kFloat || lses.t->sizes() != shape.slice(0, shape.size() - 1))
        return not_taken();
    if (!lse.none && !lse.plain(dev, c10::kFloat, rows_shape))
        return not_taken();
    int64_t rows = 1;  // each partial contiguous
    for (int64_t d = (int64_t)shape.size() - 2, step = shape.back(), lse_step = 1; d > 0; --d) {
        if (shape[d] != 1 && (o.stride(d) != step || lses.t->stride(d) != lse_step))
            return not_taken();
        step *= shape[d], lse_step *= shape[d], rows *= shape[d];
    }
    const int64_t W = shape[0], dim = shape.back();
    return PyLong_FromLong(unlocked(f, out.written(), outs.read(), lses.read<float>(), lse.written<float>(), type, (int32_t)W, rows, dim,
                                    W > 1 ? o.stride(0) : rows * dim, W > 1 ? lses.t->stride(0) : rows, stream));
}

// A call that lets no C++ exception into the interpreter, which would end the
// process.  The library's functions are C and throw none, so nothing was done yet.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    try {
        return F(self, args, n);
    } catch (...) {
        PyErr_Clear();
        return not_taken();
    }
}

PyMethodDef methods[] = {
    {"append", (PyCFunction)(void (*)(void))guarded<append>, METH_FASTCALL, nullptr},
    {"attend", (PyCFunction)(void (*)(void))guarded<attend>, METH_FASTCALL, nullptr},
    {"fold", (PyCFunction)(void (*)(void))guarded<fold>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind()
{
    const struct {
        PyObject **at;
        const char *name;
    } names[] = {{&kDescribed, "_c"}, {&kKeys, "k"}, {&kValues, "v"}, {&kKeyScale, "k_scale"}, {&kValueScale, "v_scale"}};
    for (const auto &n : names)
        if (!(*n.at = PyUnicode_InternFromString(n.name)))
            return nullptr;
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_from", DETFOLD_BUILT_FROM) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
