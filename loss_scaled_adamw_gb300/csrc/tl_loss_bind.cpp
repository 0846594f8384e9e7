// tl_loss_bind.cpp - the objectives' calls (include/tl_loss.h) and dropout (include/tl_dropout.h) as a
// CPython module that reads torch tensors directly.  It checks and marshals arguments and nothing else.
//
// Why not ctypes, as the rest of the binding: a loss call passes up to twelve tensors, and
// asking each for its type, size, layout, device and address through Python costs about 0.4 us
// apiece on a Grace core, in all more than the launch (policy call: 10.2 us through ctypes).
//
// Every function takes the context's handle and device, the call's tensors and numbers in the
// order of the Python wrapper, and the raw stream; it returns the status code, or raises
// ValueError for a tensor of the wrong type, shape, layout or device.
#include <Python.h>

#include <exception>

#include <torch/csrc/autograd/python_variable.h>

#include "../../include/tl_dropout.h"
#include "../../include/tl_loss.h"

namespace {

struct Error {};   // a Python error is set

[[noreturn]] void refuse(const char* name, const char* what) {
    PyErr_Format(PyExc_ValueError, "%s must be %s", name, what);
    throw Error{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(name, "a torch tensor");
    return THPVariable_Unpack(o);
}

bool on_device(const at::Tensor& t, long device) { return t.is_cuda() && t.get_device() == device; }

// The address of a contiguous device vector of n elements, null for None.
void* vector(PyObject* o, at::ScalarType type, int64_t n, long device, const char* name) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type || t.numel() != n || !on_device(t, device) || !t.is_contiguous()) {
        PyErr_Format(PyExc_ValueError, "%s must be a contiguous %s tensor of %lld elements on cuda:%ld", name,
                     type == at::kLong ? "int64" : "float32", static_cast<long long>(n), device);
        throw Error{};
    }
    return t.data_ptr();
}
float* floats(PyObject* o, int64_t n, long device, const char* name) {
    return static_cast<float*>(vector(o, at::kFloat, n, device, name));
}
int64_t* longs(PyObject* o, int64_t n, long device, const char* name) {
    return static_cast<int64_t*>(vector(o, at::kLong, n, device, name));
}

struct Matrix {
    void* data;
    int64_t rows, cols, ld;
    at::ScalarType type;
};
Matrix matrix(PyObject* o, long device, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != 2 || !on_device(t, device)) {
        PyErr_Format(PyExc_ValueError, "%s must be a 2-D tensor on cuda:%ld", name, device);
        throw Error{};
    }
    const int64_t rows = t.size(0), cols = t.size(1), ld = t.stride(0);
    if (t.stride(1) != 1 && cols > 1) refuse(name, "a matrix with contiguous rows");
    return {t.data_ptr(), rows, cols, rows > 1 || ld > cols ? ld : cols, t.scalar_type()};
}
int float_type(at::ScalarType t) {
    return t == at::kFloat ? TL_F32 : t == at::kBFloat16 ? TL_BF16 : t == at::kHalf ? TL_F16 : -1;
}

float number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Error{};
    return static_cast<float>(v);
}
int64_t whole(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Error{};
    return v;
}
void* address(PyObject* o) {
    if (o == Py_None) return nullptr;
    void* p = PyLong_AsVoidPtr(o);
    if (p == nullptr && PyErr_Occurred()) throw Error{};
    return p;
}

tl_logits logits(PyObject* o, PyObject* temperature, long device) {
    const Matrix m = matrix(o, device, "logits");
    const int type = float_type(m.type);
    if (type < 0) refuse("logits", "float32, bfloat16 or float16");
    return {m.data, m.rows, m.cols, m.ld, type, number(temperature)};
}

// A device float: its address as an integer, or a tensor of one element, or None.  0 is what
// tl_scale_ptr gives for a destroyed context: no seed at all would scale the gradient by 1.
const float* seed_of(PyObject* o, long device) {
    if (!PyLong_Check(o)) return floats(o, 1, device, "seed");
    const float* p = static_cast<const float*>(address(o));
    if (p == nullptr) refuse("seed", "a device address other than 0, a tensor of one element or None");
    return p;
}

void gradient(PyObject* o, const tl_logits& x, long device, void*& data, int64_t& ld) {
    const Matrix d = matrix(o, device, "dlogits");
    if (float_type(d.type) != x.dtype || d.rows != x.rows || d.cols != x.vocab)
        refuse("dlogits", "of the logits' shape and dtype");
    data = d.data;
    ld = d.ld;
}

// The three floats per row that the forward saves.
tl_token_saved* saved_of(PyObject* o, int64_t rows, long device) {
    if (o != Py_None && (tensor(o, "saved").dim() != 2 || tensor(o, "saved").size(1) != 3)) refuse("saved", "[rows, 3]");
    return reinterpret_cast<tl_token_saved*>(floats(o, 3 * rows, device, "saved"));
}

// n, seed, dlogits, logp, loss (of `losses` elements), result
tl_loss_out outputs(PyObject* n, PyObject* seed, PyObject* dlogits, PyObject* logp, PyObject* loss, int64_t losses,
                    PyObject* result, const tl_logits& x, long device) {
    tl_loss_out o{};
    o.n = whole(n);
    o.seed = seed_of(seed, device);
    if (dlogits != Py_None) gradient(dlogits, x, device, o.dlogits, o.ld_dlogits);
    o.logp = floats(logp, x.rows, device, "logp");
    o.loss = floats(loss, losses, device, "the loss output");
    o.result = reinterpret_cast<tl_loss_result*>(floats(result, 4, device, "result"));
    return o;
}

// handle, device, logits, temperature, targets, logp, stream
int token_logprob(PyObject* const* a) {
    const long device = static_cast<long>(whole(a[1]));
    const tl_logits x = logits(a[2], a[3], device);
    return tl_token_logprob(static_cast<tl_loss_ctx*>(address(a[0])), &x, longs(a[4], x.rows, device, "targets"),
                            floats(a[5], x.rows, device, "logp"), address(a[6]));
}

// handle, device, logits, temperature, n, seed, dlogits, logp, loss, result, stream, then:
// targets, old_logp, ref_logp, advantages, clip_low, clip_high, kl_weight
int policy_loss(PyObject* const* a) {
    const long device = static_cast<long>(whole(a[1]));
    const tl_logits x = logits(a[2], a[3], device);
    const tl_loss_out o = outputs(a[4], a[5], a[6], a[7], a[8], x.rows, a[9], x, device);
    const tl_policy_args p{longs(a[11], x.rows, device, "targets"), floats(a[12], x.rows, device, "old_logp"),
                           floats(a[13], x.rows, device, "ref_logp"), floats(a[14], x.rows, device, "advantages"),
                           number(a[15]), number(a[16]), number(a[17])};
    return tl_policy_loss(static_cast<tl_loss_ctx*>(address(a[0])), &x, &p, &o, address(a[10]));
}

// ... targets, seq, ref_logp, beta, label_smoothing, reward
int preference_loss(PyObject* const* a) {
    const long device = static_cast<long>(whole(a[1]));
    const tl_logits x = logits(a[2], a[3], device);
    const int64_t bounds = tensor(a[12], "seq").numel();
    if (bounds % 2 != 1) refuse("seq", "2 * pairs + 1 offsets");
    const int64_t pairs = bounds / 2;
    const tl_loss_out o = outputs(a[4], a[5], a[6], a[7], a[8], pairs, a[9], x, device);
    const tl_preference_args p{longs(a[11], x.rows, device, "targets"), longs(a[12], bounds, device, "seq"), pairs,
                               floats(a[13], x.rows, device, "ref_logp"), number(a[14]), number(a[15]),
                               floats(a[16], 2 * pairs, device, "reward")};
    return tl_preference_loss(static_cast<tl_loss_ctx*>(address(a[0])), &x, &p, &o, address(a[10]));
}

// ... targets, teacher_logits, teacher_ids, kd_weight, ce_weight
int distill_loss(PyObject* const* a) {
    const long device = static_cast<long>(whole(a[1]));
    const tl_logits x = logits(a[2], a[3], device);
    const tl_loss_out o = outputs(a[4], a[5], a[6], a[7], a[8], x.rows, a[9], x, device);
    tl_distill_args p{};
    p.target = longs(a[11], x.rows, device, "targets");
    if (a[12] != Py_None || a[13] != Py_None) {   // one without the other is refused
        const Matrix t = matrix(a[12], device, "teacher_logits"), ids = matrix(a[13], device, "teacher_ids");
        if (t.rows != x.rows || ids.rows != x.rows || ids.cols != t.cols || ids.ld != t.ld)
            refuse("teacher_logits and teacher_ids", "[rows, k] with one row stride");
        if (t.cols > INT32_MAX) refuse("k", "below 2^31");
        p.teacher = t.data;
        p.teacher_id = ids.data;
        p.ld_teacher = t.ld;
        p.k = static_cast<int32_t>(t.cols);
        p.teacher_dtype = float_type(t.type);
        p.id_bytes = ids.type == at::kInt ? 4 : ids.type == at::kLong ? 8 : -1;
    }
    p.kd_weight = number(a[14]);
    p.ce_weight = number(a[15]);
    return tl_distill_loss(static_cast<tl_loss_ctx*>(address(a[0])), &x, &p, &o, address(a[10]));
}

// handle, device, logits, temperature, targets, logp, entropy, saved, top_ids, top_logp, stream
int token_stats(PyObject* const* a) {
    const long device = static_cast<long>(whole(a[1]));
    const tl_logits x = logits(a[2], a[3], device);
    tl_token_stats_args p{};
    p.target = longs(a[4], x.rows, device, "targets");
    p.logp = floats(a[5], x.rows, device, "logp");
    p.entropy = floats(a[6], x.rows, device, "entropy");
    p.saved = saved_of(a[7], x.rows, device);
    if (a[8] != Py_None || a[9] != Py_None) {   // one without the other is refused
        const Matrix ids = matrix(a[8], device, "top_ids"), t = matrix(a[9], device, "top_logp");
        if (t.rows != x.rows || ids.rows != x.rows || ids.cols != t.cols || (t.rows > 1 && ids.ld != t.ld))
            refuse("top_ids and top_logp", "[rows, k] with one row stride");
        if (t.type != at::kFloat) refuse("top_logp", "float32");
        if (t.cols > INT32_MAX) refuse("k", "below 2^31");
        p.top_id = ids.data;
        p.top_logp = static_cast<float*>(t.data);
        p.ld_top = t.rows > 1 ? t.ld : t.cols;
        p.k = static_cast<int32_t>(t.cols);
        p.id_bytes = ids.type == at::kInt ? 4 : ids.type == at::kLong ? 8 : -1;
    }
    return tl_token_stats(static_cast<tl_loss_ctx*>(address(a[0])), &x, &p, address(a[10]));
}

// handle, device, logits, temperature, saved, dlogits, targets, grad_logp, grad_entropy, seed, stream
int token_grad(PyObject* const* a) {
    const long device = static_cast<long>(whole(a[1]));
    const tl_logits x = logits(a[2], a[3], device);
    tl_token_grad_args p{};
    p.saved = saved_of(a[4], x.rows, device);
    if (a[5] != Py_None) gradient(a[5], x, device, p.dlogits, p.ld_dlogits);
    p.target = longs(a[6], x.rows, device, "targets");
    p.grad_logp = floats(a[7], x.rows, device, "grad_logp");
    p.grad_entropy = floats(a[8], x.rows, device, "grad_entropy");
    p.seed = seed_of(a[9], device);
    return tl_token_grad(static_cast<tl_loss_ctx*>(address(a[0])), &x, &p, address(a[10]));
}

// x, y, residual, key, site, p, stream, device.  Tensors without gaps are one row, whatever their shape.
int dropout(PyObject* const* a) {
    const long device = static_cast<long>(whole(a[7]));
    const at::Tensor &x = tensor(a[0], "x"), &y = tensor(a[1], "y");
    const at::Tensor* const res = a[2] == Py_None ? nullptr : &tensor(a[2], "residual");
    tl_dropout_args p{};
    p.dtype = float_type(x.scalar_type());
    if (p.dtype < 0) refuse("x", "float32, bfloat16 or float16");
    for (const at::Tensor* t : {&x, &y, res}) {
        if (t == nullptr) continue;
        if (t->scalar_type() != x.scalar_type() || t->sizes() != x.sizes() || !on_device(*t, device))
            refuse("y and residual", "of the shape, dtype and device of x");
    }
    if (x.is_contiguous() && y.is_contiguous() && (res == nullptr || res->is_contiguous())) {
        p.x = x.data_ptr();
        p.y = y.data_ptr();
        p.residual = res ? res->data_ptr() : nullptr;
        p.rows = 1;
        p.cols = p.ldx = p.ldy = p.ldr = x.numel();
    } else {
        const Matrix mx = matrix(a[0], device, "x"), my = matrix(a[1], device, "y");
        p.x = mx.data;
        p.y = my.data;
        p.rows = mx.rows;
        p.cols = mx.cols;
        p.ldx = mx.ld;
        p.ldy = my.ld;
        if (res) {
            const Matrix mr = matrix(a[2], device, "residual");
            p.residual = mr.data;
            p.ldr = mr.ld;
        }
    }
    p.key = longs(a[3], 2, device, "key");
    const int64_t site = whole(a[4]);
    if (site < 0 || site > UINT32_MAX) refuse("site", "in [0, 2^32)");
    p.site = static_cast<uint32_t>(site);
    p.p = number(a[5]);
    p.device = static_cast<int32_t>(device);
    return tl_dropout(&p, address(a[6]));
}

// No C++ exception leaves the module.
template <int (*F)(PyObject* const*), Py_ssize_t N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", N, n);
        return nullptr;
    }
    try {
        return PyLong_FromLong(F(args));
    } catch (const Error&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

template <int (*F)(PyObject* const*), Py_ssize_t N> PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&call<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<token_logprob, 7>("token_logprob"), method<policy_loss, 18>("policy_loss"),
                         method<preference_loss, 17>("preference_loss"), method<distill_loss, 16>("distill_loss"),
                         method<token_stats, 11>("token_stats"), method<token_grad, 11>("token_grad"),
                         method<dropout, 8>("dropout"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_loss_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__loss_bind() { return PyModule_Create(&module); }
