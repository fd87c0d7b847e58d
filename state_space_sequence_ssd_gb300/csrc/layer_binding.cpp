// layer_binding.cpp -- the Python side of the layer operators (ssd_conv_*, ssd_selective_*, ssd_layer_norm_*, ssd_gated_*,
// ssd_group_norm_*, ssd_rotary_*): checks of tensors, allocation of outputs, and the call of the C entry.  layer.py holds the public functions with their
// documentation; what is here was Python there, and took 22 us of a call that launches one small kernel (one token of
// 256 sequences: 4.7 us on the device).  Nothing is computed here.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>
#include <vector>

#include "ssd.h"

namespace {

using at::Tensor;

// A Python exception that is already set.
struct Raised {};

// A reference that is given up at the end of the scope.
struct Held {
    PyObject* o = nullptr;
    Held() = default;
    Held(const Held&) = delete;
    ~Held() { Py_XDECREF(o); }
};

[[noreturn]] void refuse(PyObject* kind, const std::string& text) {
    PyErr_SetString(kind, text.c_str());
    throw Raised();
}

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

const char* type_name(at::ScalarType t) {
    return t == at::kFloat ? "torch.float32" : t == at::kInt ? "torch.int32" : t == at::kHalf ? "torch.float16"
           : t == at::kBFloat16 ? "torch.bfloat16" : c10::toString(t);
}

// The tensor behind an argument; null for None.
const Tensor* optional(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(PyExc_ValueError, std::string(name) + " must be a tensor, got " + Py_TYPE(o)->tp_name);
    return &THPVariable_Unpack(o);
}
const Tensor& tensor(PyObject* o, const char* name) {
    const Tensor* t = optional(o, name);
    if (t == nullptr) refuse(PyExc_ValueError, std::string(name) + " is required");
    return *t;
}

// What the tensor that leads a call fixes for the others.
struct Lead {
    int code;
    at::ScalarType type;
    c10::Device device;
    cudaStream_t stream;
};

// The C entries take sizes as int.
int size_int(int64_t n) {
    if (n > 2147483647) refuse(PyExc_ValueError, "a dimension of " + std::to_string(n) + " is more than a call takes");
    return (int)n;
}

Lead lead(const Tensor& t, const char* name, int ndim) {
    const auto type = t.scalar_type();
    const int code = type == at::kBFloat16 ? SSD_BF16 : type == at::kHalf ? SSD_F16 : type == at::kFloat ? SSD_F32 : -1;
    if (code < 0)
        refuse(PyExc_TypeError, std::string(name) + " must be bfloat16, float16 or float32, got " + type_name(type));
    if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor (no CPU path exists)");
    if (ndim ? t.dim() != ndim : t.dim() < 1)
        refuse(PyExc_ValueError, std::string(name) + " must have " + (ndim ? std::to_string(ndim) + " dims" : "at least 1 dim") +
                                     ", got " + shape_text(t.sizes()));
    if (t.device().index() != c10::cuda::current_device())
        refuse(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", which is not the current device");
    return {code, type, t.device(), c10::cuda::getCurrentCUDAStream(t.device().index()).stream()};
}

void check(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, const Lead& l) {
    if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor (no CPU path exists)");
    if (t.scalar_type() != type)
        refuse(PyExc_TypeError, std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
    if (t.sizes() != shape)
        refuse(PyExc_ValueError, std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
    if (t.device() != l.device) refuse(PyExc_ValueError, std::string(name) + " must be on " + l.device.str() + ", got " + t.device().str());
}

// The address of a dense tensor of this type and shape.
template <typename T = void>
T* dense(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, const Lead& l) {
    check(t, name, type, shape, l);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
    return static_cast<T*>(t.data_ptr());
}
template <typename T = void>
T* dense(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, const Lead& l) {
    const Tensor* t = optional(o, name);
    return t == nullptr ? nullptr : dense<T>(*t, name, type, shape, l);
}

// The stride of dimension d before the last `inner`, which have to be dense; 0 for a dimension of one.
void need_dense_end(const Tensor& t, const char* name, int inner) {
    int64_t need = 1;
    for (int d = (int)t.dim() - 1; d >= (int)t.dim() - inner; --d) {
        if (t.size(d) != 1 && t.stride(d) != need)
            refuse(PyExc_ValueError, "the last " + std::to_string(inner) + " dimension(s) of " + name +
                                         " must be dense, got strides " + shape_text(t.strides()));
        need *= t.size(d);
    }
}
long long stride(const Tensor& t, int d) { return t.size(d) == 1 ? 0 : t.stride(d); }

Tensor empty(at::IntArrayRef shape, at::ScalarType type, const Lead& l) {
    return Tensor(at::detail::empty_cuda(shape, type, l.device, std::nullopt));
}

PyObject* g_fail = nullptr;  // called with the entry's name and its status

void done(const char* entry, int status) {
    if (status == SSD_OK) return;
    PyObject* r = PyObject_CallFunction(g_fail, "si", entry, status);
    Py_XDECREF(r);
    if (r != nullptr) PyErr_SetString(PyExc_RuntimeError, entry);
    throw Raised();
}

bool truth(PyObject* o) {
    const int r = PyObject_IsTrue(o);
    if (r < 0) throw Raised();
    return r != 0;
}

// One to three positive sizes that add up to `channels`.
std::vector<int64_t> sizes_of(PyObject* o, int64_t channels) {
    if (o == Py_None) return {channels};
    std::vector<int64_t> v;
    PyObject* seq = PySequence_Fast(o, "splits must be a sequence of sizes");
    if (seq == nullptr) throw Raised();
    bool ok = PySequence_Fast_GET_SIZE(seq) >= 1 && PySequence_Fast_GET_SIZE(seq) <= 3;
    int64_t sum = 0;
    for (Py_ssize_t i = 0; ok && i < PySequence_Fast_GET_SIZE(seq); ++i) {
        v.push_back(PyLong_AsLongLong(PySequence_Fast_GET_ITEM(seq, i)));
        ok = !PyErr_Occurred() && v.back() >= 1;
        sum += v.back();
    }
    Py_DECREF(seq);
    if (PyErr_Occurred()) throw Raised();
    if (!ok || sum != channels)
        refuse(PyExc_ValueError, "splits must be one to three positive sizes that add up to " + std::to_string(channels));
    return v;
}

struct Outputs {
    Tensor t[3];
    void* p[3] = {nullptr, nullptr, nullptr};
    int n[3] = {0, 0, 0};
    size_t count;
};
Outputs outputs(std::vector<int64_t> shape, const std::vector<int64_t>& parts, const Lead& l) {
    Outputs o;
    o.count = parts.size();
    shape.push_back(0);
    for (size_t i = 0; i < parts.size(); ++i) {
        shape.back() = parts[i];
        o.t[i] = empty(shape, l.type, l);
        o.p[i] = o.t[i].data_ptr();
        o.n[i] = (int)parts[i];
    }
    return o;
}

PyObject* wrap(const Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    PyObject* o = THPVariable_Wrap(t);
    if (o == nullptr) throw Raised();
    return o;
}
PyObject* tuple_of(std::initializer_list<PyObject*> items) {
    PyObject* t = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    for (PyObject* o : items) PyTuple_SET_ITEM(t, i++, o);
    return t;
}
PyObject* pieces(const Outputs& o, bool single) {
    if (single) return wrap(o.t[0]);
    PyObject* t = PyTuple_New((Py_ssize_t)o.count);
    for (size_t i = 0; i < o.count; ++i) PyTuple_SET_ITEM(t, (Py_ssize_t)i, wrap(o.t[i]));
    return t;
}
PyObject* dict_of(std::initializer_list<std::pair<const char*, const Tensor*>> items) {
    PyObject* d = PyDict_New();
    for (auto& it : items) {
        PyObject* o = wrap(*it.second);
        PyDict_SetItemString(d, it.first, o);
        Py_DECREF(o);
    }
    return d;
}

// Taps and biases of the convolution.
struct Taps {
    int64_t width;
    float *weight, *bias;
};
Taps taps(PyObject* weight, PyObject* bias, int64_t channels, const Lead& l) {
    const Tensor& w = tensor(weight, "weight");
    if (w.dim() != 2) refuse(PyExc_ValueError, "weight must be a (channels, width) tensor");
    const int64_t W = w.size(1);
    return {W, dense<float>(w, "weight", at::kFloat, {channels, W}, l), dense<float>(bias, "bias", at::kFloat, {channels}, l)};
}

// x, weight, bias, init_state, lengths, silu, splits, want_final
PyObject* conv_forward(PyObject* const* a) {
    const Tensor& x = tensor(a[0], "x");
    const Lead l = lead(x, "x", 3);
    const int64_t b = x.size(0), L = x.size(1), ch = x.size(2);
    const Taps w = taps(a[1], a[2], ch, l);
    void* init = dense(a[3], "init_state", l.type, {b, w.width - 1, ch}, l);
    int* lengths = dense<int>(a[4], "lengths", at::kInt, {b}, l);
    need_dense_end(x, "x", 1);
    const auto parts = sizes_of(a[6], ch);
    Outputs y = outputs({b, L}, parts, l);
    Tensor final_state;
    if (truth(a[7])) final_state = empty({b, w.width - 1, ch}, l.type, l);
    done("ssd_conv_forward",
         ssd_conv_forward(l.code, x.data_ptr(), stride(x, 0), stride(x, 1), w.weight, w.bias, init, lengths, size_int(b), size_int(L), size_int(ch),
                          size_int(w.width), truth(a[5]), y.p[0], y.n[0], y.p[1], y.n[1], y.p[2], y.n[2],
                          final_state.defined() ? final_state.data_ptr() : nullptr, l.stream));
    return tuple_of({pieces(y, a[6] == Py_None), wrap(final_state)});
}

// x, weight, bias, dy, init_state, lengths, silu, dfinal, dx, want_dinit
PyObject* conv_backward(PyObject* const* a) {
    const Tensor& x = tensor(a[0], "x");
    const Lead l = lead(x, "x", 3);
    const int64_t b = x.size(0), L = x.size(1), ch = x.size(2);
    const Taps w = taps(a[1], a[2], ch, l);
    Held seq;  // until the call is made: it may be all that holds the pieces (of an iterator that makes them)
    const void *dy[3] = {nullptr, nullptr, nullptr};
    int n[3] = {0, 0, 0}, f32[3] = {0, 0, 0};
    auto piece = [&](PyObject* o, int i) {
        const std::string name = "dy[" + std::to_string(i) + "]";
        const Tensor& t = tensor(o, name.c_str());
        if (t.dim() != 3) refuse(PyExc_ValueError, name + " must have 3 dims, got " + shape_text(t.sizes()));
        f32[i] = t.scalar_type() == at::kFloat;
        dy[i] = dense(t, name.c_str(), f32[i] ? at::kFloat : l.type, {b, L, t.size(2)}, l);
        n[i] = (int)t.size(2);
    };
    if (THPVariable_Check(a[3])) {
        piece(a[3], 0);
    } else {
        seq.o = PySequence_Fast(a[3], "dy must be a tensor or a sequence of one to three");
        if (seq.o == nullptr) throw Raised();
        const Py_ssize_t count = PySequence_Fast_GET_SIZE(seq.o);
        if (count < 1 || count > 3) refuse(PyExc_ValueError, "dy must be a tensor or a sequence of one to three");
        for (Py_ssize_t i = 0; i < count; ++i) piece(PySequence_Fast_GET_ITEM(seq.o, i), (int)i);
    }
    if ((int64_t)n[0] + n[1] + n[2] != ch) refuse(PyExc_ValueError, "the pieces of dy must add up to x's " + std::to_string(ch) + " channels");
    void* init = dense(a[4], "init_state", l.type, {b, w.width - 1, ch}, l);
    int* lengths = dense<int>(a[5], "lengths", at::kInt, {b}, l);
    void* dfinal = dense(a[7], "dfinal", l.type, {b, w.width - 1, ch}, l);
    need_dense_end(x, "x", 1);
    const Tensor* given = optional(a[8], "dx");
    if (given != nullptr) {
        check(*given, "dx", l.type, {b, L, ch}, l);
        need_dense_end(*given, "dx", 1);
    }
    Tensor dx = given != nullptr ? *given : empty({b, L, ch}, l.type, l);
    Tensor dweight = empty({ch, w.width}, at::kFloat, l), dbias, dinit;
    if (w.bias != nullptr) dbias = empty({ch}, at::kFloat, l);
    if (truth(a[9])) dinit = empty({b, w.width - 1, ch}, l.type, l);
    done("ssd_conv_backward",
         ssd_conv_backward(l.code, x.data_ptr(), stride(x, 0), stride(x, 1), w.weight, w.bias, init, lengths, size_int(b), size_int(L), size_int(ch),
                           size_int(w.width), truth(a[6]), dy[0], n[0], f32[0], dy[1], n[1], f32[1], dy[2], n[2], f32[2], dfinal,
                           dx.data_ptr(), stride(dx, 0), stride(dx, 1), dweight.data_ptr<float>(),
                           dbias.defined() ? dbias.data_ptr<float>() : nullptr, dinit.defined() ? dinit.data_ptr() : nullptr,
                           l.stream));
    return dict_of({{"dx", &dx}, {"dweight", &dweight}, {"dbias", &dbias}, {"dinit", &dinit}});
}

// A pool of states and the rows' slots in it.
struct Pool {
    void* state;
    int* slots;
    int64_t n;
};
Pool pool(PyObject* state, PyObject* slots, int64_t batch, int64_t d1, int64_t d2, at::ScalarType type, const Lead& l) {
    const Tensor& s = tensor(state, "state");
    if (s.dim() != 3)
        refuse(PyExc_ValueError, "state must be a (slots, " + std::to_string(d1) + ", " + std::to_string(d2) + ") tensor");
    const int64_t n = s.size(0);
    int* at_slots = dense<int>(slots, "slots", at::kInt, {batch}, l);
    if (at_slots == nullptr && n < batch)
        refuse(PyExc_ValueError, "state holds " + std::to_string(n) + " rows for a batch of " + std::to_string(batch));
    return {dense(s, "state", type, {n, d1, d2}, l), at_slots, n};
}

// x, weight, bias, state, slots, silu, splits
PyObject* conv_step(PyObject* const* a) {
    const Tensor& x = tensor(a[0], "x");
    const Lead l = lead(x, "x", 2);
    const int64_t b = x.size(0), ch = x.size(1);
    const Taps w = taps(a[1], a[2], ch, l);
    const Pool p = pool(a[3], a[4], b, w.width - 1, ch, l.type, l);
    need_dense_end(x, "x", 1);
    Outputs y = outputs({b}, sizes_of(a[6], ch), l);
    done("ssd_conv_step",
         ssd_conv_step(l.code, x.data_ptr(), stride(x, 0), w.weight, w.bias, p.state, p.slots, size_int(p.n), size_int(b), size_int(ch),
                       size_int(w.width), truth(a[5]), y.p[0], y.n[0], y.p[1], y.n[1], y.p[2], y.n[2], l.stream));
    return pieces(y, a[6] == Py_None);
}

// What the selective scan's entries share, from x, dt, A, B, C, D, dt_bias, dt_softplus, dt_limit, z.
struct Scan {
    Lead l;
    int64_t b, L, ch, G, N;
    const void *x, *dt, *B, *C;
    const float *A, *D;
    ssd_selective_strides st;
    ssd_input_options o;
};
Scan scan(PyObject* ox, PyObject* odt, PyObject* oA, PyObject* oB, PyObject* oC, PyObject* oD, PyObject* obias,
          PyObject* osoft, PyObject* olimit, PyObject* oz, int ndim) {
    const Tensor& x = tensor(ox, "x");
    Scan s{lead(x, "x", ndim)};
    const Lead& l = s.l;
    const Tensor &dt = tensor(odt, "dt"), &A = tensor(oA, "A"), &B = tensor(oB, "B"), &C = tensor(oC, "C");
    const Tensor* z = optional(oz, "z");
    const bool tokens = ndim == 3;
    s.b = x.size(0);
    s.L = tokens ? x.size(1) : 1;
    s.ch = x.size(ndim - 1);
    if (B.dim() != ndim + 1)
        refuse(PyExc_ValueError, "B must be a tensor with " + std::to_string(ndim + 1) + " dims (..., ngroups, dstate)");
    s.G = B.size(ndim - 1);
    s.N = B.size(ndim);
    if (s.G < 1 || s.ch % s.G != 0)
        refuse(PyExc_ValueError, "ngroups (" + std::to_string(s.G) + ") must divide channels (" + std::to_string(s.ch) + ")");
    const std::vector<int64_t> bc = tokens ? std::vector<int64_t>{s.b, s.L, s.G, s.N} : std::vector<int64_t>{s.b, s.G, s.N};
    check(dt, "dt", l.type, x.sizes(), l);
    check(B, "B", l.type, bc, l);
    check(C, "C", l.type, bc, l);
    need_dense_end(x, "x", 1);
    need_dense_end(dt, "dt", 1);
    need_dense_end(B, "B", 2);
    need_dense_end(C, "C", 2);
    if (z != nullptr) {
        check(*z, "z", l.type, x.sizes(), l);
        need_dense_end(*z, "z", 1);
    }
    auto token = [&](const Tensor& t) { return tokens ? stride(t, 1) : 0; };
    s.st = {stride(x, 0), token(x), stride(dt, 0), token(dt), z ? stride(*z, 0) : 0, z ? token(*z) : 0,
            stride(B, 0), token(B), stride(C, 0), token(C)};
    s.x = x.data_ptr();
    s.dt = dt.data_ptr();
    s.B = B.data_ptr();
    s.C = C.data_ptr();
    s.A = dense<float>(A, "A", at::kFloat, {s.ch, s.N}, l);
    s.D = dense<float>(oD, "D", at::kFloat, {s.ch}, l);
    s.o = {};
    s.o.dt_bias = dense<float>(obias, "dt_bias", at::kFloat, {s.ch}, l);
    s.o.dt_softplus = truth(osoft);
    s.o.z = z ? z->data_ptr() : nullptr;
    if (olimit != Py_None) {
        PyObject* seq = PySequence_Fast(olimit, "dt_limit must be a pair");
        if (seq == nullptr) throw Raised();
        const bool two = PySequence_Fast_GET_SIZE(seq) == 2;
        if (two) {
            s.o.dt_limit = 1;
            s.o.dt_min = (float)PyFloat_AsDouble(PySequence_Fast_GET_ITEM(seq, 0));
            s.o.dt_max = (float)PyFloat_AsDouble(PySequence_Fast_GET_ITEM(seq, 1));
        }
        Py_DECREF(seq);
        if (PyErr_Occurred()) throw Raised();
        if (!two) refuse(PyExc_ValueError, "dt_limit must be a pair");
    }
    return s;
}

// x, dt, A, B, C, D, init_state, lengths, dt_bias, dt_softplus, dt_limit, z, want_final
PyObject* selective_forward(PyObject* const* a) {
    const Scan s = scan(a[0], a[1], a[2], a[3], a[4], a[5], a[8], a[9], a[10], a[11], 3);
    const float* init = dense<float>(a[6], "init_state", at::kFloat, {s.b, s.ch, s.N}, s.l);
    const int* lengths = dense<int>(a[7], "lengths", at::kInt, {s.b}, s.l);
    Tensor y = empty({s.b, s.L, s.ch}, s.l.type, s.l), final_state;
    if (truth(a[12])) final_state = empty({s.b, s.ch, s.N}, at::kFloat, s.l);
    done("ssd_selective_forward",
         ssd_selective_forward(s.l.code, s.x, s.dt, s.A, s.B, s.C, s.D, init, lengths, &s.st, size_int(s.b), size_int(s.L), size_int(s.ch), size_int(s.G),
                               size_int(s.N), &s.o, y.data_ptr(), final_state.defined() ? final_state.data_ptr<float>() : nullptr,
                               s.l.stream));
    return tuple_of({wrap(y), wrap(final_state)});
}

// x, dt, A, B, C, D, dy, init_state, lengths, dt_bias, dt_softplus, dt_limit, z, dfinal, want_dinit
PyObject* selective_backward(PyObject* const* a) {
    const Scan s = scan(a[0], a[1], a[2], a[3], a[4], a[5], a[9], a[10], a[11], a[12], 3);
    const Lead& l = s.l;
    const void* dy = dense(tensor(a[6], "dy"), "dy", l.type, {s.b, s.L, s.ch}, l);
    const float* init = dense<float>(a[7], "init_state", at::kFloat, {s.b, s.ch, s.N}, l);
    const int* lengths = dense<int>(a[8], "lengths", at::kInt, {s.b}, l);
    const float* dfinal = dense<float>(a[13], "dfinal", at::kFloat, {s.b, s.ch, s.N}, l);
    Tensor dx = empty({s.b, s.L, s.ch}, l.type, l), ddt = empty({s.b, s.L, s.ch}, l.type, l), dA = empty({s.ch, s.N}, at::kFloat, l),
           dB = empty({s.b, s.L, s.G, s.N}, at::kFloat, l), dC = empty({s.b, s.L, s.G, s.N}, at::kFloat, l), dD, dbias, dinit, dz;
    if (s.D != nullptr) dD = empty({s.ch}, at::kFloat, l);
    if (s.o.dt_bias != nullptr) dbias = empty({s.ch}, at::kFloat, l);
    if (truth(a[14])) dinit = empty({s.b, s.ch, s.N}, at::kFloat, l);
    if (s.o.z != nullptr) dz = empty({s.b, s.L, s.ch}, l.type, l);
    auto p = [](const Tensor& t) { return t.defined() ? t.data_ptr<float>() : nullptr; };
    done("ssd_selective_backward",
         ssd_selective_backward(l.code, s.x, s.dt, s.A, s.B, s.C, s.D, init, lengths, &s.st, size_int(s.b), size_int(s.L), size_int(s.ch), size_int(s.G),
                                size_int(s.N), &s.o, dy, dfinal, dx.data_ptr(), ddt.data_ptr(), p(dA), p(dB), p(dC), p(dD),
                                dz.defined() ? dz.data_ptr() : nullptr, p(dbias), p(dinit), l.stream));
    if (dz.defined())
        return dict_of({{"dx", &dx}, {"ddt", &ddt}, {"dA", &dA}, {"dB", &dB}, {"dC", &dC}, {"dD", &dD}, {"ddt_bias", &dbias},
                        {"dinit", &dinit}, {"dz", &dz}});
    return dict_of({{"dx", &dx}, {"ddt", &ddt}, {"dA", &dA}, {"dB", &dB}, {"dC", &dC}, {"dD", &dD}, {"ddt_bias", &dbias}, {"dinit", &dinit}});
}

// x, dt, A, B, C, D, state, slots, dt_bias, dt_softplus, dt_limit, z
PyObject* selective_step(PyObject* const* a) {
    const Scan s = scan(a[0], a[1], a[2], a[3], a[4], a[5], a[8], a[9], a[10], a[11], 2);
    const Pool p = pool(a[6], a[7], s.b, s.ch, s.N, at::kFloat, s.l);
    Tensor y = empty({s.b, s.ch}, s.l.type, s.l);
    done("ssd_selective_step",
         ssd_selective_step(s.l.code, s.x, s.dt, s.A, s.B, s.C, s.D, static_cast<float*>(p.state), p.slots, size_int(p.n), &s.st, size_int(s.b),
                            size_int(s.ch), size_int(s.G), size_int(s.N), &s.o, y.data_ptr(), s.l.stream));
    return wrap(y);
}

// What the gated recurrence's entries share, from x, r, i, A.
struct Gated {
    Lead l;
    int64_t b, L, ch;
    const void *x, *r, *i;
    const float* A;
    ssd_gated_strides st;
};
Gated gated(PyObject* ox, PyObject* orr, PyObject* oi, PyObject* oA, int ndim) {
    const Tensor& x = tensor(ox, "x");
    Gated s{lead(x, "x", ndim)};
    const Tensor &r = tensor(orr, "r"), &i = tensor(oi, "i"), &A = tensor(oA, "A");
    const bool tokens = ndim == 3;
    s.b = x.size(0);
    s.L = tokens ? x.size(1) : 1;
    s.ch = x.size(ndim - 1);
    check(r, "r", s.l.type, x.sizes(), s.l);
    check(i, "i", s.l.type, x.sizes(), s.l);
    need_dense_end(x, "x", 1);
    need_dense_end(r, "r", 1);
    need_dense_end(i, "i", 1);
    auto token = [&](const Tensor& t) { return tokens ? stride(t, 1) : 0; };
    s.st = {stride(x, 0), token(x), stride(r, 0), token(r), stride(i, 0), token(i)};
    s.x = x.data_ptr();
    s.r = r.data_ptr();
    s.i = i.data_ptr();
    s.A = dense<float>(A, "A", at::kFloat, {s.ch}, s.l);
    return s;
}
float* floats(const Tensor& t) { return t.defined() ? t.data_ptr<float>() : nullptr; }
int64_t gated_spans(int64_t L) { return (L + SSD_GATED_SPAN - 1) / SSD_GATED_SPAN; }

// x, r, i, A, init_state, lengths, want_final, want_states
PyObject* gated_forward(PyObject* const* a) {
    const Gated s = gated(a[0], a[1], a[2], a[3], 3);
    const float* init = dense<float>(a[4], "init_state", at::kFloat, {s.b, s.ch}, s.l);
    const int* lengths = dense<int>(a[5], "lengths", at::kInt, {s.b}, s.l);
    Tensor y = empty({s.b, s.L, s.ch}, s.l.type, s.l), final_state, states;
    if (truth(a[6])) final_state = empty({s.b, s.ch}, at::kFloat, s.l);
    if (truth(a[7])) states = empty({s.b, gated_spans(s.L), s.ch}, at::kFloat, s.l);
    done("ssd_gated_forward", ssd_gated_forward(s.l.code, s.x, s.r, s.i, s.A, init, lengths, &s.st, size_int(s.b), size_int(s.L), size_int(s.ch),
                                                y.data_ptr(), floats(final_state), floats(states), s.l.stream));
    return tuple_of({wrap(y), wrap(final_state), wrap(states)});
}

// x, r, i, A, dy, init_state, lengths, states, dfinal, want_dinit
PyObject* gated_backward(PyObject* const* a) {
    const Gated s = gated(a[0], a[1], a[2], a[3], 3);
    const Lead& l = s.l;
    const void* dy = dense(tensor(a[4], "dy"), "dy", l.type, {s.b, s.L, s.ch}, l);
    const float* init = dense<float>(a[5], "init_state", at::kFloat, {s.b, s.ch}, l);
    const int* lengths = dense<int>(a[6], "lengths", at::kInt, {s.b}, l);
    const float* states = dense<float>(a[7], "states", at::kFloat, {s.b, gated_spans(s.L), s.ch}, l);
    const float* dfinal = dense<float>(a[8], "dfinal", at::kFloat, {s.b, s.ch}, l);
    Tensor dx = empty({s.b, s.L, s.ch}, l.type, l), dr = empty({s.b, s.L, s.ch}, l.type, l), di = empty({s.b, s.L, s.ch}, l.type, l),
           dA = empty({s.ch}, at::kFloat, l), dinit;
    if (truth(a[9])) dinit = empty({s.b, s.ch}, at::kFloat, l);
    done("ssd_gated_backward", ssd_gated_backward(l.code, s.x, s.r, s.i, s.A, init, lengths, &s.st, size_int(s.b), size_int(s.L), size_int(s.ch), states, dy,
                                                  dfinal, dx.data_ptr(), dr.data_ptr(), di.data_ptr(), floats(dA), floats(dinit), l.stream));
    return dict_of({{"dx", &dx}, {"dr", &dr}, {"di", &di}, {"dA", &dA}, {"dinit", &dinit}});
}

// x, r, i, A, state, slots
PyObject* gated_step(PyObject* const* a) {
    const Gated s = gated(a[0], a[1], a[2], a[3], 2);
    const Tensor& state = tensor(a[4], "state");
    if (state.dim() != 2) refuse(PyExc_ValueError, "state must be a (slots, " + std::to_string(s.ch) + ") tensor");
    const int64_t n = state.size(0);
    const int* slots = dense<int>(a[5], "slots", at::kInt, {s.b}, s.l);
    if (slots == nullptr && n < s.b)
        refuse(PyExc_ValueError, "state holds " + std::to_string(n) + " rows for a batch of " + std::to_string(s.b));
    float* p = dense<float>(state, "state", at::kFloat, {n, s.ch}, s.l);
    Tensor y = empty({s.b, s.ch}, s.l.type, s.l);
    done("ssd_gated_step", ssd_gated_step(s.l.code, s.x, s.r, s.i, s.A, p, slots, size_int(n), &s.st, size_int(s.b), size_int(s.ch), y.data_ptr(), s.l.stream));
    return wrap(y);
}

// Rows of the last dimension whose leading dimensions run through one stride.
struct Flat {
    long long step, rows;
};
Flat flat(const Tensor& t, const char* name) {
    need_dense_end(t, name, 1);
    Flat f = {0, 1};
    for (int d = (int)t.dim() - 2; d >= 0; --d) {
        if (t.size(d) == 1) continue;
        if (f.rows == 1) f.step = t.stride(d);
        else if (t.stride(d) != f.step * f.rows)
            refuse(PyExc_ValueError, std::string("the rows of ") + name + " must be evenly spaced, got shape " +
                                         shape_text(t.sizes()) + ", strides " + shape_text(t.strides()));
        f.rows *= t.size(d);
    }
    if (f.rows == 1) f.step = t.size(-1);
    return f;
}

// x, weight, bias, eps
PyObject* norm_forward(PyObject* const* a) {
    const Tensor& x = tensor(a[0], "x");
    const Lead l = lead(x, "x", 0);
    const int64_t width = x.size(-1);
    const float *w = dense<float>(a[1], "weight", at::kFloat, {width}, l), *bias = dense<float>(a[2], "bias", at::kFloat, {width}, l);
    const double eps = PyFloat_AsDouble(a[3]);
    if (PyErr_Occurred()) throw Raised();
    const Flat f = flat(x, "x");
    const auto rows = x.sizes().slice(0, x.dim() - 1);
    Tensor y = empty(x.sizes(), l.type, l), mean = empty(rows, at::kFloat, l), rstd = empty(rows, at::kFloat, l);
    done("ssd_layer_norm_forward",
         ssd_layer_norm_forward(l.code, x.data_ptr(), f.step, w, bias, (float)eps, f.rows, size_int(width), y.data_ptr(),
                                mean.data_ptr<float>(), rstd.data_ptr<float>(), l.stream));
    return tuple_of({wrap(y), wrap(mean), wrap(rstd)});
}

// x, weight, mean, rstd, dy, want_dbias
PyObject* norm_backward(PyObject* const* a) {
    const Tensor& x = tensor(a[0], "x");
    const Lead l = lead(x, "x", 0);
    const int64_t width = x.size(-1);
    const auto rows = x.sizes().slice(0, x.dim() - 1);
    const float* w = dense<float>(a[1], "weight", at::kFloat, {width}, l);
    const float *mean = dense<float>(tensor(a[2], "mean"), "mean", at::kFloat, rows, l),
                *rstd = dense<float>(tensor(a[3], "rstd"), "rstd", at::kFloat, rows, l);
    const Tensor& dy = tensor(a[4], "dy");
    check(dy, "dy", l.type, x.sizes(), l);
    const Flat f = flat(x, "x"), g = flat(dy, "dy");
    Tensor dx = empty(x.sizes(), l.type, l), dweight, dbias;
    if (w != nullptr) dweight = empty({width}, at::kFloat, l);
    if (truth(a[5])) dbias = empty({width}, at::kFloat, l);
    done("ssd_layer_norm_backward",
         ssd_layer_norm_backward(l.code, x.data_ptr(), f.step, w, mean, rstd, dy.data_ptr(), g.step, f.rows, size_int(width),
                                 dx.data_ptr(), dweight.defined() ? dweight.data_ptr<float>() : nullptr,
                                 dbias.defined() ? dbias.data_ptr<float>() : nullptr, l.stream));
    return dict_of({{"dx", &dx}, {"dweight", &dweight}, {"dbias", &dbias}});
}

// What the grouped norm's entries share, from x, groups, weight, bias, z, gate_first, silu.
struct GroupNorm {
    Lead l;
    int64_t width, groups;
    Flat x, z;
    const void *px, *pz;
    const float *weight, *bias;
    int gate;
    std::vector<int64_t> stats;  // shape of mean and rstd
};
GroupNorm group_norm(PyObject* ox, PyObject* ogroups, PyObject* oweight, PyObject* obias, PyObject* oz, PyObject* ofirst, PyObject* osilu) {
    const Tensor& x = tensor(ox, "x");
    GroupNorm s{lead(x, "x", 0)};
    s.width = x.size(-1);
    s.groups = PyLong_AsLongLong(ogroups);
    if (PyErr_Occurred()) throw Raised();
    if (s.groups < 1 || s.width % s.groups != 0)
        refuse(PyExc_ValueError, "groups (" + std::to_string(s.groups) + ") must divide x's " + std::to_string(s.width) + " channels");
    s.weight = dense<float>(oweight, "weight", at::kFloat, {s.width}, s.l);
    s.bias = dense<float>(obias, "bias", at::kFloat, {s.width}, s.l);
    const Tensor* z = optional(oz, "z");
    const bool first = truth(ofirst), silu = truth(osilu);
    if (silu && z != nullptr) refuse(PyExc_ValueError, "silu and a gate z exclude one another");
    if (first && z == nullptr) refuse(PyExc_ValueError, "gate_first needs a gate z");
    s.gate = z == nullptr ? (silu ? SSD_GATE_SILU : SSD_GATE_NONE) : first ? SSD_GATE_BEFORE : SSD_GATE_AFTER;
    s.x = flat(x, "x");
    s.z = {0, 0};
    s.px = x.data_ptr();
    s.pz = nullptr;
    if (z != nullptr) {
        check(*z, "z", s.l.type, x.sizes(), s.l);
        s.z = flat(*z, "z");
        s.pz = z->data_ptr();
    }
    s.stats = x.sizes().slice(0, x.dim() - 1).vec();
    s.stats.push_back(s.groups);
    return s;
}

// x, groups, weight, bias, z, gate_first, silu, rms, eps
PyObject* group_norm_forward(PyObject* const* a) {
    const GroupNorm s = group_norm(a[0], a[1], a[2], a[3], a[4], a[5], a[6]);
    const bool rms = truth(a[7]);
    const double eps = PyFloat_AsDouble(a[8]);
    if (PyErr_Occurred()) throw Raised();
    Tensor y = empty(tensor(a[0], "x").sizes(), s.l.type, s.l), mean, rstd = empty(s.stats, at::kFloat, s.l);
    if (!rms) mean = empty(s.stats, at::kFloat, s.l);
    done("ssd_group_norm_forward",
         ssd_group_norm_forward(s.l.code, s.px, s.x.step, s.pz, s.z.step, s.weight, s.bias, (float)eps, s.gate, rms, s.x.rows, size_int(s.width),
                                size_int(s.groups), y.data_ptr(), floats(mean), floats(rstd), s.l.stream));
    return tuple_of({wrap(y), wrap(mean), wrap(rstd)});
}

// x, groups, weight, bias, mean, rstd, dy, z, gate_first, silu
PyObject* group_norm_backward(PyObject* const* a) {
    const GroupNorm s = group_norm(a[0], a[1], a[2], a[3], a[7], a[8], a[9]);
    const auto shape = tensor(a[0], "x").sizes();
    const float *mean = dense<float>(a[4], "mean", at::kFloat, s.stats, s.l), *rstd = dense<float>(tensor(a[5], "rstd"), "rstd", at::kFloat, s.stats, s.l);
    const Tensor& dy = tensor(a[6], "dy");
    check(dy, "dy", s.l.type, shape, s.l);
    const Flat g = flat(dy, "dy");
    Tensor dx = empty(shape, s.l.type, s.l), dz, dweight, dbias;
    if (s.pz != nullptr) dz = empty(shape, s.l.type, s.l);
    if (s.weight != nullptr) dweight = empty({s.width}, at::kFloat, s.l);
    if (s.bias != nullptr) dbias = empty({s.width}, at::kFloat, s.l);
    done("ssd_group_norm_backward",
         ssd_group_norm_backward(s.l.code, s.px, s.x.step, s.pz, s.z.step, s.weight, s.bias, s.gate, mean, rstd, dy.data_ptr(), g.step, s.x.rows,
                                 size_int(s.width), size_int(s.groups), dx.data_ptr(), dz.defined() ? dz.data_ptr() : nullptr, floats(dweight), floats(dbias),
                                 s.l.stream));
    if (dz.defined()) return dict_of({{"dx", &dx}, {"dz", &dz}, {"dweight", &dweight}, {"dbias", &dbias}});
    return dict_of({{"dx", &dx}, {"dweight", &dweight}, {"dbias", &dbias}});
}

// B, C, table, positions, lengths, interleaved, scale, inverse, step
PyObject* rotary(PyObject* const* a) {
    const bool step = truth(a[8]);
    const int ndim = step ? 3 : 4;
    const Tensor& B = tensor(a[0], "B");
    const Tensor* C = optional(a[1], "C");
    const Lead l = lead(B, "B", ndim);
    const int64_t b = B.size(0), L = step ? 1 : B.size(1), dim = B.size(ndim - 1), G = B.size(ndim - 2), G2 = C == nullptr ? 0 : C->dim() == ndim ? C->size(ndim - 2) : 0;
    auto shape = [&](int64_t heads) { return step ? std::vector<int64_t>{b, heads, dim} : std::vector<int64_t>{b, L, heads, dim}; };
    need_dense_end(B, "B", 2);
    if (C != nullptr) {
        check(*C, "C", l.type, shape(G2), l);
        need_dense_end(*C, "C", 2);
    }
    const Tensor& table = tensor(a[2], "table");
    if (table.dim() != 1) refuse(PyExc_ValueError, "table must have 1 dim, got " + shape_text(table.sizes()));
    const void* turns = dense(table, "table", at::kLong, {table.size(0)}, l);
    const Tensor* positions = optional(a[3], "positions");
    const bool each = positions != nullptr && positions->dim() == 2;
    const int* at = nullptr;
    if (positions != nullptr) at = dense<int>(*positions, "positions", at::kInt, each ? std::vector<int64_t>{b, L} : std::vector<int64_t>{b}, l);
    const int* lengths = dense<int>(a[4], "lengths", at::kInt, {b}, l);
    const double scale = PyFloat_AsDouble(a[6]);
    if (PyErr_Occurred()) throw Raised();
    const Tensor y = empty(shape(G), l.type, l);
    Tensor y2;
    if (C != nullptr) y2 = empty(shape(G2), l.type, l);
    auto token = [&](const Tensor& t) { return step ? 0 : stride(t, 1); };
    done("ssd_rotary",
         ssd_rotary(l.code, B.data_ptr(), stride(B, 0), token(B), size_int(G), C == nullptr ? nullptr : C->data_ptr(), C == nullptr ? 0 : stride(*C, 0),
                    C == nullptr ? 0 : token(*C), size_int(G2), static_cast<const unsigned long long*>(turns), size_int(2 * table.size(0)), at, each, lengths,
                    (float)scale, truth(a[5]), truth(a[7]), size_int(b), size_int(L), size_int(dim), y.data_ptr(), C == nullptr ? nullptr : y2.data_ptr(),
                    l.stream));
    return C == nullptr ? wrap(y) : tuple_of({wrap(y), wrap(y2)});
}

// For the tests without a GPU: (step, rows) of a tensor's rows, and the strides before its last `inner` dimensions.
PyObject* flat_rows(PyObject* const* a) {
    const Flat f = flat(tensor(a[0], "t"), "t");
    return Py_BuildValue("LL", f.step, f.rows);
}
PyObject* row_strides(PyObject* const* a) {
    const Tensor& t = tensor(a[0], "t");
    const long inner = PyLong_AsLong(a[1]);
    if (PyErr_Occurred()) throw Raised();
    need_dense_end(t, "t", (int)inner);
    PyObject* list = PyList_New(0);
    for (int d = 0; d < t.dim() - inner; ++d) {
        PyObject* v = PyLong_FromLongLong(stride(t, d));
        PyList_Append(list, v);
        Py_DECREF(v);
    }
    return list;
}
PyObject* set_fail(PyObject* const* a) {
    Py_INCREF(a[0]);
    Py_XDECREF(g_fail);
    g_fail = a[0];
    Py_RETURN_NONE;
}

// The Python face of a function of N positional arguments: C++ exceptions become Python ones.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    if (count != N) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}
template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<conv_forward, 8>("conv_forward"),
    method<conv_backward, 10>("conv_backward"),
    method<conv_step, 7>("conv_step"),
    method<selective_forward, 13>("selective_forward"),
    method<selective_backward, 15>("selective_backward"),
    method<selective_step, 12>("selective_step"),
    method<norm_forward, 4>("norm_forward"),
    method<norm_backward, 6>("norm_backward"),
    method<gated_forward, 8>("gated_forward"),
    method<gated_backward, 10>("gated_backward"),
    method<gated_step, 6>("gated_step"),
    method<group_norm_forward, 9>("group_norm_forward"),
    method<group_norm_backward, 10>("group_norm_backward"),
    method<rotary, 9>("rotary"),
    method<flat_rows, 1>("flat_rows"),
    method<row_strides, 2>("row_strides"),
    method<set_fail, 1>("set_fail"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "ssd_layer_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ssd_layer_binding(void) { return PyModule_Create(&g_module); }
