// py_cache.cpp -- Python marshalling of the rotary and 8-bit cache calls
// (module gist_token_chunk_b200._cache): checks of the tensors, outputs, device and
// stream, then the C ABI of libssa, whose addresses bind() takes.  These calls take
// 2 to 15 us on the device and up to 14 tensors; checked in Python and passed
// through ctypes they cost 17 to 30 us of host time.
//
// A function returns its outputs, or the status as an int when the call failed.
// Errors of the arguments raise ValueError or TypeError before anything is enqueued.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <optional>
#include <stdexcept>
#include <string>

#include "../../include/ssa.h"

namespace {

struct Api {
    decltype(&ssa_rope) rope = nullptr;
    decltype(&ssa_cache_append_q8) append = nullptr;
    decltype(&ssa_cache_read_q8) read = nullptr;
    decltype(&ssa_workspace_size_q8) workspace = nullptr;
    decltype(&ssa_decode_q8) decode = nullptr;
} api;

struct Refused : std::runtime_error {  // ValueError
    using std::runtime_error::runtime_error;
};
struct WrongType : std::runtime_error {  // TypeError
    using std::runtime_error::runtime_error;
};

std::string text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

// A call's arguments, in order.
struct Args {
    PyObject* const* a;
    Py_ssize_t n, at = 0;
    Args(PyObject* const* args, Py_ssize_t count, Py_ssize_t want) : a(args), n(count) {
        if (count != want) throw WrongType("wrong number of arguments");
    }
    PyObject* next() { return a[at++]; }
    const at::Tensor& tensor(const char* name) {
        PyObject* o = next();
        if (!THPVariable_Check(o)) throw WrongType(std::string(name) + " must be a tensor");
        return THPVariable_Unpack(o);
    }
    const at::Tensor* maybe(const char* name) {
        if (a[at] == Py_None) {
            ++at;
            return nullptr;
        }
        return &tensor(name);
    }
    long long integer(const char* name) {
        PyObject* o = next();
        const long long v = PyLong_AsLongLong(o);
        if (v == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            throw WrongType(std::string(name) + " must be an integer");
        }
        return v;
    }
    int32_t i32(const char* name) {
        const long long v = integer(name);
        if (v < INT32_MIN || v > INT32_MAX) throw Refused(std::string(name) + " does not fit 32 bits");
        return (int32_t)v;
    }
    double number(const char* name) {
        const double v = PyFloat_AsDouble(next());
        if (v == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            throw WrongType(std::string(name) + " must be a number");
        }
        return v;
    }
};

int32_t dtype_code(const at::Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return SSA_BF16;
    if (t.scalar_type() == at::kFloat) return SSA_FP32;
    throw WrongType("unsupported dtype " + std::string(at::toString(t.scalar_type())));
}

int32_t dim32(int64_t v) {
    if (v > INT32_MAX) throw Refused("a size does not fit 32 bits");
    return (int32_t)v;
}

// The call's device and stream; outputs made while it lives belong to them.
struct Place {
    c10::Device device;
    cudaStream_t raw;
    std::optional<c10::cuda::CUDAGuard> on_device;
    std::optional<c10::cuda::CUDAStreamGuard> on_stream;

    // stream: None (the device's current one) or a raw handle; stream_device: the
    // device a torch stream is on, -1 for a handle.
    Place(const at::Tensor& t, PyObject* stream, int stream_device) : device(t.device()) {
        if (!device.is_cuda()) throw Refused("tensors must be CUDA tensors");
        if (stream == Py_None) {
            on_device.emplace(device);
            raw = c10::cuda::getCurrentCUDAStream(device.index()).stream();
            return;
        }
        if (stream_device >= 0 && stream_device != device.index())
            throw Refused("the stream is on cuda:" + std::to_string(stream_device) + ", the tensors on " +
                          device.str());
        const unsigned long long h = PyLong_AsUnsignedLongLong(stream);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            throw WrongType("stream must be a torch.cuda.Stream or a handle");
        }
        raw = reinterpret_cast<cudaStream_t>(h);
        on_stream.emplace(c10::cuda::getStreamFromExternal(raw, device.index()));
    }
};

// Other Python threads run while this lives: an allocation may wait for the device, and
// a launch for room in its queue. Made once the arguments are unpacked (the caller holds
// the tensors); ended before a Python object is made, or by the exception that refuses.
class NoGil {
    PyThreadState* state_;

public:
    NoGil() : state_(PyEval_SaveThread()) {}
    ~NoGil() { PyEval_RestoreThread(state_); }
    NoGil(const NoGil&) = delete;
};
using Unlocked = std::optional<NoGil>;

template <class T = void>
T* want(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type,
        const c10::Device& device) {
    if (t.sizes() != shape || t.scalar_type() != type)
        throw Refused(std::string(name) + ": " + at::toString(t.scalar_type()) + " " + text(t.sizes()) +
                      ", wanted " + at::toString(type) + " " + text(shape));
    if (t.device() != device)
        throw Refused(std::string(name) + " is on " + t.device().str() + ", not on " + device.str());
    if (!t.is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
    return static_cast<T*>(t.data_ptr());
}

// Codes: one byte an element, as uint8 or float8_e4m3fn.
uint8_t* codes(const at::Tensor& t, const char* name, at::IntArrayRef shape, const c10::Device& device) {
    const bool f8 = t.scalar_type() == at::kFloat8_e4m3fn;
    return want<uint8_t>(t, name, shape, f8 ? at::kFloat8_e4m3fn : at::kByte, device);
}

// Rows [B,H,T,d] of any strides, each contiguous; a dim of one element takes stride 0.
struct Rows {
    void* p = nullptr;
    int64_t strides[3] = {0, 0, 0};
    Rows() = default;
    Rows(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type,
         const c10::Device& device, bool output) {
        if (t.sizes() != shape || t.scalar_type() != type)
            throw Refused(std::string(name) + ": " + at::toString(t.scalar_type()) + " " + text(t.sizes()) +
                          ", wanted " + at::toString(type) + " " + text(shape));
        if (t.device() != device)
            throw Refused(std::string(name) + " is on " + t.device().str() + ", not on " + device.str());
        if (shape[3] > 1 && t.stride(3) != 1)
            throw Refused(std::string(name) + ": the elements of a row must be contiguous");
        for (int i = 0; i < 3; ++i) {
            strides[i] = shape[i] > 1 ? t.stride(i) : 0;
            if (output && shape[i] > 1 && strides[i] == 0)
                throw Refused(std::string(name) + ": rows of an output must not share memory");
        }
        p = t.data_ptr();
    }
};

void four_dims(const at::Tensor& t, const char* name) {
    if (t.dim() != 4) throw Refused(std::string(name) + ": wanted four dims, got " + text(t.sizes()));
}

PyObject* pair(const at::Tensor& a, const at::Tensor* b) {
    PyObject* r = PyTuple_New(2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(a));
    if (b) {
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(*b));
    } else {
        Py_INCREF(Py_None);
        PyTuple_SET_ITEM(r, 1, Py_None);
    }
    return r;
}

// rope(q, k, pos, freqs, layout, scale, inverse, q_out, k_out, stream, stream_device)
PyObject* rope(Args& a) {
    const at::Tensor& q = a.tensor("q");
    const at::Tensor* k = a.maybe("k");
    const at::Tensor& pos = a.tensor("pos");
    const at::Tensor& freqs = a.tensor("freqs");
    const int32_t layout = a.i32("layout");
    const double scale = a.number("scale");
    const bool inverse = a.integer("inverse") != 0;
    const at::Tensor* qo = a.maybe("q_out");
    const at::Tensor* ko = a.maybe("k_out");
    PyObject* stream = a.next();
    Place at(q, stream, a.i32("stream_device"));
    Unlocked gil(std::in_place);
    four_dims(q, "q");
    const int64_t B = q.size(0), Hq = q.size(1), T = q.size(2), d = q.size(3);
    if (k) four_dims(*k, "k");
    const int64_t Hkv = k ? k->size(1) : 1;
    if (freqs.dim() != 1) throw Refused("freqs must be one-dimensional");
    const bool rows = pos.dim() == 2;
    at::Tensor q_new, k_new;
    if (!qo) {
        q_new = at::empty({B, Hq, T, d}, q.options());
        qo = &q_new;
    }
    if (k && !ko) {
        k_new = at::empty({B, Hkv, T, d}, q.options());
        ko = &k_new;
    }
    const ssa_shape shape = {dim32(B), dim32(Hq), dim32(Hkv), dim32(d), 0, dtype_code(q)};
    const auto type = q.scalar_type();
    const int64_t qs[4] = {B, Hq, T, d}, ks[4] = {B, Hkv, T, d};
    const Rows rq(q, "q", qs, type, at.device, false), rqo(*qo, "q_out", qs, type, at.device, true);
    Rows rk, rko;
    if (k) {
        rk = Rows(*k, "k", ks, type, at.device, false);
        rko = Rows(*ko, "k_out", ks, type, at.device, true);
    }
    const int64_t by_row[2] = {B, T};
    const int32_t* p = want<int32_t>(pos, "pos", at::IntArrayRef(by_row, rows ? 2 : 1), at::kInt, at.device);
    const double* f = want<double>(freqs, "freqs", freqs.sizes(), at::kDouble, at.device);
    const ssa_status st =
        api.rope(&shape, dim32(T), rq.p, rq.strides, rqo.p, rqo.strides, rk.p, rk.strides, rko.p, rko.strides,
                 p, rows, f, dim32(2 * freqs.numel()), layout, (float)scale, inverse, at.raw);
    gil.reset();
    if (st != SSA_OK) return PyLong_FromLong(st);
    return pair(*qo, k ? ko : nullptr);
}

// Rows and blocks of a pair of 8-bit cache arrays [B,Hkv,N,d] (or [B,Hkv,M,g,d])
// with scales [B,Hkv,N / R].
struct Cache {
    int64_t N, R;
    uint8_t *k, *v = nullptr;
    float *ks, *vs = nullptr;
    Cache(const at::Tensor& kc, const at::Tensor* vc, const at::Tensor& ksc, const at::Tensor* vsc,
          int64_t B, int64_t Hkv, int64_t d, const c10::Device& device) {
        if (kc.dim() < 4 || kc.size(0) != B || kc.size(1) != Hkv || kc.size(-1) != d)
            throw Refused("k_q8: " + text(kc.sizes()) + ", wanted [" + std::to_string(B) + ", " +
                          std::to_string(Hkv) + ", ..., " + std::to_string(d) + "]");
        const int64_t blocks = ksc.dim() == 3 ? ksc.size(2) : 0;
        N = 1;
        for (int64_t i = 2; i < kc.dim() - 1; ++i) N *= kc.size(i);
        if (blocks < 1 || N % blocks)
            throw Refused(std::to_string(N) + " rows do not divide into " + std::to_string(blocks) + " blocks");
        R = N / blocks;
        const int64_t sc[3] = {B, Hkv, blocks};
        k = codes(kc, "k_q8", kc.sizes(), device);
        ks = want<float>(ksc, "k_scale", sc, at::kFloat, device);
        if (vc) {
            if (!vsc) throw WrongType("v_scale must be a tensor");
            v = codes(*vc, "v_q8", kc.sizes(), device);
            vs = want<float>(*vsc, "v_scale", sc, at::kFloat, device);
        }
    }
};

// append(k_new, v_new, start, k_q8, v_q8, k_scale, v_scale, count, stream, stream_device)
PyObject* append(Args& a) {
    const at::Tensor& k = a.tensor("k_new");
    const at::Tensor* v = a.maybe("v_new");
    const at::Tensor& start = a.tensor("start");
    const at::Tensor& kc = a.tensor("k_q8");
    const at::Tensor* vc = a.maybe("v_q8");
    const at::Tensor& ks = a.tensor("k_scale");
    const at::Tensor* vs = a.maybe("v_scale");
    const at::Tensor* count = a.maybe("count");
    PyObject* stream = a.next();
    Place at(k, stream, a.i32("stream_device"));
    Unlocked gil(std::in_place);
    four_dims(k, "k_new");
    const int64_t B = k.size(0), Hkv = k.size(1), T = k.size(2), d = k.size(3);
    const ssa_shape bare = {dim32(B), dim32(Hkv), dim32(Hkv), dim32(d), 0, dtype_code(k)};
    if (v && !vc) throw WrongType("v_q8 must be a tensor");
    const Cache c(kc, v ? vc : nullptr, ks, v ? vs : nullptr, B, Hkv, d, at.device);
    ssa_shape shape = bare;
    shape.n_max = dim32(c.N);
    const int64_t s[4] = {B, Hkv, T, d};
    const Rows rk(k, "k_new", s, k.scalar_type(), at.device, false);
    Rows rv;
    if (v) rv = Rows(*v, "v_new", s, k.scalar_type(), at.device, false);
    const int32_t* sp = want<int32_t>(start, "start", B, at::kInt, at.device);
    const int32_t* cp = count ? want<int32_t>(*count, "count", B, at::kInt, at.device) : nullptr;
    const ssa_status st = api.append(&shape, dim32(T), dim32(c.R), rk.p, rk.strides, rv.p, rv.strides, sp, cp,
                                     c.k, c.v, c.ks, c.vs, at.raw);
    gil.reset();
    if (st != SSA_OK) return PyLong_FromLong(st);
    Py_RETURN_NONE;
}

// read(k_q8, v_q8, k_scale, v_scale, start, T, count, fp32, k_out, v_out, stream, stream_device)
PyObject* read(Args& a) {
    const at::Tensor& kc = a.tensor("k_q8");
    const at::Tensor* vc = a.maybe("v_q8");
    const at::Tensor& ks = a.tensor("k_scale");
    const at::Tensor* vs = a.maybe("v_scale");
    const at::Tensor& start = a.tensor("start");
    const int32_t T = a.i32("T");
    const at::Tensor* count = a.maybe("count");
    const bool fp32 = a.integer("fp32") != 0;
    const at::Tensor* ko = a.maybe("k_out");
    const at::Tensor* vo = a.maybe("v_out");
    PyObject* stream = a.next();
    Place at(kc, stream, a.i32("stream_device"));
    Unlocked gil(std::in_place);
    if (kc.dim() < 4) throw Refused("k_q8: wanted [B, Hkv, ..., d], got " + text(kc.sizes()));
    const int64_t B = kc.size(0), Hkv = kc.size(1), d = kc.size(-1);
    const Cache c(kc, vc, ks, vs, B, Hkv, d, at.device);
    const auto type = ko ? ko->scalar_type() : fp32 ? at::kFloat : at::kBFloat16;
    const auto options = kc.options().dtype(type);
    if (T < 0) throw Refused("T must be >= 0");
    const int64_t s[4] = {B, Hkv, T, d};
    at::Tensor k_new, v_new;
    auto make = [&] { return count ? at::zeros(s, options) : at::empty(s, options); };
    if (!ko) {
        k_new = make();
        ko = &k_new;
    }
    if (vc && !vo) {
        v_new = make();
        vo = &v_new;
    }
    void* kop = want(*ko, "k_out", s, type, at.device);
    void* vop = vc ? want(*vo, "v_out", s, type, at.device) : nullptr;
    const int32_t* sp = want<int32_t>(start, "start", B, at::kInt, at.device);
    const int32_t* cp = count ? want<int32_t>(*count, "count", B, at::kInt, at.device) : nullptr;
    const ssa_shape shape = {dim32(B), dim32(Hkv), dim32(Hkv), dim32(d), dim32(c.N), dtype_code(*ko)};
    const ssa_status st =
        api.read(&shape, T, dim32(c.R), c.k, c.v, c.ks, c.vs, sp, cp, kop, vop, at.raw);
    gil.reset();
    if (st != SSA_OK) return PyLong_FromLong(st);
    return pair(*ko, vc ? vo : nullptr);
}

// decode(q, k_raw, v_raw, k_gist, v_gist, four scales, seq_lens, C, g, topk, out, sel_idx, ws, stream,
//        stream_device)
PyObject* decode(Args& a) {
    const at::Tensor& q = a.tensor("q");
    const at::Tensor& kr = a.tensor("k_raw");
    const at::Tensor& vr = a.tensor("v_raw");
    const at::Tensor& kg = a.tensor("k_gist");
    const at::Tensor& vg = a.tensor("v_gist");
    const at::Tensor& krs = a.tensor("k_raw_scale");
    const at::Tensor& vrs = a.tensor("v_raw_scale");
    const at::Tensor& kgs = a.tensor("k_gist_scale");
    const at::Tensor& vgs = a.tensor("v_gist_scale");
    const at::Tensor& lens = a.tensor("seq_lens");
    const int32_t C = a.i32("C"), g = a.i32("g"), topk = a.i32("topk");
    const at::Tensor* out = a.maybe("out");
    const at::Tensor* sel = a.maybe("sel_idx");
    const at::Tensor* ws = a.maybe("ws");
    PyObject* stream = a.next();
    Place at(q, stream, a.i32("stream_device"));
    Unlocked gil(std::in_place);
    if (q.dim() != 3) throw Refused("q: wanted [B, Hq, d], got " + text(q.sizes()));
    four_dims(kr, "k_raw");
    const int64_t B = q.size(0), Hq = q.size(1), d = q.size(2), Hkv = kr.size(1), n_max = kr.size(2);
    const ssa_shape shape = {dim32(B), dim32(Hq), dim32(Hkv), dim32(d), dim32(n_max), dtype_code(q)};
    size_t need = 0;
    ssa_status st = api.workspace(&shape, C, g, topk, &need);  // checks the sizes
    if (st != SSA_OK) {
        gil.reset();
        return PyLong_FromLong(st);
    }
    const int64_t M = n_max / C;
    const int64_t s_q[3] = {B, Hq, d}, s_raw[4] = {B, Hkv, n_max, d}, s_gist[5] = {B, Hkv, M, g, d};
    const int64_t s_scale[3] = {B, Hkv, M}, s_sel[3] = {B, Hkv, topk};
    const void* qp = want(q, "q", s_q, q.scalar_type(), at.device);
    const uint8_t* krp = codes(kr, "k_raw", s_raw, at.device);
    const uint8_t* vrp = codes(vr, "v_raw", s_raw, at.device);
    const uint8_t* kgp = codes(kg, "k_gist", s_gist, at.device);
    const uint8_t* vgp = codes(vg, "v_gist", s_gist, at.device);
    const float* krsp = want<float>(krs, "k_raw_scale", s_scale, at::kFloat, at.device);
    const float* vrsp = want<float>(vrs, "v_raw_scale", s_scale, at::kFloat, at.device);
    const float* kgsp = want<float>(kgs, "k_gist_scale", s_scale, at::kFloat, at.device);
    const float* vgsp = want<float>(vgs, "v_gist_scale", s_scale, at::kFloat, at.device);
    const int32_t* lp = want<int32_t>(lens, "seq_lens", B, at::kInt, at.device);
    at::Tensor out_new, sel_new, ws_new;
    if (!out) {
        out_new = at::empty(s_q, q.options().dtype(at::kFloat));
        out = &out_new;
    }
    if (!sel) {
        sel_new = at::empty(s_sel, q.options().dtype(at::kInt));
        sel = &sel_new;
    }
    if (!ws) {
        ws_new = at::empty({(int64_t)need}, q.options().dtype(at::kByte));
        ws = &ws_new;
    }
    float* op = want<float>(*out, "out", s_q, at::kFloat, at.device);
    int32_t* selp = want<int32_t>(*sel, "sel_idx", s_sel, at::kInt, at.device);
    if (ws->device() != at.device) throw Refused("ws is on " + ws->device().str() + ", not on " + at.device.str());
    if (!ws->is_contiguous()) throw Refused("ws must be contiguous");
    st = api.decode(&shape, qp, krp, vrp, kgp, vgp, krsp, vrsp, kgsp, vgsp, lp, C, g, topk, op, selp,
                    ws->data_ptr(), ws->nbytes(), at.raw);
    gil.reset();
    if (st != SSA_OK) return PyLong_FromLong(st);
    return pair(*out, sel);
}

// bind(addresses of the C functions, in Api's order)
PyObject* bind(Args& a) {
    auto fn = [&](auto& f) {
        f = reinterpret_cast<std::decay_t<decltype(f)>>((uintptr_t)a.integer("address"));
    };
    fn(api.rope);
    fn(api.append);
    fn(api.read);
    fn(api.workspace);
    fn(api.decode);
    Py_RETURN_NONE;
}

template <PyObject* (*F)(Args&), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    try {
        Args a(args, n, N);
        return F(a);
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const WrongType& e) {
        PyErr_SetString(PyExc_TypeError, e.what());
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(PyExc_MemoryError, e.what_without_backtrace());
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define SSA_METHOD(name, n) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {SSA_METHOD(rope, 11), SSA_METHOD(append, 10), SSA_METHOD(read, 12),
                         SSA_METHOD(decode, 18), SSA_METHOD(bind, 5), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cache", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__cache(void) { return PyModule_Create(&module); }
