// binding.cpp -- the native side of adamw.py and mx4.py: checks of tensors and lists of tensors, and the call
// of the C entry points (whose addresses `init` is given, so that this module links to nothing of
// the library's). A step over hundreds of tensors needs each one's type, device, layout, length
// and address: about 1.1 us a tensor in Python, 20 ns here (a step over 240 small tensors: 272 us
// through ctypes, of which the GPU works 6).
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include <ATen/ATen.h>
#include <ATen/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>
#include <string>
#include <vector>

#include "adamw_clip.h"
#include "onebit_adam.h"

namespace py = pybind11;

namespace {

decltype(&onebit_adamw_step) p_step = nullptr;
decltype(&onebit_adamw8_step) p_step8 = nullptr;
decltype(&onebit_adamw8_get_state) p_get = nullptr;
decltype(&onebit_adamw8_set_state) p_set = nullptr;
decltype(&onebit_grad_norm) p_norm = nullptr;
decltype(&onebit_internal_adamw_clipped_step) p_clipped = nullptr;
decltype(&onebit_mx4_layout) p_mx4_layout = nullptr;
decltype(&onebit_mx4_quantize) p_mx4_quantize = nullptr;
decltype(&onebit_mx4_dequantize) p_mx4_dequantize = nullptr;
decltype(&onebit_mx4_matmul) p_mx4_matmul = nullptr;
decltype(&onebit_mx4_linear) p_mx4_linear = nullptr;
decltype(&onebit_mx4_linear_needs) p_mx4_linear_needs = nullptr;
PyObject* g_error = nullptr;  // OneBitError
constexpr int kScaleOffset = 12;  // of the clip factor in the norm's work, in bytes

template <typename F>
void address(F& f, const py::dict& d, const char* name) {
    f = reinterpret_cast<F>(py::cast<uintptr_t>(d[name]));
}

void init(const py::dict& addresses, const py::object& error) {
    address(p_step, addresses, "onebit_adamw_step");
    address(p_step8, addresses, "onebit_adamw8_step");
    address(p_get, addresses, "onebit_adamw8_get_state");
    address(p_set, addresses, "onebit_adamw8_set_state");
    address(p_norm, addresses, "onebit_grad_norm");
    address(p_clipped, addresses, "onebit_internal_adamw_clipped_step");
    address(p_mx4_layout, addresses, "onebit_mx4_layout");
    address(p_mx4_quantize, addresses, "onebit_mx4_quantize");
    address(p_mx4_dequantize, addresses, "onebit_mx4_dequantize");
    address(p_mx4_matmul, addresses, "onebit_mx4_matmul");
    address(p_mx4_linear, addresses, "onebit_mx4_linear");
    address(p_mx4_linear_needs, addresses, "onebit_mx4_linear_needs");
    g_error = error.inc_ref().ptr();
}

void refuse(int rc, const char* where) {
    if (rc == ONEBIT_OK) return;
    const py::object e =
        py::reinterpret_borrow<py::object>(g_error)(rc, where, py::arg("reason") = true);
    PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(e.ptr())), e.ptr());
    throw py::error_already_set();
}

std::string type_name(at::ScalarType t) {
    return py::str(reinterpret_cast<PyObject*>(torch::getTHPDtype(t)));
}

int32_t dtype_code(at::ScalarType t, const std::string& name) {
    if (t == at::kFloat) return ONEBIT_F32;
    if (t == at::kBFloat16) return ONEBIT_BF16;
    throw py::type_error(name + " must be float32 or bfloat16, got " + type_name(t));
}

void check_cuda(const at::Tensor& t, const std::string& name, const c10::Device* device) {
    if (!t.is_cuda())
        throw py::value_error(name + " must be a CUDA tensor, got device " + t.device().str());
    if (device != nullptr && t.device() != *device)
        throw py::value_error(name + " is on " + t.device().str() + ", expected " + device->str());
}

// One vector: a contiguous CUDA tensor of a type with at least so many elements.
const at::Tensor& vector(const py::handle& o, at::ScalarType type, int64_t numel,
                         const std::string& name, const c10::Device* device) {
    if (!THPVariable_Check(o.ptr())) throw py::type_error(name + " must be a torch.Tensor");
    const at::Tensor& t = THPVariable_Unpack(o.ptr());
    check_cuda(t, name, device);
    if (t.scalar_type() != type)
        throw py::type_error(name + " must be " + type_name(type) + ", got " +
                             type_name(t.scalar_type()));
    if (!t.is_contiguous()) throw py::value_error(name + " must be contiguous");
    if (t.numel() < numel)
        throw py::value_error(name + " holds " + std::to_string(t.numel()) +
                              " elements, needs at least " + std::to_string(numel));
    return t;
}

// A list of tensors of one type on one device. The tensors are the Python objects' own: the list
// (kept alive here) holds them, and the GIL is not given up before the call is over.
struct List {
    py::object seq;
    std::vector<const at::Tensor*> tensors;
    std::vector<int64_t> numel;
    std::vector<void*> data;
    at::ScalarType type = at::kFloat;
    int32_t n() const { return (int32_t)tensors.size(); }
};

List list_of(const py::handle& o, const char* name, const c10::Device* device,
             const std::vector<int64_t>* numel) {
    List l;
    l.seq = py::reinterpret_steal<py::object>(
        PySequence_Fast(o.ptr(), (std::string(name) + " must be a list of tensors").c_str()));
    if (!l.seq) throw py::error_already_set();
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(l.seq.ptr());
    if (n > INT32_MAX) throw py::value_error(std::string(name) + ": too many tensors");
    l.tensors.resize(n);
    l.numel.resize(n);
    l.data.resize(n);
    c10::Device first(c10::kCPU);
    for (Py_ssize_t i = 0; i < n; ++i) {
        PyObject* p = PySequence_Fast_GET_ITEM(l.seq.ptr(), i);
        if (!THPVariable_CheckExact(p) && !THPVariable_Check(p))
            throw py::type_error(std::string(name) + " must be a list of tensors");
        const at::Tensor& t = THPVariable_Unpack(p);
        if (i == 0) {
            check_cuda(t, name, device);
            l.type = t.scalar_type();
            first = t.device();
        } else if (t.scalar_type() != l.type || t.device() != first) {
            throw py::value_error(std::string(name) + " must be of one type on one device, got " +
                                  type_name(l.type) + " on " + first.str() + " and " +
                                  type_name(t.scalar_type()) + " on " + t.device().str());
        }
        if (!t.is_contiguous()) throw py::value_error(std::string(name) + " must be contiguous");
        l.tensors[i] = &t;
        l.numel[i] = t.numel();
        l.data[i] = t.data_ptr();
    }
    if (numel != nullptr && l.numel != *numel)
        throw py::value_error(std::string(name) + " have lengths other than the parameters'");
    return l;
}

// The device and stream of one call: the tensors' device is made current, and tensors are marked
// as used on the stream where that is not the device's current one.
class Queue {
  public:
    Queue(const c10::Device& device, const py::handle& stream)
        : guard_(device),
          current_(c10::cuda::getCurrentCUDAStream(device.index())),
          stream_(current_) {
        if (stream.is_none()) return;
        uintptr_t handle;
        if (py::isinstance<py::int_>(stream)) {
            handle = py::cast<uintptr_t>(stream);
        } else {
            const py::object d = stream.attr("device");
            if (!THPDevice_Check(d.ptr()) ||
                reinterpret_cast<THPDevice*>(d.ptr())->device != device)
                throw py::value_error("stream is on " + std::string(py::str(d)) +
                                      ", the tensors are on " + device.str());
            handle = py::cast<uintptr_t>(stream.attr("cuda_stream"));
        }
        stream_ = handle == 0 ? c10::cuda::getDefaultCUDAStream(device.index())
                              : c10::cuda::getStreamFromExternal(
                                    reinterpret_cast<cudaStream_t>(handle), device.index());
    }
    void* handle() const { return reinterpret_cast<void*>(stream_.stream()); }
    void uses(const at::Tensor& t) const {
        if (stream_.stream() != current_.stream() && t.defined() && t.numel() > 0)
            t.record_stream(stream_.unwrap());
    }
    void uses(const std::vector<const at::Tensor*>& ts) const {
        if (stream_.stream() == current_.stream()) return;
        for (const at::Tensor* t : ts) uses(*t);
    }
    // Memory of the call's own stream for a result. The current stream's pool may hand out a block
    // that work queued there still uses, which the call's stream does not wait for. The caller goes
    // on with the result on the current stream: it is marked as used there.
    template <typename F>
    at::Tensor make(F&& allocate) const {
        if (stream_.stream() == current_.stream()) return allocate();
        const c10::cuda::CUDAStreamGuard on(stream_);
        const at::Tensor t = allocate();
        if (t.numel() > 0) t.record_stream(current_.unwrap());
        return t;
    }

  private:
    c10::cuda::CUDAGuard guard_;
    c10::cuda::CUDAStream current_, stream_;
};

// Autograd takes note of the change.
void changed(const std::vector<const at::Tensor*>& ts) {
    for (const at::Tensor* t : ts)
        if (!t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

int64_t blocks_of(const std::vector<int64_t>& numel) {
    int64_t b = 0;
    for (const int64_t n : numel) b += (n + ONEBIT_ADAMW_BLOCK - 1) / ONEBIT_ADAMW_BLOCK;
    return b;
}

// seed None: fp32 states (m, v); else 8-bit ones (m, v, m_exp, v_exp). lengths: None, or what the
// parameters' lengths have to be. clip: None, or (work, max_norm): the gradients' norm first, whose
// factor is the step's grad_scale; the lists are read and checked once for both.
void step(const char* where, const py::object& params, const py::object& grads,
          const py::tuple& state, const py::object& ctl_o, const py::object& lr_o, double beta1,
          double beta2, double eps, const py::object& decay, const py::object& copies,
          const py::object& scale_o, bool bias, const py::object& stream, const py::object& seed,
          const py::object& lengths, const py::object& clip) {
    const bool eight = !seed.is_none();
    const Py_ssize_t np = PyObject_Length(params.ptr()), ng = PyObject_Length(grads.ptr());
    if (np < 0 || ng < 0) throw py::error_already_set();
    if (np != ng)
        throw py::value_error(std::to_string(ng) + " gradients for " + std::to_string(np) +
                              " parameters");
    const at::Tensor& ctl =
        vector(ctl_o, at::kLong, ONEBIT_ADAMW_CTL_BYTES / 8, "ctl", nullptr);
    const c10::Device device = ctl.device();
    const List p = list_of(params, "params", &device, nullptr);
    if (!lengths.is_none()) {
        const py::list want = py::cast<py::list>(lengths);
        bool same = (int64_t)want.size() == p.n();
        for (int32_t i = 0; same && i < p.n(); ++i)
            same = PyLong_AsLongLong(PyList_GET_ITEM(want.ptr(), i)) == p.numel[i];
        if (PyErr_Occurred()) throw py::error_already_set();
        if (!same) throw py::value_error("params have lengths other than the optimizer's");
    }
    const List g = list_of(grads, "grads", &device, &p.numel);
    const int32_t pt = dtype_code(p.type, "params"), gt = dtype_code(g.type, "grads");
    List c;
    if (!copies.is_none()) {
        c = list_of(copies, "copies", &device, nullptr);
        if (c.n() != p.n())
            throw py::value_error(std::to_string(c.n()) + " copies for " + std::to_string(np) +
                                  " parameters");
        if (c.n() > 0 && c.type != at::kBFloat16)
            throw py::type_error("copies must be torch.bfloat16, got " + type_name(c.type));
        if (c.numel != p.numel)
            throw py::value_error("copies have lengths other than the parameters'");
    }
    const int64_t blocks = blocks_of(p.numel), total = blocks * ONEBIT_ADAMW_BLOCK;
    static const char* const names[] = {"m", "v", "m_exp", "v_exp"};
    const at::Tensor* st[4] = {};
    for (int k = 0; k < (eight ? 4 : 2); ++k)
        st[k] = &vector(state[k], eight ? at::kByte : at::kFloat, k < 2 ? total : blocks, names[k],
                        &device);
    std::vector<double> wd;
    if (!PySequence_Check(decay.ptr())) {
        wd.assign(p.n(), py::cast<double>(py::float_(decay)));
    } else {
        const py::object seq = py::reinterpret_steal<py::object>(
            PySequence_Fast(decay.ptr(), "weight_decay must be a number or a list of numbers"));
        if (!seq) throw py::error_already_set();
        wd.resize(PySequence_Fast_GET_SIZE(seq.ptr()));
        for (size_t i = 0; i < wd.size(); ++i)
            wd[i] = PyFloat_AsDouble(PySequence_Fast_GET_ITEM(seq.ptr(), i));
        if (PyErr_Occurred()) throw py::error_already_set();
        if ((int64_t)wd.size() != p.n())
            throw py::value_error(std::to_string(wd.size()) + " weight decays for " +
                                  std::to_string(np) + " parameters");
    }
    at::Tensor scale, lr_dev, work;
    double max_norm = 0.0;
    if (!clip.is_none()) {
        if (!scale_o.is_none())
            throw py::value_error("grad_scale and max_norm exclude each other");
        const py::tuple both = py::cast<py::tuple>(clip);
        work = vector(both[0], at::kByte, ONEBIT_GRAD_NORM_BYTES, "work", &device);
        max_norm = py::cast<double>(both[1]);
    }
    if (!scale_o.is_none()) scale = vector(scale_o, at::kFloat, 1, "grad_scale", &device);
    double lr = 0.0;
    if (THPVariable_Check(lr_o.ptr()))
        lr_dev = vector(lr_o, at::kDouble, 1, "lr", &device);
    else
        lr = py::cast<double>(lr_o);
    const auto* scale_p = scale.defined() ? scale.data_ptr<float>() : nullptr;
    const auto* lr_p = lr_dev.defined() ? lr_dev.data_ptr<double>() : nullptr;
    void* const* cp = copies.is_none() ? nullptr : c.data.data();
    const uint64_t key = eight ? PyLong_AsUnsignedLongLongMask(seed.ptr()) : 0;
    if (PyErr_Occurred()) throw py::error_already_set();

    const Queue q(device, stream);
    int rc;
    bool queued = false;   // a refusal queues nothing; what is queued uses its tensors, come what may
    if (work.defined()) {
        OneBitAdamwClip a{};
        a.ntensors = p.n();
        a.numel = p.numel.data();
        a.params = p.data.data();
        a.param_dtype = pt;
        a.grads = g.data.data();
        a.grad_dtype = gt;
        a.copies = cp;
        a.m = st[0]->data_ptr();
        a.v = st[1]->data_ptr();
        a.eight = eight;
        if (eight) {
            a.m_exp = st[2]->data_ptr<uint8_t>();
            a.v_exp = st[3]->data_ptr<uint8_t>();
        }
        a.seed = key;
        a.ctl = ctl.data_ptr();
        a.weight_decay = wd.data();
        a.max_norm = max_norm;
        a.work = work.data_ptr();
        a.lr_dev = lr_p;
        a.lr = lr;
        a.beta1 = beta1;
        a.beta2 = beta2;
        a.eps = eps;
        a.bias_correction = bias ? 1 : 0;
        a.stream = q.handle();
        rc = p_clipped(&a, &queued);
    } else {
        rc = eight
                 ? p_step8(p.n(), p.numel.data(), p.data.data(), pt, g.data.data(), gt, cp,
                           st[0]->data_ptr<uint8_t>(), st[1]->data_ptr<uint8_t>(),
                           st[2]->data_ptr<uint8_t>(), st[3]->data_ptr<uint8_t>(), ctl.data_ptr(),
                           key, wd.data(), scale_p, lr_p, lr, beta1, beta2, eps, bias ? 1 : 0,
                           q.handle())
                 : p_step(p.n(), p.numel.data(), p.data.data(), pt, g.data.data(), gt, cp,
                          st[0]->data_ptr<float>(), st[1]->data_ptr<float>(), ctl.data_ptr(),
                          wd.data(), scale_p, lr_p, lr, beta1, beta2, eps, bias ? 1 : 0,
                          q.handle());
        queued = rc == ONEBIT_OK || rc == ONEBIT_ERR_CUDA;
    }
    if (queued) {
        changed(p.tensors);
        changed(c.tensors);
        q.uses(p.tensors);
        q.uses(g.tensors);
        q.uses(c.tensors);
        for (const at::Tensor* t : st)
            if (t != nullptr) q.uses(*t);
        q.uses(ctl);
        q.uses(scale);
        q.uses(lr_dev);
        q.uses(work);
    }
    refuse(rc, where);
}

// The 8-bit states of one call.
struct State8 {
    at::Tensor m, v, mk, vk;
    int64_t total;
};

State8 state8(const py::handle& m, const py::handle& v, const py::handle& mk,
              const py::handle& vk) {
    State8 s;
    s.m = vector(m, at::kByte, 0, "m", nullptr);
    s.total = s.m.numel();
    if (s.total % ONEBIT_ADAMW_BLOCK != 0)
        throw py::value_error("m holds " + std::to_string(s.total) + " codes, not a multiple of " +
                              std::to_string(ONEBIT_ADAMW_BLOCK));
    const c10::Device device = s.m.device();
    s.v = vector(v, at::kByte, s.total, "v", &device);
    s.mk = vector(mk, at::kByte, s.total / ONEBIT_ADAMW_BLOCK, "m_exp", &device);
    s.vk = vector(vk, at::kByte, s.total / ONEBIT_ADAMW_BLOCK, "v_exp", &device);
    return s;
}

py::tuple get_state8(const py::object& m, const py::object& v, const py::object& mk,
                     const py::object& vk, const py::object& m_out, const py::object& v_out,
                     const py::object& dtype, const py::object& stream) {
    const State8 s = state8(m, v, mk, vk);
    const c10::Device device = s.m.device();
    at::ScalarType type = at::kFloat;
    if (!dtype.is_none()) {
        if (!THPDtype_Check(dtype.ptr())) throw py::type_error("dtype must be a torch.dtype");
        type = reinterpret_cast<THPDtype*>(dtype.ptr())->scalar_type;
    } else {
        for (const py::object* o : {&m_out, &v_out})
            if (THPVariable_Check(o->ptr())) type = THPVariable_Unpack(o->ptr()).scalar_type();
    }
    const int32_t code = dtype_code(type, "the values");
    const Queue q(device, stream);
    at::Tensor out[2];
    const py::object* given[2] = {&m_out, &v_out};
    static const char* const names[2] = {"m_out", "v_out"};
    for (int k = 0; k < 2; ++k)
        out[k] = given[k]->is_none()
                     ? q.make([&] { return at::empty({s.total}, s.m.options().dtype(type)); })
                     : vector(*given[k], type, s.total, names[k], &device);
    refuse(p_get(s.total, s.m.data_ptr<uint8_t>(), s.v.data_ptr<uint8_t>(),
                 s.mk.data_ptr<uint8_t>(), s.vk.data_ptr<uint8_t>(), out[0].data_ptr(),
                 out[1].data_ptr(), code, q.handle()),
           "onebit_adamw8_get_state");
    for (const at::Tensor& t : {s.m, s.v, s.mk, s.vk, out[0], out[1]}) q.uses(t);
    return py::make_tuple(out[0], out[1]);
}

void set_state8(const py::object& m, const py::object& v, const py::object& mk,
                const py::object& vk, const py::object& m_in, const py::object& v_in,
                const py::object& stream) {
    const State8 s = state8(m, v, mk, vk);
    const c10::Device device = s.m.device();
    const at::Tensor& a = vector(m_in, at::kFloat, s.total, "m_in", &device);
    const at::Tensor& b = vector(v_in, at::kFloat, s.total, "v_in", &device);
    const Queue q(device, stream);
    refuse(p_set(s.total, s.m.data_ptr<uint8_t>(), s.v.data_ptr<uint8_t>(),
                 s.mk.data_ptr<uint8_t>(), s.vk.data_ptr<uint8_t>(), a.data_ptr<float>(),
                 b.data_ptr<float>(), q.handle()),
           "onebit_adamw8_set_state");
    for (const at::Tensor& t : {s.m, s.v, s.mk, s.vk, a, b}) q.uses(t);
}

py::tuple grad_norm(const py::object& grads, double max_norm, const py::object& work_o,
                    bool accumulate, const py::object& stream) {
    at::Tensor work;
    if (work_o.is_none() && accumulate)
        throw py::value_error("accumulate needs the work of the first call");
    if (!work_o.is_none()) work = vector(work_o, at::kByte, ONEBIT_GRAD_NORM_BYTES, "work", nullptr);
    const c10::Device expected = work.defined() ? work.device() : c10::Device(c10::kCUDA);
    const List g = list_of(grads, "grads", work.defined() ? &expected : nullptr, nullptr);
    if (!work.defined() && g.n() == 0)
        throw py::value_error("no gradients and no work to say where");
    const int32_t code = dtype_code(g.type, "grads");
    const c10::Device device = work.defined() ? expected : g.tensors[0]->device();
    const Queue q(device, stream);
    if (!work.defined())
        work = q.make([&] {
            return at::zeros({ONEBIT_GRAD_NORM_BYTES}, g.tensors[0]->options().dtype(at::kByte));
        });
    refuse(p_norm(g.n(), g.numel.data(), g.data.data(), code, max_norm, accumulate ? 1 : 0,
                  work.data_ptr(), q.handle()),
           "onebit_grad_norm");
    q.uses(g.tensors);
    q.uses(work);
    const at::Tensor both = work.slice(0, kScaleOffset - 4, kScaleOffset + 4).view(at::kFloat);
    return py::make_tuple(both.select(0, 0), both.select(0, 1));
}

// ------------------------------------------------------------------------------------------
// matrices in microscaled 4-bit floating point

const at::Tensor& tensor(const py::handle& o, const std::string& name, const c10::Device* device) {
    if (!THPVariable_Check(o.ptr())) throw py::type_error(name + " must be a torch.Tensor");
    const at::Tensor& t = THPVariable_Unpack(o.ptr());
    check_cuda(t, name, device);
    return t;
}

// A plain matrix: two dimensions, consecutive columns, rows apart by its stride.
const at::Tensor& plain(const py::handle& o, const std::string& name, const c10::Device* device) {
    const at::Tensor& t = tensor(o, name, device);
    if (t.dim() != 2)
        throw py::value_error(name + " must have two dimensions, got " + std::to_string(t.dim()));
    if (t.size(1) > 1 && t.stride(1) != 1)
        throw py::value_error(name + " must have consecutive columns");
    return t;
}

// A matrix in 4 bits: codes and exponents of its size, in memory of their own or (scales undefined)
// the exponents behind the codes.
struct Packed {
    at::Tensor codes, scales;
    int64_t rows = 0, cols = 0, code_bytes = 0;
    uint8_t* c() const { return codes.defined() ? codes.data_ptr<uint8_t>() : nullptr; }
    uint8_t* s() const {
        if (scales.defined()) return scales.data_ptr<uint8_t>();
        return codes.defined() ? codes.data_ptr<uint8_t>() + code_bytes : nullptr;
    }
};

void mx4_bytes(int64_t rows, int64_t cols, int64_t& codes, int64_t& scales) {
    refuse(p_mx4_layout(rows, cols, &codes, &scales), "onebit_mx4_layout");
}

// From (codes, scales or None, rows, cols).
Packed packed(const py::handle& o, const char* name, const c10::Device* device) {
    if (!PyTuple_Check(o.ptr()) || PyTuple_GET_SIZE(o.ptr()) != 4)
        throw py::type_error(std::string(name) + " must be an Mx4");
    Packed p;
    p.rows = PyLong_AsLongLong(PyTuple_GET_ITEM(o.ptr(), 2));
    p.cols = PyLong_AsLongLong(PyTuple_GET_ITEM(o.ptr(), 3));
    if (PyErr_Occurred()) throw py::error_already_set();
    int64_t ns;
    mx4_bytes(p.rows, p.cols, p.code_bytes, ns);
    const py::handle scales = PyTuple_GET_ITEM(o.ptr(), 1);
    p.codes = vector(PyTuple_GET_ITEM(o.ptr(), 0), at::kByte,
                     scales.is_none() ? p.code_bytes + ns : p.code_bytes, name, device);
    if (!scales.is_none()) {
        const c10::Device d = p.codes.device();
        p.scales = vector(scales, at::kByte, ns, name, &d);
    }
    return p;
}

// A new tensor on the current device, from the allocator itself (through the dispatcher a product's
// call takes 5.3 us of the host, so 4.7).
at::Tensor new_tensor(const Queue& q, at::IntArrayRef sizes, at::ScalarType type) {
    return q.make([&] {
        return at::Tensor(at::detail::empty_generic(sizes, c10::cuda::CUDACachingAllocator::get(),
                                                    c10::DispatchKeySet(c10::DispatchKey::CUDA), type,
                                                    c10::nullopt));
    });
}
at::Tensor new_bytes(const Queue& q, int64_t n) { return new_tensor(q, {n}, at::kByte); }
Packed new_packed(const Queue& q, int64_t rows, int64_t cols) {
    Packed p;
    p.rows = rows;
    p.cols = cols;
    int64_t ns;
    mx4_bytes(rows, cols, p.code_bytes, ns);
    p.codes = new_bytes(q, p.code_bytes + ns);
    return p;
}

// out: None, or (codes, scales, rows, cols) of each form that is asked for, which are then written.
// Returns the two forms' new memory (codes, then scales), None for one that is given or not asked for.
py::tuple mx4_quantize(const py::object& x_o, bool rows, bool columns, bool stochastic,
                       const py::object& seed, const py::object& residual,
                       const py::object& out_rows, const py::object& out_columns,
                       const py::object& stream) {
    const at::Tensor& x = plain(x_o, "x", nullptr);
    const c10::Device device = x.device();
    const int32_t code = dtype_code(x.scalar_type(), "x");
    const int64_t r = x.size(0), c = x.size(1);
    at::Tensor e;
    if (!residual.is_none()) {
        e = plain(residual, "residual", &device);
        if (e.scalar_type() != at::kFloat)
            throw py::type_error("residual must be torch.float32, got " + type_name(e.scalar_type()));
        if (e.sizes() != x.sizes()) throw py::value_error("residual has another size than x");
    }
    Packed p[2];
    const py::object* given[2] = {&out_rows, &out_columns};
    const bool want[2] = {rows, columns};
    for (int k = 0; k < 2; ++k) {
        if (!want[k] || given[k]->is_none()) continue;
        p[k] = packed(*given[k], "out", &device);
        if (p[k].rows != (k ? c : r) || p[k].cols != (k ? r : c))
            throw py::value_error("out is of another size");
    }
    const uint64_t key = PyLong_AsUnsignedLongLongMask(seed.ptr());
    if (PyErr_Occurred()) throw py::error_already_set();
    const Queue q(device, stream);
    for (int k = 0; k < 2; ++k)
        if (want[k] && !p[k].codes.defined()) p[k] = new_packed(q, k ? c : r, k ? r : c);
    const int rc = p_mx4_quantize(
        r, c, x.data_ptr(), code, x.stride(0), p[0].c(), p[0].s(), p[1].c(), p[1].s(),
        stochastic ? 1 : 0, key, e.defined() ? e.data_ptr<float>() : nullptr,
        e.defined() ? e.stride(0) : 0, q.handle());
    if (rc == ONEBIT_OK || rc == ONEBIT_ERR_CUDA) {
        q.uses({&x, &e, &p[0].codes, &p[0].scales, &p[1].codes, &p[1].scales});
        if (e.defined()) changed({&e});
        for (int k = 0; k < 2; ++k) {
            if (!want[k] || given[k]->is_none()) continue;
            changed({&p[k].codes});
            if (p[k].scales.defined()) changed({&p[k].scales});
        }
    }
    refuse(rc, "onebit_mx4_quantize");
    const auto made = [&](int k) {
        return want[k] && given[k]->is_none() ? py::cast(p[k].codes) : py::object(py::none());
    };
    return py::make_tuple(made(0), made(1));
}

at::ScalarType result_type(const py::object& dtype, const py::object& out, at::ScalarType other) {
    if (!dtype.is_none()) {
        if (!THPDtype_Check(dtype.ptr())) throw py::type_error("dtype must be a torch.dtype");
        return reinterpret_cast<THPDtype*>(dtype.ptr())->scalar_type;
    }
    return THPVariable_Check(out.ptr()) ? THPVariable_Unpack(out.ptr()).scalar_type() : other;
}

// A result of a size and type: a given one, checked, or a new one.
at::Tensor result(const py::object& out, const Queue& q, const at::Tensor& like, int64_t rows,
                  int64_t cols, at::ScalarType type) {
    const c10::Device device = like.device();
    if (out.is_none()) return new_tensor(q, {rows, cols}, type);
    const at::Tensor& t = plain(out, "out", &device);
    if (t.scalar_type() != type)
        throw py::type_error("out must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
    if (t.size(0) != rows || t.size(1) != cols) throw py::value_error("out is of another size");
    return t;
}

at::Tensor mx4_dequantize(const py::object& matrix, const py::object& dtype, const py::object& out,
                          const py::object& stream) {
    const Packed p = packed(matrix, "q", nullptr);
    const at::ScalarType type = result_type(dtype, out, at::kFloat);
    const int32_t code = dtype_code(type, "the values");
    const Queue q(p.codes.device(), stream);
    const at::Tensor t = result(out, q, p.codes, p.rows, p.cols, type);
    const int rc = p_mx4_dequantize(p.rows, p.cols, p.c(), p.s(), t.data_ptr(), code, t.stride(0),
                                    q.handle());
    if (rc == ONEBIT_OK || rc == ONEBIT_ERR_CUDA) {
        changed({&t});
        q.uses(p.codes);
        q.uses(p.scales);
        q.uses(t);
    }
    refuse(rc, "onebit_mx4_dequantize");
    return t;
}

at::Tensor mx4_matmul(const py::object& a_o, const py::object& b_o, const py::object& out,
                      const py::object& dtype, bool accumulate, const py::object& stream) {
    const Packed a = packed(a_o, "a", nullptr);
    const c10::Device device = a.codes.device();
    const Packed b = packed(b_o, "b", &device);
    if (a.cols != b.cols)
        throw py::value_error("a has " + std::to_string(a.cols) + " columns, b " +
                              std::to_string(b.cols));
    if (accumulate && out.is_none()) throw py::value_error("accumulate needs out");
    const at::ScalarType type = result_type(dtype, out, at::kBFloat16);
    const int32_t code = dtype_code(type, "out");
    const Queue q(device, stream);
    const at::Tensor t = result(out, q, a.codes, a.rows, b.rows, type);
    const int rc = p_mx4_matmul(a.rows, b.rows, a.cols, a.c(), a.s(), b.c(), b.s(), t.data_ptr(),
                                code, t.stride(0), accumulate ? 1 : 0, q.handle());
    if (rc == ONEBIT_OK || rc == ONEBIT_ERR_CUDA) {
        changed({&t});
        for (const at::Tensor* x : {&a.codes, &a.scales, &b.codes, &b.scales, &t}) q.uses(*x);
    }
    refuse(rc, "onebit_mx4_matmul");
    return t;
}

// ------------------------------------------------------------------------------------------
// a linear layer's passes

// x [..., width] as rows: how many, and how far apart.
struct Rows {
    const at::Tensor& t;
    int64_t n, ld;
    int32_t code;
};
Rows rows_of(const py::handle& o, int64_t width, const char* name, const c10::Device& device) {
    const at::Tensor& t = tensor(o, name, &device);
    const int32_t code = dtype_code(t.scalar_type(), name);
    if (t.dim() < 1 || t.size(-1) != width) {
        std::string shape;
        for (const int64_t x : t.sizes()) shape += (shape.empty() ? "" : ", ") + std::to_string(x);
        throw py::value_error(std::string(name) + " must have " + std::to_string(width) +
                              " columns, got a shape of (" + shape + ")");
    }
    int64_t n = 1;
    for (int64_t i = 0; i + 1 < t.dim(); ++i) n *= t.size(i);
    if (t.dim() == 2) {
        if (width > 1 && t.stride(1) != 1)
            throw py::value_error(std::string(name) + " must have consecutive columns");
        return {t, n, t.stride(0), code};
    }
    if (!t.is_contiguous())
        throw py::value_error(std::string(name) + " must be contiguous, or a matrix");
    return {t, n, width, code};
}

// A new result [..., width] for rows of another width.
at::Tensor new_result(const Queue& q, const at::Tensor& x, int64_t width, at::ScalarType type) {
    c10::SmallVector<int64_t, 6> sizes(x.sizes().begin(), x.sizes().end());
    sizes.back() = width;
    return new_tensor(q, sizes, type);
}

bool was_queued(int rc) { return rc == ONEBIT_OK || rc == ONEBIT_ERR_CUDA; }

// y = x W^T of w, the weights (codes, scales, outer, inner). keep: (y, memory of the transposed x in 4
// bits).
py::object mx4_forward(const py::object& x_o, const py::object& w_o, bool keep,
                       const py::object& dtype, const py::object& stream) {
    const Packed w = packed(w_o, "the weights", nullptr);
    const c10::Device device = w.codes.device();
    const Rows x = rows_of(x_o, w.cols, "x", device);
    const at::ScalarType type = result_type(dtype, x_o, x.t.scalar_type());
    const int32_t code = dtype_code(type, "y");
    const Queue q(device, stream);
    const at::Tensor y = new_result(q, x.t, w.rows, type);
    Packed kept;
    if (keep) kept = new_packed(q, w.cols, x.n);
    at::Tensor work;
    uint8_t *codes = nullptr, *scales = nullptr;
    if (keep || p_mx4_linear_needs(x.n, w.rows, w.cols)) {
        int64_t nc, ns;
        mx4_bytes(x.n, w.cols, nc, ns);
        work = new_bytes(q, nc + ns);
        codes = work.data_ptr<uint8_t>();
        scales = codes + nc;
    }
    const int rc = p_mx4_linear(x.n, w.rows, w.cols, x.t.data_ptr(), x.code, x.ld, w.c(), w.s(), codes,
                                scales, kept.c(), kept.s(), y.data_ptr(), code, w.rows, q.handle());
    if (was_queued(rc))
        q.uses({&x.t, &w.codes, &w.scales, &y, &work, &kept.codes});
    refuse(rc, "onebit_mx4_linear");
    if (!keep) return py::cast(y);
    return py::make_tuple(y, kept.codes);
}

// (dx, dW) of dy: dx with the transposed weights wt (or None), dW with what forward kept (or None),
// into grad if that is given.
py::tuple mx4_backward(const py::object& dy_o, const py::object& wt_o, const py::object& kept_o,
                       int64_t outer, int64_t inner, const py::object& seed, const py::object& grad,
                       bool accumulate, const py::object& dtype, const py::object& stream) {
    const bool to_x = !wt_o.is_none(), to_w = !kept_o.is_none();
    const c10::Device device = tensor(dy_o, "dy", nullptr).device();
    Packed wt, kept;
    if (to_x) wt = packed(wt_o, "the weights", &device);
    if (to_w) kept = packed(kept_o, "kept", &device);
    const Rows dy = rows_of(dy_o, outer, "dy", device);
    if (to_w && (kept.rows != inner || kept.cols != dy.n))
        throw py::value_error("kept is " + std::to_string(kept.rows) + " x " + std::to_string(kept.cols) +
                              ", expected " + std::to_string(inner) + " x " + std::to_string(dy.n));
    const at::ScalarType xt = result_type(dtype, dy_o, dy.t.scalar_type());
    const at::ScalarType gt = result_type(py::none(), grad, at::kFloat);
    const int32_t xcode = dtype_code(xt, "dx"), gcode = dtype_code(gt, "grad");
    const uint64_t key = PyLong_AsUnsignedLongLongMask(seed.ptr());
    if (PyErr_Occurred()) throw py::error_already_set();
    const Queue q(device, stream);
    at::Tensor dx, dw;
    if (to_w) dw = result(grad, q, kept.codes, outer, inner, gt);
    if (to_x) dx = new_result(q, dy.t, inner, xt);
    // dy in 4 bits, along its rows and along its columns, in one piece of memory
    int64_t nc = 0, ns = 0, tc = 0, ts = 0;
    if (to_x) mx4_bytes(dy.n, outer, nc, ns);
    if (to_w) mx4_bytes(outer, dy.n, tc, ts);
    const at::Tensor work = new_bytes(q, nc + ns + tc + ts);
    uint8_t* const base = work.data_ptr<uint8_t>();
    uint8_t* const c = to_x ? base : nullptr;
    uint8_t* const ct = to_w ? base + nc + ns : nullptr;
    const char* where = "onebit_mx4_quantize";
    bool queued = false;
    int rc = p_mx4_quantize(dy.n, outer, dy.t.data_ptr(), dy.code, dy.ld, c, c ? c + nc : nullptr, ct,
                            ct ? ct + tc : nullptr, 1, key, nullptr, 0, q.handle());
    queued = was_queued(rc);
    if (rc == ONEBIT_OK && to_x) {
        where = "onebit_mx4_matmul";
        rc = p_mx4_matmul(dy.n, inner, outer, c, c + nc, wt.c(), wt.s(), dx.data_ptr(), xcode, inner, 0,
                          q.handle());
    }
    if (rc == ONEBIT_OK && to_w) {
        where = "onebit_mx4_matmul";
        rc = p_mx4_matmul(outer, inner, dy.n, ct, ct + tc, kept.c(), kept.s(), dw.data_ptr(), gcode,
                          dw.stride(0), accumulate ? 1 : 0, q.handle());
        if (was_queued(rc)) changed({&dw});
    }
    if (queued)
        q.uses({&dy.t, &wt.codes, &wt.scales, &kept.codes, &kept.scales, &work, &dx, &dw});
    refuse(rc, where);
    const auto or_none = [](const at::Tensor& t) {
        return t.defined() ? py::cast(t) : py::object(py::none());
    };
    return py::make_tuple(or_none(dx), or_none(dw));
}

}  // namespace

PYBIND11_MODULE(_binding, m) {
    m.def("init", &init);
    m.def("step", &step);
    m.def("get_state8", &get_state8);
    m.def("set_state8", &set_state8);
    m.def("grad_norm", &grad_norm);
    m.def("mx4_quantize", &mx4_quantize);
    m.def("mx4_dequantize", &mx4_dequantize);
    m.def("mx4_matmul", &mx4_matmul);
    m.def("mx4_forward", &mx4_forward);
    m.def("mx4_backward", &mx4_backward);
}
