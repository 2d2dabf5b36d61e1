// binding.cpp -- the native side of adamw.py: checks of tensors and lists of tensors, and the call
// of the C entry points (whose addresses `init` is given, so that this module links to nothing of
// the library's). A step over hundreds of tensors needs each one's type, device, layout, length
// and address: about 1.1 us a tensor in Python, 20 ns here (a step over 240 small tensors: 272 us
// through ctypes, of which the GPU works 6).
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include <ATen/ATen.h>
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

}  // namespace

PYBIND11_MODULE(_binding, m) {
    m.def("init", &init);
    m.def("step", &step);
    m.def("get_state8", &get_state8);
    m.def("set_state8", &set_state8);
    m.def("grad_norm", &grad_norm);
}
