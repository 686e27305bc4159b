// vsl_binding.cpp - the Python side of the calls whose own time is a few
// microseconds: argument checks, output tensors and the call into libvsl
// without an interpreter's cost for each of them.  It holds no arithmetic.
//
// Every function takes positional arguments from the functions of the same
// names in __init__.py, which document them, and raises what they promise:
// ValueError and TypeError for the tensors, VslError for a status of the
// library.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <exception>
#include <memory>
#include <optional>
#include <string>
#include <vector>

#include "../../include/vsl.h"

namespace {

PyObject* g_error_class = nullptr;  // VslError

// A Python exception is set: unwinds to the entry point.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw Raised();
}

void check_status(vsl_status status, const char* where) {
  if (status == VSL_OK) return;
  PyObject* e = PyObject_CallFunction(g_error_class, "is", static_cast<int>(status), where);
  if (e != nullptr) {
    PyErr_SetObject(g_error_class, e);
    Py_DECREF(e);
  }
  throw Raised();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a tensor, not %s", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

std::string describe(at::ScalarType type, at::IntArrayRef shape, at::Device device) {
  std::string s = type == at::kFloat ? "torch.float32" : type == at::kBFloat16 ? "torch.bfloat16" : "torch.int32";
  s += " [";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + "] tensor on " + device.str();
}

// The address of a contiguous tensor of this type and shape (None: null where allowed).
void* address(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, at::Device device,
              bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous() || t.device() != device)
    raise(PyExc_ValueError, "%s must be a contiguous %s", name, describe(type, shape, device).c_str());
  return t.data_ptr();
}

// A list or tuple; of any other iterable a list, which alone may hold its
// tensors: their addresses are good as long as this lives.
struct Sequence {
  PyObject* fast;
  Py_ssize_t size;
  Sequence(PyObject* o, const char* name) : fast(PySequence_Fast(o, name)) {
    if (fast == nullptr) throw Raised();
    size = PySequence_Fast_GET_SIZE(fast);
  }
  ~Sequence() { Py_XDECREF(fast); }
  Sequence(const Sequence&) = delete;
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(fast, i); }
};

using Addresses = std::vector<void*>;

int as_int(int64_t v, const char* name) {
  if (v < 0 || v > 0x7FFFFFFF) raise(PyExc_ValueError, "%s is beyond 32 bits", name);
  return static_cast<int>(v);
}

// The logits slices of a call.
struct Slices {
  Sequence list;
  Addresses at;
  int R = 0, S = 0, V_s = 0;
  at::Device device = at::Device(at::kCPU);

  Slices(PyObject* o, const char* where) : list(o, "logits_slices must be a list of tensors") {
    if (list.size == 0) raise(PyExc_ValueError, "%s: no logits slices", where);
    const at::Tensor& first = tensor(list[0], "logits_slices");
    if (first.dim() != 2) raise(PyExc_ValueError, "%s: logits slices must be [R, V_s]", where);
    device = first.device();
    R = as_int(first.size(0), "R");
    V_s = as_int(first.size(1), "V_s");
    S = as_int(list.size, "S");
    at.reserve(S);
    for (int s = 0; s < S; ++s) {
      const at::Tensor& t = tensor(list[s], "logits_slices");
      if (t.scalar_type() != at::kFloat || t.sizes() != first.sizes() || !t.is_contiguous() || t.device() != device)
        raise(PyExc_ValueError, "%s: logits slices must be contiguous fp32 [R, V_s] on one device", where);
      at.push_back(t.data_ptr());
    }
  }
  const float* const* logits() const { return reinterpret_cast<const float* const*>(at.data()); }
};

void need_cuda(at::Device d) {
  if (!d.is_cuda()) raise(PyExc_ValueError, "libvsl needs CUDA tensors, got a tensor on %s", d.str().c_str());
}

// The device and stream of a call (the given handle, or the device's current
// stream), current while the call lasts: what it allocates comes from the pool
// of the stream that writes it.
class Launch {
 public:
  Launch(PyObject* handle, at::Device d) {
    if (handle == Py_None) {
      device_.emplace(d);
      stream_ = c10::cuda::getCurrentCUDAStream(d.index()).stream();
      return;
    }
    void* at = PyLong_AsVoidPtr(handle);
    if (at == nullptr && PyErr_Occurred()) throw Raised();
    stream_ = static_cast<cudaStream_t>(at);
    on_.emplace(c10::cuda::getStreamFromExternal(stream_, d.index()));
  }
  void* stream() const { return stream_; }

 private:
  std::optional<c10::cuda::CUDAGuard> device_;
  std::optional<c10::cuda::CUDAStreamGuard> on_;
  cudaStream_t stream_ = nullptr;
};

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, at::Device d) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(d));
}

// A contiguous piece of a fresh tensor as a tensor of its own over the same
// storage (a view without the dispatcher, which takes a microsecond).
at::Tensor piece(const at::Tensor& whole, int64_t first, at::IntArrayRef shape) {
  at::Tensor t =
      at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(), whole.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(first);
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}

PyObject* wrap(const at::Tensor& t) {
  PyObject* o = THPVariable_Wrap(t);
  if (o == nullptr) throw Raised();
  return o;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v == 1;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}

// Output slices [R, V_s]: the given ones, or new ones of one allocation where
// that keeps every slice aligned.
struct OutSlices {
  Addresses at;
  PyObject* list = nullptr;  // owned
  at::ScalarType type;

  OutSlices(PyObject* given, const char* name, at::ScalarType want, bool any_type, const Slices& in) : type(want) {
    at.reserve(in.S);
    if (given != Py_None) {
      Sequence l(given, name);
      if (l.size != in.S) raise(PyExc_ValueError, "%s must hold %d slices", name, in.S);
      if (any_type) {
        type = tensor(l[0], name).scalar_type();
        if (type != at::kFloat && type != at::kBFloat16) raise(PyExc_TypeError, "the gradient is float32 or bfloat16");
      }
      for (int s = 0; s < in.S; ++s) at.push_back(address(l[s], name, type, {in.R, in.V_s}, in.device));
      list = l.fast;
      Py_INCREF(list);
      return;
    }
    need_cuda(in.device);
    list = PyList_New(in.S);
    if (list == nullptr) throw Raised();
    const bool one = static_cast<int64_t>(in.R) * in.V_s % 8 == 0;
    const int64_t entries = static_cast<int64_t>(in.R) * in.V_s;
    at::Tensor all;
    if (one) all = empty({in.S * entries}, type, in.device);
    for (int s = 0; s < in.S; ++s) {
      const at::Tensor t = one ? piece(all, s * entries, {in.R, in.V_s}) : empty({in.R, in.V_s}, type, in.device);
      at.push_back(t.data_ptr());
      PyList_SET_ITEM(list, s, wrap(t));
    }
  }
  ~OutSlices() { Py_XDECREF(list); }
  OutSlices(const OutSlices&) = delete;
  PyObject* take() {
    PyObject* l = list;
    list = nullptr;
    return l;
  }
};

void need(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) raise(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
}

// token_logprobs(slices, token_ids, temperature, entropy, logprob, entropy_out, row_stats, stream): the three
// outputs, given or None (new ones)
PyObject* token_logprobs(PyObject* const* a, Py_ssize_t n) {
  need(n, 8);
  const Slices in(a[0], "token_logprobs");
  const void* tokens = address(a[1], "token_ids", at::kInt, {in.R}, in.device);
  const float temperature = static_cast<float>(number(a[2]));
  const bool entropy = truth(a[3]);
  need_cuda(in.device);
  const Launch launch(a[7], in.device);
  PyObject* out[3] = {a[4], a[5], a[6]};
  at::Tensor fresh[3];
  void* at[3] = {nullptr, nullptr, nullptr};
  const char* names[3] = {"out.logprob", "out.entropy", "out.row_stats"};
  for (int i = 0; i < 3; ++i) {
    if (i == 1 && !entropy) continue;
    if (out[i] != Py_None) {
      at[i] = i == 2 ? address(out[i], names[i], at::kFloat, {in.R, 2}, in.device)
                     : address(out[i], names[i], at::kFloat, {in.R}, in.device);
    } else {
      fresh[i] = i == 2 ? empty({in.R, 2}, at::kFloat, in.device) : empty({in.R}, at::kFloat, in.device);
      at[i] = fresh[i].data_ptr();
    }
  }
  check_status(vsl_token_logprobs(in.logits(), in.R, in.S, in.V_s, static_cast<const int32_t*>(tokens), temperature,
                                  static_cast<float*>(at[0]), static_cast<float*>(at[1]), static_cast<float*>(at[2]),
                                  launch.stream()),
               "vsl_token_logprobs");
  PyObject* result = PyTuple_New(3);
  if (result == nullptr) throw Raised();
  for (int i = 0; i < 3; ++i) {
    PyObject* o = out[i];
    if (fresh[i].defined())
      o = wrap(fresh[i]);
    else
      Py_INCREF(o);
    PyTuple_SET_ITEM(result, i, o);
  }
  return result;
}

at::ScalarType grad_type(PyObject* bf16) { return truth(bf16) ? at::kBFloat16 : at::kFloat; }

// token_logprobs_grad(slices, token_ids, temperature, row_stats, entropy, d_logprob, d_entropy, grad, bf16, stream)
PyObject* token_logprobs_grad(PyObject* const* a, Py_ssize_t n) {
  need(n, 10);
  const Slices in(a[0], "token_logprobs_grad");
  const void* tokens = address(a[1], "token_ids", at::kInt, {in.R}, in.device);
  const float temperature = static_cast<float>(number(a[2]));
  const void* stats = address(a[3], "forward.row_stats", at::kFloat, {in.R, 2}, in.device);
  const void* d_logprob = address(a[5], "d_logprob", at::kFloat, {in.R}, in.device);
  const void* d_entropy = address(a[6], "d_entropy", at::kFloat, {in.R}, in.device, true);
  if (d_entropy != nullptr && a[4] == Py_None) raise(PyExc_ValueError, "d_entropy needs a forward call with entropy=True");
  const void* entropy =
      d_entropy != nullptr ? address(a[4], "forward.entropy", at::kFloat, {in.R}, in.device) : nullptr;
  need_cuda(in.device);
  const Launch launch(a[9], in.device);
  OutSlices grad(a[7], "grad", grad_type(a[8]), true, in);
  check_status(vsl_token_logprobs_grad(in.logits(), in.R, in.S, in.V_s, static_cast<const int32_t*>(tokens), temperature,
                                       static_cast<const float*>(stats), static_cast<const float*>(entropy),
                                       static_cast<const float*>(d_logprob), static_cast<const float*>(d_entropy),
                                       grad.at.data(), grad.type == at::kBFloat16 ? VSL_GRAD_BF16 : VSL_GRAD_FP32,
                                       launch.stream()),
               "vsl_token_logprobs_grad");
  return grad.take();
}

// policy_loss(slices, token_ids, old_logprob, advantages, weights, ref_logprob, clip_low, clip_high, kl_coef,
// entropy_coef, temperature, grad (False: none, None: new), bf16, stream): (loss, logprob, kl, entropy, grad)
PyObject* policy_loss(PyObject* const* a, Py_ssize_t n) {
  need(n, 14);
  const Slices in(a[0], "policy_loss");
  vsl_policy_inputs i{};
  i.token_ids = static_cast<const int32_t*>(address(a[1], "token_ids", at::kInt, {in.R}, in.device));
  i.old_logprob = static_cast<const float*>(address(a[2], "old_logprob", at::kFloat, {in.R}, in.device));
  i.advantages = static_cast<const float*>(address(a[3], "advantages", at::kFloat, {in.R}, in.device));
  i.weights = static_cast<const float*>(address(a[4], "weights", at::kFloat, {in.R}, in.device, true));
  i.ref_logprob = static_cast<const float*>(address(a[5], "ref_logprob", at::kFloat, {in.R}, in.device, true));
  i.clip_low = static_cast<float>(number(a[6]));
  i.clip_high = static_cast<float>(number(a[7]));
  i.kl_coef = static_cast<float>(number(a[8]));
  i.entropy_coef = static_cast<float>(number(a[9]));
  i.temperature = static_cast<float>(number(a[10]));
  need_cuda(in.device);
  const Launch launch(a[13], in.device);
  const bool with_grad = a[11] != Py_False;
  const at::Tensor rows = empty({4 * static_cast<int64_t>(in.R)}, at::kFloat, in.device);
  float* at = rows.data_ptr<float>();
  vsl_policy_outputs o{};
  o.loss = at;
  o.logprob = at + in.R;
  o.kl = at + 2 * static_cast<int64_t>(in.R);
  o.entropy = at + 3 * static_cast<int64_t>(in.R);
  PyObject* grad_list = nullptr;
  {
    std::unique_ptr<OutSlices> grad;
    if (with_grad) {
      grad.reset(new OutSlices(a[11], "grad", grad_type(a[12]), true, in));
      o.grad_slices = grad->at.data();
      o.grad_type = grad->type == at::kBFloat16 ? VSL_GRAD_BF16 : VSL_GRAD_FP32;
    }
    check_status(vsl_policy_loss(in.logits(), in.R, in.S, in.V_s, &i, &o, launch.stream()), "vsl_policy_loss");
    if (with_grad) grad_list = grad->take();
  }
  PyObject* result = PyTuple_New(5);
  if (result == nullptr) {
    Py_XDECREF(grad_list);
    throw Raised();
  }
  if (grad_list == nullptr) {
    grad_list = Py_None;
    Py_INCREF(grad_list);
  }
  PyTuple_SET_ITEM(result, 4, grad_list);
  for (int k = 0; k < 4; ++k) PyTuple_SET_ITEM(result, k, wrap(piece(rows, k * static_cast<int64_t>(in.R), {in.R})));
  return result;
}

// preference_loss(logprob, ref_logprob, offsets, weights, beta, label_smoothing, stream): (loss, rewards, d_logprob)
PyObject* preference_loss(PyObject* const* a, Py_ssize_t n) {
  need(n, 7);
  const at::Tensor& logprob = tensor(a[0], "logprob");
  const at::Device device = logprob.device();
  const int R = as_int(logprob.numel(), "R");
  const at::Tensor& offsets = tensor(a[2], "offsets");
  const int64_t entries = offsets.numel();
  if (entries < 3 || entries % 2 == 0) raise(PyExc_ValueError, "offsets must hold 2 * pairs + 1 entries");
  const int pairs = as_int((entries - 1) / 2, "pairs");
  const void* lp = address(a[0], "logprob", at::kFloat, {R}, device);
  const void* ref = address(a[1], "ref_logprob", at::kFloat, {R}, device, true);
  const void* at = address(a[2], "offsets", at::kInt, {entries}, device);
  const void* weights = address(a[3], "weights", at::kFloat, {pairs}, device, true);
  const float beta = static_cast<float>(number(a[4])), smoothing = static_cast<float>(number(a[5]));
  need_cuda(device);
  const Launch launch(a[6], device);
  const at::Tensor loss = empty({pairs}, at::kFloat, device), rewards = empty({pairs, 2}, at::kFloat, device);
  const at::Tensor d = empty({R}, at::kFloat, device);
  check_status(vsl_preference_loss(static_cast<const float*>(lp), static_cast<const float*>(ref),
                                   static_cast<const int32_t*>(at), static_cast<const float*>(weights), R, pairs, beta,
                                   smoothing, loss.data_ptr<float>(), rewards.data_ptr<float>(), d.data_ptr<float>(),
                                   launch.stream()),
               "vsl_preference_loss");
  PyObject* result = PyTuple_New(3);
  if (result == nullptr) throw Raised();
  PyTuple_SET_ITEM(result, 0, wrap(loss));
  PyTuple_SET_ITEM(result, 1, wrap(rewards));
  PyTuple_SET_ITEM(result, 2, wrap(d));
  return result;
}

// adapters_add(slices, hidden, a, b_slices, adapter_ids, scale, out, tile_stats (None: none), workspace, stream): out
PyObject* adapters_add(PyObject* const* a, Py_ssize_t n) {
  need(n, 10);
  const Slices in(a[0], "adapters_add");
  const at::Tensor& pool = tensor(a[2], "a");
  if (pool.dim() != 3) raise(PyExc_ValueError, "a must be [n, rank, H]");
  const int adapters = as_int(pool.size(0), "n"), rank = as_int(pool.size(1), "rank"), H = as_int(pool.size(2), "H");
  Sequence b(a[3], "b_slices must be a list of tensors");
  if (tensor(a[1], "hidden").scalar_type() != at::kBFloat16 || pool.scalar_type() != at::kBFloat16)
    raise(PyExc_TypeError, "hidden states and adapters must be bfloat16");
  const void* hidden = address(a[1], "hidden", at::kBFloat16, {in.R, H}, in.device);
  const void* pool_at = address(a[2], "a", at::kBFloat16, {adapters, rank, H}, in.device);
  if (b.size != in.S) raise(PyExc_ValueError, "b_slices must hold %d slices", in.S);
  Addresses b_at;
  b_at.reserve(in.S);
  for (int s = 0; s < in.S; ++s) {
    if (tensor(b[s], "b_slices").scalar_type() != at::kBFloat16)
      raise(PyExc_TypeError, "hidden states and adapters must be bfloat16");
    b_at.push_back(address(b[s], "b_slices", at::kBFloat16, {adapters, in.V_s, rank}, in.device));
  }
  const void* ids = address(a[4], "adapter_ids", at::kInt, {in.R}, in.device);
  const void* scale = address(a[5], "scale", at::kFloat, {adapters}, in.device, true);
  need_cuda(in.device);
  const Launch launch(a[9], in.device);
  OutSlices out(a[6], "out", at::kFloat, false, in);
  void* stats = a[7] == Py_None ? nullptr
                                : address(a[7], "tile_stats", at::kFloat,
                                          {in.R, static_cast<int64_t>(in.S) * ((in.V_s + 127) / 128), 8}, in.device);
  at::Tensor workspace;
  if (a[8] != Py_None) {
    workspace = tensor(a[8], "workspace");
    if (workspace.scalar_type() != at::kByte || !workspace.is_contiguous() || workspace.device() != in.device)
      raise(PyExc_ValueError, "workspace must be a contiguous uint8 tensor on %s", in.device.str().c_str());
  } else {
    workspace = empty({static_cast<int64_t>(vsl_adapters_workspace_bytes(in.R, adapters, rank))}, at::kByte, in.device);
  }
  check_status(vsl_adapters_add(in.logits(), reinterpret_cast<float* const*>(out.at.data()), hidden, in.R, H, in.S,
                                in.V_s, pool_at, b_at.data(), static_cast<const float*>(scale), adapters, rank,
                                static_cast<const int32_t*>(ids), static_cast<float*>(stats), workspace.data_ptr(),
                                static_cast<size_t>(workspace.numel()), launch.stream()),
               "vsl_adapters_add");
  return out.take();
}

// No C++ exception leaves an entry point.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  // outputs and their views are made without the bookkeeping of gradients (a
  // microsecond of a small call)
  const at::AutoDispatchBelowADInplaceOrView no_grad;
  try {
    return F(args, n);
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyObject* set_error_class(PyObject*, PyObject* c) {
  Py_INCREF(c);
  Py_XSETREF(g_error_class, c);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F>));
}

PyMethodDef g_methods[] = {
    {"token_logprobs", fast<token_logprobs>(), METH_FASTCALL, nullptr},
    {"token_logprobs_grad", fast<token_logprobs_grad>(), METH_FASTCALL, nullptr},
    {"policy_loss", fast<policy_loss>(), METH_FASTCALL, nullptr},
    {"preference_loss", fast<preference_loss>(), METH_FASTCALL, nullptr},
    {"adapters_add", fast<adapters_add>(), METH_FASTCALL, nullptr},
    {"set_error_class", set_error_class, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
