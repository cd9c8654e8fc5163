// torch_binding.cpp — the Python side of the operators around the 4-bit layers:
// checks of tensors, allocation of outputs and workspace, and the call of the
// C entry point, in one native step. Only argument marshalling lives here.
//
// Their small calls are bound by the caller: the same steps in Python through
// ctypes cost 9.4 us a call for one vector through gemm_mxfp4_few, 11.2 for four
// through quantize_mxfp4_act; here 4.8 and 6.4, of which the C entry point and
// its launch are 3.6.
//
// Every function takes positional arguments (None where optional), works on
// torch's current stream of the tensors' device, raises TypeError or ValueError
// for tensors that do not fit, and returns the entry point's code as an int
// where that is not 0.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <exception>
#include <initializer_list>
#include <string>

#include "gemm_w4a4.h"

namespace {

using at::ScalarType;
using at::Tensor;

// A Python exception is set; unwinds to the function's end.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& text) {
  PyErr_SetString(type, text.c_str());
  throw Raised{};
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

const char* type_text(ScalarType t) { return c10::toString(t); }

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

// 16-bit floating tensor on a GPU: whether it is binary16 (else bfloat16).
bool half_of(const Tensor& t, const char* name) {
  if (t.scalar_type() != at::kHalf && t.scalar_type() != at::kBFloat16)
    raise(PyExc_TypeError, std::string(name) + " must be bfloat16 or float16, got " + type_text(t.scalar_type()));
  if (!t.is_cuda()) raise(PyExc_ValueError, "tensors must live on a GPU device");
  return t.scalar_type() == at::kHalf;
}

void want(const Tensor& t, const char* name, ScalarType type, std::initializer_list<int64_t> shape, int device) {
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, std::string(name) + " must be " + type_text(type) + ", got " + type_text(t.scalar_type()));
  if (!t.sizes().equals(at::IntArrayRef(shape)))
    raise(PyExc_ValueError, std::string(name) + " must have shape " + shape_text(at::IntArrayRef(shape)) + ", got " + shape_text(t.sizes()));
  if (!t.is_cuda() || t.get_device() != device)
    raise(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", expected cuda:" + std::to_string(device));
  if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
}

// A tensor like `x` (type, shape, device), any strides.
void same_kind(const Tensor& t, const char* name, const Tensor& x, at::IntArrayRef shape) {
  if (t.scalar_type() != x.scalar_type())
    raise(PyExc_TypeError, std::string(name) + " must be " + type_text(x.scalar_type()) + ", got " + type_text(t.scalar_type()));
  if (!t.sizes().equals(shape))
    raise(PyExc_ValueError, std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
  if (t.device() != x.device()) raise(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", expected " + x.device().str());
}

Tensor empty(at::IntArrayRef shape, ScalarType type, const c10::Device& device) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(device));
}

// Given, after a check, or allocated.
Tensor output(PyObject* o, const char* name, std::initializer_list<int64_t> shape, ScalarType type, const c10::Device& device) {
  if (o == Py_None) return empty(at::IntArrayRef(shape), type, device);
  const Tensor& t = tensor(o, name);
  want(t, name, type, shape, device.index());
  return t;
}

// A tensor that the caller gave has been written: for autograd an in-place change, so
// that a backward pass that saved it raises instead of reading the new values.
void written(PyObject* o) {
  if (o == Py_None) return;
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();   // (inference tensors have no version)
}

PyObject* g_stream_of = nullptr;   // torch._C._cuda_getCurrentRawStream

// The device made current for the call, and its current stream.
class OnDevice {
 public:
  explicit OnDevice(const c10::Device& d) : impl_(d.type()), was_(impl_.getDevice()) {
    if (was_ != d) impl_.setDevice(d);
    now_ = d;
    PyObject* i = PyLong_FromLong(d.index());
    PyObject* s = i ? PyObject_CallOneArg(g_stream_of, i) : nullptr;
    Py_XDECREF(i);
    if (!s) throw Raised{};
    stream = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    if (PyErr_Occurred()) throw Raised{};
  }
  ~OnDevice() {
    if (was_ != now_) impl_.uncheckedSetDevice(was_);
  }
  void* stream = nullptr;

 private:
  c10::impl::VirtualGuardImpl impl_;
  c10::Device was_, now_{c10::DeviceType::CPU};
};

int dim_of(int64_t n, const char* name) {
  if (n > INT32_MAX) raise(PyExc_ValueError, std::string(name) + " is too large");
  return int(n);
}

template <class T>
T* ptr(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }

// ---------------------------------------------------------------- the operators

PyObject* quantize(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const bool f16 = half_of(x, "x");
  if (x.dim() != 2) raise(PyExc_ValueError, "x must be 2-D");
  if (!x.is_contiguous()) raise(PyExc_ValueError, "x must be contiguous");
  const c10::Device device = x.device();
  const int M = dim_of(x.size(0), "x"), K = dim_of(x.size(1), "x");
  int R = 0;
  const void* down = nullptr;
  if (a[1] != Py_None) {
    const Tensor& d = tensor(a[1], "lora_down");
    if (d.dim() != 2) raise(PyExc_ValueError, "lora_down must be 2-D");
    R = dim_of(d.size(0), "lora_down");
    want(d, "lora_down", x.scalar_type(), {R, K}, device.index());
    down = R ? d.data_ptr() : nullptr;
  }
  const Tensor act = output(a[2], "act", {M, K / 2}, at::kByte, device);
  const Tensor scales = output(a[3], "ascales", {K / 32, M}, at::kByte, device);
  Tensor low;
  if (R > 0) low = output(a[4], "lora_act_in", {M, R}, x.scalar_type(), device);
  const OnDevice on(device);
  const int64_t need = quantize_mxfp4_workspace(M, K, R);
  if (need < 0) return PyLong_FromLong(long(need));
  Tensor ws;
  if (need > 0) ws = empty({need}, at::kByte, device);
  const int rc = (f16 ? quantize_mxfp4_act_f16 : quantize_mxfp4_act)(
      ptr<uint16_t>(x), static_cast<const uint16_t*>(down), ptr<uint8_t>(act), ptr<uint8_t>(scales),
      R > 0 ? ptr<uint16_t>(low) : nullptr, M, K, R, need > 0 ? ws.data_ptr() : nullptr, need, on.stream);
  if (rc != GEMM_W4A4_OK) return PyLong_FromLong(rc);
  written(a[2]);
  written(a[3]);
  if (R > 0) written(a[4]);
  PyObject* r = PyTuple_New(3);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, wrap(act));
  PyTuple_SET_ITEM(r, 1, wrap(scales));
  PyTuple_SET_ITEM(r, 2, R > 0 ? wrap(low) : Py_NewRef(Py_None));
  return r;
}

// Scale bytes as uint8 or float8_e8m0fnu.
const Tensor& scale_bytes(PyObject* o, const char* name, int64_t blocks, int64_t rows, int device) {
  const Tensor& t = tensor(o, name);
  want(t, name, t.scalar_type() == ScalarType::Float8_e8m0fnu ? ScalarType::Float8_e8m0fnu : at::kByte, {blocks, rows}, device);
  return t;
}

PyObject* few(PyObject* const* a) {
  const Tensor& act = tensor(a[0], "act");
  const Tensor& wgt = tensor(a[2], "wgt");
  if (!act.is_cuda()) raise(PyExc_ValueError, "tensors must live on a GPU device");
  if (act.dim() != 2 || wgt.dim() != 2) raise(PyExc_ValueError, "act and wgt must be 2-D");
  const c10::Device device = act.device();
  const int index = device.index();
  const int M = dim_of(act.size(0), "act"), N = dim_of(wgt.size(0), "wgt");
  const int64_t half = act.size(1);
  const int K = dim_of(2 * half, "act");
  want(act, "act", at::kByte, {M, half}, index);
  want(wgt, "wgt", at::kByte, {N, half}, index);
  const Tensor& as = scale_bytes(a[1], "ascales", half / 16, M, index);
  const Tensor& ws = scale_bytes(a[3], "wscales", half / 16, N, index);
  const Tensor& wc = tensor(a[4], "wcscale");
  const Tensor& bias = tensor(a[5], "bias");
  want(wc, "wcscale", at::kFloat, {N}, index);
  want(bias, "bias", at::kFloat, {N}, index);
  if ((a[6] == Py_None) != (a[7] == Py_None)) raise(PyExc_ValueError, "lora_act_in and lora_up go together");
  // the 16-bit type: dtype, else that of out, else of lora_act_in, else bfloat16
  ScalarType type = at::kBFloat16;
  if (a[9] != Py_None) {
    if (!THPDtype_Check(a[9])) raise(PyExc_TypeError, "dtype must be a torch.dtype");
    type = reinterpret_cast<THPDtype*>(a[9])->scalar_type;
  } else if (a[8] != Py_None) {
    type = tensor(a[8], "out").scalar_type();
  } else if (a[6] != Py_None) {
    type = tensor(a[6], "lora_act_in").scalar_type();
  }
  if (type != at::kBFloat16 && type != at::kHalf)
    raise(PyExc_TypeError, std::string("the LoRA/output type must be bfloat16 or float16, got ") + type_text(type));
  int R = 0;
  const uint16_t *la = nullptr, *lu = nullptr;
  if (a[6] != Py_None) {
    const Tensor& l = tensor(a[6], "lora_act_in");
    const Tensor& u = tensor(a[7], "lora_up");
    if (l.dim() != 2) raise(PyExc_ValueError, "lora_act_in must be 2-D");
    R = dim_of(l.size(1), "lora_act_in");
    want(l, "lora_act_in", type, {M, R}, index);
    want(u, "lora_up", type, {R, N}, index);
    la = ptr<uint16_t>(l);
    lu = ptr<uint16_t>(u);
  }
  const Tensor out = output(a[8], "out", {M, N}, type, device);
  const OnDevice on(device);
  const int rc = (type == at::kHalf ? gemm_mxfp4_few_f16 : gemm_mxfp4_few)(
      ptr<uint8_t>(act), ptr<uint8_t>(as), ptr<uint8_t>(wgt), ptr<uint8_t>(ws), ptr<float>(wc), ptr<float>(bias), la, lu,
      ptr<uint16_t>(out), M, N, K, R, on.stream);
  if (rc != GEMM_W4A4_OK) return PyLong_FromLong(rc);
  written(a[8]);
  return wrap(out);
}

void outer_strides(int64_t (&to)[3], const Tensor& t, const char* name) {
  if (t.size(3) > 1 && t.stride(3) != 1) raise(PyExc_ValueError, std::string("the last dimension of ") + name + " must be dense");
  for (int i = 0; i < 3; ++i) to[i] = t.stride(i);
}

bool truth(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw Raised{};
  return r != 0;
}

PyObject* rotary(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const Tensor& pos = tensor(a[1], "positions");
  const Tensor& freq = tensor(a[2], "inv_freq");
  rotary_axes_t r{};
  PyObject* seq = PySequence_Fast(a[3], "sections must be a sequence");
  if (!seq) throw Raised{};
  const Py_ssize_t axes = PySequence_Fast_GET_SIZE(seq);
  int64_t pairs = 0;
  bool fit = true;   // every section in 0 .. INT32_MAX
  for (Py_ssize_t i = 0; i < axes && i < ROTARY_AXES_MAX && fit; ++i) {
    int past = 0;    // sign of what long does not hold
    const long n = PyLong_AsLongAndOverflow(PySequence_Fast_GET_ITEM(seq, i), &past);
    fit = past == 0 && n >= 0 && n <= INT32_MAX;
    r.sections[i] = fit ? int(n) : 0;
    pairs += r.sections[i];
  }
  Py_DECREF(seq);
  if (PyErr_Occurred()) throw Raised{};
  if (axes < 1 || axes > ROTARY_AXES_MAX)
    raise(PyExc_ValueError, "1 to " + std::to_string(ROTARY_AXES_MAX) + " axes, got " + std::to_string(axes));
  if (!fit) raise(PyExc_ValueError, "sections must be 0 or more pairs each, below 2^31");
  r.f16 = half_of(x, "x");
  if (x.dim() != 4) raise(PyExc_ValueError, "x must be [batch, tokens, heads, head_dim]");
  r.batch = dim_of(x.size(0), "x");
  r.tokens = dim_of(x.size(1), "x");
  r.heads = dim_of(x.size(2), "x");
  r.head_dim = dim_of(x.size(3), "x");
  r.axes = int(axes);
  if (pos.scalar_type() != at::kInt || freq.scalar_type() != at::kFloat)
    raise(PyExc_TypeError, "positions must be int32 and inv_freq float32");
  const bool per_batch = pos.sizes().equals({r.batch, r.tokens, axes});
  if (!per_batch && !pos.sizes().equals({r.tokens, axes}))
    raise(PyExc_ValueError, "positions must be " + shape_text({r.batch, r.tokens, axes}) + " or " + shape_text({r.tokens, axes}) +
                                ", got " + shape_text(pos.sizes()));
  if (!freq.sizes().equals({pairs}) || !freq.is_contiguous())
    raise(PyExc_ValueError, "inv_freq must be contiguous, one value per pair");
  if (pos.device() != x.device() || freq.device() != x.device())
    raise(PyExc_ValueError, "positions and inv_freq must be on " + x.device().str());
  if (axes > 1 && pos.stride(-1) != 1) raise(PyExc_ValueError, "the last dimension of positions must be dense");
  r.pos_stride[0] = per_batch ? pos.stride(0) : 0;
  r.pos_stride[1] = pos.stride(per_batch ? 1 : 0);
  r.interleaved = truth(a[4]);
  r.inverse = truth(a[5]);
  Tensor out;
  if (a[6] == Py_None) {
    out = empty(x.sizes(), x.scalar_type(), x.device());
  } else {
    out = tensor(a[6], "out");
    same_kind(out, "out", x, x.sizes());
  }
  outer_strides(r.x_stride, x, "x");
  outer_strides(r.out_stride, out, "out");
  r.x = x.data_ptr();
  r.out = out.data_ptr();
  r.positions = ptr<int32_t>(pos);
  r.inv_freq = ptr<float>(freq);
  const OnDevice on(x.device());
  const int rc = rotary_axes(&r, on.stream);
  if (rc != GEMM_W4A4_OK) return PyLong_FromLong(rc);
  written(a[6]);
  return wrap(out);
}

PyObject* attention(PyObject* const* a) {
  const Tensor& q = tensor(a[0], "q");
  const Tensor& k = tensor(a[1], "k");
  const Tensor& v = tensor(a[2], "v");
  cross_attention_t c{};
  c.f16 = half_of(q, "q");
  if (q.dim() != 4 || k.dim() != 4) raise(PyExc_ValueError, "q, k and v must be 4-D");
  const c10::Device device = q.device();
  c.batch = dim_of(q.size(0), "q");
  c.q_len = dim_of(q.size(1), "q");
  c.q_heads = dim_of(q.size(2), "q");
  c.head_dim = dim_of(q.size(3), "q");
  c.kv_len = dim_of(k.size(1), "k");
  c.kv_heads = dim_of(k.size(2), "k");
  const int64_t keys[4] = {c.batch, c.kv_len, c.kv_heads, c.head_dim};
  same_kind(k, "k", q, keys);
  same_kind(v, "v", q, keys);
  if (a[3] != Py_None) {
    const Tensor& lens = tensor(a[3], "kv_lens");
    want(lens, "kv_lens", at::kInt, {c.batch}, device.index());
    c.kv_lens = ptr<int32_t>(lens);
  }
  c.scale = a[4] == Py_None ? float(1.0 / std::sqrt(double(c.head_dim))) : float(PyFloat_AsDouble(a[4]));
  if (PyErr_Occurred()) throw Raised{};
  Tensor out;
  if (a[6] == Py_None) {
    out = empty(q.sizes(), q.scalar_type(), device);
  } else {
    out = tensor(a[6], "out");
    same_kind(out, "out", q, q.sizes());
  }
  Tensor lse;
  if (truth(a[5])) {
    lse = empty({c.batch, c.q_heads, c.q_len}, at::kFloat, device);
    c.lse = ptr<float>(lse);
  }
  outer_strides(c.q_stride, q, "q");
  outer_strides(c.k_stride, k, "k");
  outer_strides(c.v_stride, v, "v");
  outer_strides(c.out_stride, out, "out");
  c.q = q.data_ptr();
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.out = out.data_ptr();
  const OnDevice on(device);
  c.workspace_bytes = cross_attention_workspace(&c);
  if (c.workspace_bytes < 0) return PyLong_FromLong(long(c.workspace_bytes));
  Tensor ws;
  if (c.workspace_bytes > 0) {
    ws = empty({c.workspace_bytes}, at::kByte, device);
    c.workspace = ws.data_ptr();
  }
  const int rc = cross_attention(&c, on.stream);
  if (rc != GEMM_W4A4_OK) return PyLong_FromLong(rc);
  written(a[6]);
  if (!lse.defined()) return wrap(out);
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, wrap(out));
  PyTuple_SET_ITEM(r, 1, wrap(lse));
  return r;
}

// ---------------------------------------------------------------- the module

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
    return nullptr;
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());   // as torch's own calls raise
  }
  return nullptr;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<quantize, 5>("quantize_mxfp4_act"),   // x, lora_down, act, ascales, lora_act_in
    method<few, 10>("gemm_mxfp4_few"),           // act .. lora_up, out, dtype
    method<rotary, 7>("rotary_axes"),            // x, positions, inv_freq, sections, interleaved, inverse, out
    method<attention, 7>("cross_attention"),     // q, k, v, kv_lens, scale, return_lse, out
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_binding() {
  PyObject* c = PyImport_ImportModule("torch._C");
  if (!c) return nullptr;
  g_stream_of = PyObject_GetAttrString(c, "_cuda_getCurrentRawStream");
  Py_DECREF(c);
  return g_stream_of ? PyModule_Create(&g_module) : nullptr;
}
