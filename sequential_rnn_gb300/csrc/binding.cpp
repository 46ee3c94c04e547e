// Python calls of the language-model operators: checks of the tensors, the
// outputs' and workspace's allocation on the current stream, the C entry point.
//
// Written against PyTorch's C++ interface because the calls of single tokens are bound by
// what the host does: marshalled in Python (three allocations, five checked tensors, ctypes) a norm
// of 16 rows took 15.7 us, of which 3.2 were the C call with its launch; here 6.
// A call returns its tensors, or the entry point's status where that is not RNN_OK.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstring>
#include <string>

#include "rnn.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;
typedef c10::SmallVector<int64_t, 6> Shape;

// The library's entry points: set once by connect(), from the handle that the package loaded.
struct {
  decltype(&rnn_rms_norm) norm;
  decltype(&rnn_rms_norm_bwd_workspace_size) norm_bwd_ws;
  decltype(&rnn_rms_norm_bwd) norm_bwd;
  decltype(&rnn_quantize_weight) quantize;
  decltype(&rnn_input_proj_fp8) proj;
  decltype(&rnn_linattn_workspace_size) la_ws;
  decltype(&rnn_linattn_fwd) la_fwd;
  decltype(&rnn_linattn_bwd) la_bwd;
  decltype(&rnn_linattn_step) la_step;
} api;

constexpr int64_t kBlock = 128;  // columns (and weight rows) that share a scale
constexpr ScalarType kE4m3 = at::kFloat8_e4m3fn;

// (raised with the GIL held)
[[noreturn]] void fail(PyObject* type, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw python_error();
}
const char* type_name(ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kInt: return "torch.int32";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return c10::toString(t);
  }
}

const Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s: expected a torch.Tensor", name);
  return THPVariable_Unpack(o);
}
const Tensor* optional(const char* name, PyObject* o) { return o == Py_None ? nullptr : &tensor(name, o); }
template <class T = void>
T* at_of(const Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

std::string text(IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

// the leading operand's device, which has to be the current one
at::Device device_of(const char* name, const Tensor& t) {
  if (!t.is_cuda()) fail(PyExc_ValueError, "%s: tensor must live on a CUDA device", name);
  if (t.device().index() != c10::cuda::current_device())
    fail(PyExc_ValueError, "%s: tensor must live on the current CUDA device", name);
  return t.device();
}
int dtype_of(const char* name, const Tensor& t) {
  if (t.scalar_type() == at::kFloat) return RNN_F32;
  if (t.scalar_type() == at::kBFloat16) return RNN_BF16;
  fail(PyExc_TypeError, "%s: unsupported dtype %s", name, type_name(t.scalar_type()));
}
void want(const char* name, const Tensor& t, IntArrayRef shape, ScalarType type, at::Device dev,
          bool contiguous = true) {
  if (t.scalar_type() != type)
    fail(PyExc_TypeError, "%s: expected %s, got %s", name, type_name(type), type_name(t.scalar_type()));
  if (t.sizes() != shape)
    fail(PyExc_ValueError, "%s: expected shape %s, got %s", name, text(shape).c_str(), text(t.sizes()).c_str());
  if (t.device() != dev)
    fail(PyExc_ValueError, "%s: expected a tensor on %s, got %s", name, dev.str().c_str(), t.device().str().c_str());
  if (contiguous && !t.is_contiguous()) fail(PyExc_ValueError, "%s: tensor must be contiguous", name);
}
void want(const char* name, const Tensor* t, IntArrayRef shape, ScalarType type, at::Device dev) {
  if (t) want(name, *t, shape, type, dev);
}
int32_t count(const char* name, int64_t n) {
  if (n > INT32_MAX) fail(PyExc_ValueError, "%s: a size of more than 2^31 - 1", name);
  return (int32_t)n;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v == 1;
}

Tensor make(IntArrayRef shape, ScalarType type, at::Device dev) {
  return Tensor(at::detail::empty_cuda(shape, type, dev, std::nullopt));
}
void* current_stream() { return c10::cuda::getCurrentCUDAStream().stream(); }

// allocations and the launch may wait for the device: other Python threads go on meanwhile
struct NoGil {
  PyThreadState* s = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(s); }
};

PyObject* status(int st) { return PyLong_FromLong(st); }
void put(PyObject* d, const char* key, PyObject* value) {  // (takes over the reference)
  PyObject* k = PyUnicode_InternFromString(key);
  PyDict_SetItem(d, k, value);
  Py_DECREF(k);
  Py_DECREF(value);
}
void put(PyObject* d, const char* key, const Tensor& t) { put(d, key, THPVariable_Wrap(t)); }

PyObject* pair(const Tensor& a, const Tensor& b) {
  PyObject* t = PyTuple_New(2);
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
  return t;
}

void arity(const char* name, Py_ssize_t n, Py_ssize_t expected) {
  if (n != expected) fail(PyExc_TypeError, "%s: expected %zd arguments, got %zd", name, expected, n);
}

// ------------------------------------------------------------------ norm --
// x, weight, residual or None, eps, quantize, train
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity("rms_norm", n, 6);
  const Tensor &x = tensor("x", a[0]), &weight = tensor("weight", a[1]);
  const Tensor* residual = optional("residual", a[2]);
  const float eps = (float)number(a[3]);
  const bool quantize = truth(a[4]), train = truth(a[5]);
  const at::Device dev = device_of("x", x);
  const int dt = dtype_of("x", x);
  if (x.dim() == 0) fail(PyExc_ValueError, "x: expected at least one dimension");
  const IntArrayRef shape = x.sizes(), lead = shape.slice(0, shape.size() - 1);
  const int64_t N = shape.back();
  want("x", x, shape, x.scalar_type(), dev);
  want("weight", weight, {N}, at::kFloat, dev);
  want("residual", residual, shape, x.scalar_type(), dev);
  const int32_t rows = count("x", N ? x.numel() / N : 0), cols = count("x", N);
  Tensor h, y, scale, rstd;
  int st;
  {
    NoGil free;
    if (residual) h = make(shape, x.scalar_type(), dev);
    y = make(shape, quantize ? kE4m3 : x.scalar_type(), dev);
    if (quantize) {
      Shape s(lead.begin(), lead.end());
      s.push_back((N + kBlock - 1) / kBlock);
      scale = make(s, at::kFloat, dev);
    }
    if (train) rstd = make(lead, at::kFloat, dev);
    st = api.norm(dt, rows, cols, eps, x.data_ptr(), at_of(residual), at_of<const float>(&weight),
                  residual ? h.data_ptr() : nullptr, y.data_ptr(), quantize ? at_of<float>(&scale) : nullptr,
                  train ? at_of<float>(&rstd) : nullptr, current_stream());
  }
  if (st) return status(st);
  PyObject* out = PyDict_New();
  if (residual)
    put(out, "h", h);
  else
    put(out, "h", Py_NewRef(a[0]));
  if (quantize) put(out, "scale", scale);
  if (train) put(out, "rstd", rstd);
  put(out, "y", y);
  return out;
  END_HANDLE_TH_ERRORS
}

// dy, h, weight, rstd, dh or None
PyObject* rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity("rms_norm_backward", n, 5);
  const Tensor &dy = tensor("dy", a[0]), &h = tensor("h", a[1]), &weight = tensor("weight", a[2]),
               &rstd = tensor("rstd", a[3]);
  const Tensor* dh = optional("dh", a[4]);
  const at::Device dev = device_of("h", h);
  const int dt = dtype_of("h", h);
  if (h.dim() == 0) fail(PyExc_ValueError, "h: expected at least one dimension");
  const IntArrayRef shape = h.sizes();
  const int64_t N = shape.back();
  want("h", h, shape, h.scalar_type(), dev);
  want("dy", dy, shape, h.scalar_type(), dev);
  want("weight", weight, {N}, at::kFloat, dev);
  want("rstd", rstd, shape.slice(0, shape.size() - 1), at::kFloat, dev);
  want("dh", dh, shape, h.scalar_type(), dev);
  const int32_t rows = count("h", N ? h.numel() / N : 0), cols = count("h", N);
  Tensor dx, dw, ws;
  int st;
  {
    NoGil free;
    const size_t bytes = api.norm_bwd_ws(rows, cols);
    dx = make(shape, h.scalar_type(), dev);
    dw = make({N}, at::kFloat, dev);
    ws = make({(int64_t)bytes}, at::kByte, dev);
    st = api.norm_bwd(dt, rows, cols, dy.data_ptr(), h.data_ptr(), at_of<const float>(&weight),
                      at_of<const float>(&rstd), at_of(dh), dx.data_ptr(), at_of<float>(&dw), ws.data_ptr(), bytes,
                      current_stream());
  }
  if (st) return status(st);
  PyObject* out = PyDict_New();
  put(out, "dx", dx);
  put(out, "dw", dw);
  return out;
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------ projection --
// W
PyObject* quantize_weight(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity("quantize_weight", n, 1);
  const Tensor& W = tensor("W", a[0]);
  const at::Device dev = device_of("W", W);
  const int dt = dtype_of("W", W);
  if (W.dim() != 2) fail(PyExc_ValueError, "W: expected [N, K]");
  want("W", W, W.sizes(), W.scalar_type(), dev);
  const int32_t N = count("W", W.size(0)), K = count("W", W.size(1));
  Tensor Wq, Ws;
  int st;
  {
    NoGil free;
    Wq = make(W.sizes(), kE4m3, dev);
    Ws = make({(N + kBlock - 1) / kBlock, (K + kBlock - 1) / kBlock}, at::kFloat, dev);
    st = api.quantize(dt, N, K, W.data_ptr(), Wq.data_ptr(), at_of<float>(&Ws), current_stream());
  }
  if (st) return status(st);
  return pair(Wq, Ws);
  END_HANDLE_TH_ERRORS
}

// xq, xs, Wq, Ws, bias or None -> (y, workspace)
PyObject* input_proj_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity("input_proj_fp8", n, 5);
  const Tensor &xq = tensor("xq", a[0]), &xs = tensor("xs", a[1]), &Wq = tensor("Wq", a[2]), &Ws = tensor("Ws", a[3]);
  const Tensor* bias = optional("bias", a[4]);
  const at::Device dev = device_of("xq", xq);
  if (xq.dim() < 1 || Wq.dim() != 2) fail(PyExc_ValueError, "expected xq [..., K] and Wq [N, K]");
  const IntArrayRef lead = xq.sizes().slice(0, xq.dim() - 1);
  const int64_t K = xq.sizes().back(), N = Wq.size(0), kb = (K + kBlock - 1) / kBlock;
  Shape s(lead.begin(), lead.end());
  s.push_back(kb);
  want("xq", xq, xq.sizes(), kE4m3, dev);
  want("xs", xs, s, at::kFloat, dev);
  want("Wq", Wq, {N, K}, kE4m3, dev);
  want("Ws", Ws, {(N + kBlock - 1) / kBlock, kb}, at::kFloat, dev);
  want("bias", bias, {N}, at::kFloat, dev);
  const int32_t rows = count("xq", K ? xq.numel() / K : 0), n32 = count("Wq", N), k32 = count("xq", K);
  s.back() = N;
  Tensor y, ws;
  int st;
  {
    NoGil free;
    y = make(s, at::kBFloat16, dev);
    ws = make({256}, at::kByte, dev);
    st = api.proj(rows, n32, k32, xq.data_ptr(), at_of<const float>(&xs), Wq.data_ptr(),
                  at_of<const float>(&Ws), at_of<const float>(bias), y.data_ptr(), ws.data_ptr(), 256,
                  current_stream());
  }
  if (st) return status(st);
  return pair(y, ws);
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------ linear attention --
struct Attention {
  rnn_linattn_desc_t desc;
  rnn_linattn_strides_t strides;
  bool strided = false;
  at::Device dev;
  ScalarType type;
  int64_t T, B, NH, Dk, Dv;
  const rnn_linattn_strides_t* st() const { return strided ? &strides : nullptr; }

  // lead: dimensions before the heads' (2: [T, B, NH, D], 1: [B, NH, D]); out: strided as the outputs are, or null
  Attention(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& g, PyObject* scale, int lead,
            const Tensor* out)
      : dev(device_of("q", q)), type(q.scalar_type()) {
    const int dt = dtype_of("q", q);
    if (q.dim() != lead + 2 || v.dim() != lead + 2)
      fail(PyExc_ValueError, "expected q, k, v of shape %s", lead == 2 ? "[T, B, NH, D]" : "[B, NH, D]");
    T = lead == 2 ? q.size(0) : 1, B = q.size(lead - 1), NH = q.size(lead), Dk = q.size(lead + 1),
    Dv = v.size(lead + 1);
    Shape sv(q.sizes().begin(), q.sizes().end());
    sv.back() = Dv;
    want("k", k, q.sizes(), type, dev, false);
    want("v", v, sv, type, dev, false);
    want("log_decay", g, {NH}, at::kFloat, dev);
    if (out) want("do", *out, {T, B, NH, Dv}, type, dev, false);
    desc = {};
    desc.dtype = dt;
    desc.T = count("q", T), desc.B = count("q", B), desc.NH = count("q", NH), desc.Dk = count("q", Dk);
    desc.Dv = count("v", Dv);
    desc.scale = (float)(scale == Py_None ? std::pow((double)(Dk > 0 ? Dk : 1), -0.5) : number(scale));
    if (q.is_contiguous() && k.is_contiguous() && v.is_contiguous() && (!out || out->is_contiguous())) return;
    strided = true;
    strides_of("q", q, strides.q);
    strides_of("k", k, strides.k);
    strides_of("v", v, strides.v);
    if (out)
      strides_of("do", *out, strides.o);
    else
      strides.o[0] = B * NH * Dv, strides.o[1] = NH * Dv, strides.o[2] = Dv;
  }
  static void strides_of(const char* name, const Tensor& t, int64_t (&s)[3]) {
    if (t.strides().back() != 1) fail(PyExc_ValueError, "%s: the last dimension must be contiguous", name);
    s[0] = 0;
    for (int i = 3 - (int)t.dim() + 1, d = 0; i < 3; ++i, ++d)
      s[i] = t.size(d) > 1 ? t.stride(d) : 0;  // (a dimension of one element has no stride to speak of)
  }
  size_t workspace(int pass) const {
    const size_t n = api.la_ws(&desc, pass);
    return n > 256 ? n : 256;
  }
  Tensor tokens(int64_t D) const { return make({T, B, NH, D}, type, dev); }
  Tensor states() const { return make({B, NH, Dk, Dv}, at::kFloat, dev); }
  void want_state(const char* name, const Tensor* t) const { want(name, t, {B, NH, Dk, Dv}, at::kFloat, dev); }
};

// q, k, v, log_decay, state or None, lens or None, scale or None
PyObject* linear_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity("linear_attention", n, 7);
  const Tensor &q = tensor("q", a[0]), &k = tensor("k", a[1]), &v = tensor("v", a[2]), &g = tensor("log_decay", a[3]);
  const Tensor *state = optional("state", a[4]), *lens = optional("lens", a[5]);
  const Attention la(q, k, v, g, a[6], 2, nullptr);
  la.want_state("state", state);
  want("lens", lens, {la.B}, at::kInt, la.dev);
  Tensor o, fin, ws;
  int st;
  {
    NoGil free;
    const size_t bytes = la.workspace(0);
    o = la.tokens(la.Dv), fin = la.states(), ws = make({(int64_t)bytes}, at::kByte, la.dev);
    st = api.la_fwd(&la.desc, la.st(), q.data_ptr(), k.data_ptr(), v.data_ptr(), at_of<const float>(&g),
                    at_of<const int32_t>(lens), at_of<const float>(state), o.data_ptr(), at_of<float>(&fin),
                    ws.data_ptr(), bytes, current_stream());
  }
  if (st) return status(st);
  PyObject* out = PyDict_New();
  put(out, "o", o);
  put(out, "state", fin);
  put(out, "workspace", ws);
  return out;
  END_HANDLE_TH_ERRORS
}

// q, k, v, log_decay, do, state or None, dstate or None, lens or None, scale or None
PyObject* linear_attention_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity("linear_attention_backward", n, 9);
  const Tensor &q = tensor("q", a[0]), &k = tensor("k", a[1]), &v = tensor("v", a[2]), &g = tensor("log_decay", a[3]),
               &dout = tensor("do", a[4]);
  const Tensor *state = optional("state", a[5]), *dstate = optional("dstate", a[6]), *lens = optional("lens", a[7]);
  const Attention la(q, k, v, g, a[8], 2, &dout);
  la.want_state("state", state);
  la.want_state("dstate", dstate);
  want("lens", lens, {la.B}, at::kInt, la.dev);
  Tensor dq, dk, dv, ds0, ws;
  int st;
  {
    NoGil free;
    const size_t bytes = la.workspace(1);
    dq = la.tokens(la.Dk), dk = la.tokens(la.Dk), dv = la.tokens(la.Dv), ds0 = la.states();
    ws = make({(int64_t)bytes}, at::kByte, la.dev);
    st = api.la_bwd(&la.desc, la.st(), q.data_ptr(), k.data_ptr(), v.data_ptr(), at_of<const float>(&g),
                    at_of<const int32_t>(lens), at_of<const float>(state), dout.data_ptr(),
                    at_of<const float>(dstate), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), at_of<float>(&ds0),
                    ws.data_ptr(), bytes, current_stream());
  }
  if (st) return status(st);
  PyObject* out = PyDict_New();
  put(out, "dq", dq);
  put(out, "dk", dk);
  put(out, "dv", dv);
  put(out, "dstate", ds0);
  put(out, "workspace", ws);
  return out;
  END_HANDLE_TH_ERRORS
}

// q, k, v, log_decay, state, slots or None, scale or None
PyObject* linear_attention_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity("linear_attention_step", n, 7);
  const Tensor &q = tensor("q", a[0]), &k = tensor("k", a[1]), &v = tensor("v", a[2]), &g = tensor("log_decay", a[3]);
  const Attention la(q, k, v, g, a[6], 1, nullptr);
  if (!THPVariable_Check(a[4]) || THPVariable_Unpack(a[4]).dim() != 4)
    fail(PyExc_ValueError, "state: expected [n_slots, NH, Dk, Dv]");
  const Tensor &state = THPVariable_Unpack(a[4]), *slots = optional("slots", a[5]);
  want("state", state, {state.size(0), la.NH, la.Dk, la.Dv}, at::kFloat, la.dev);
  want("slots", slots, {la.B}, at::kInt, la.dev);
  const int32_t n_slots = count("state", state.size(0));
  Tensor o;
  int st;
  {
    NoGil free;
    o = make({la.B, la.NH, la.Dv}, la.type, la.dev);
    st = api.la_step(&la.desc, la.st(), q.data_ptr(), k.data_ptr(), v.data_ptr(), at_of<const float>(&g),
                     at_of<const int32_t>(slots), n_slots, at_of<float>(&state), o.data_ptr(),
                     current_stream());
  }
  return st ? status(st) : THPVariable_Wrap(o);
  END_HANDLE_TH_ERRORS
}

// the entry points' addresses, in the order of `api`
PyObject* connect(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  void* p[sizeof(api) / sizeof(void*)];
  arity("connect", n, sizeof(p) / sizeof(p[0]));
  for (Py_ssize_t i = 0; i < n; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) fail(PyExc_ValueError, "connect: null entry point");
  }
  memcpy(&api, p, sizeof(api));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define CALL(name) {#name, (PyCFunction)(void (*)())name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(rms_norm), CALL(rms_norm_backward), CALL(quantize_weight), CALL(input_proj_fp8),
                         CALL(linear_attention), CALL(linear_attention_backward), CALL(linear_attention_step),
                         CALL(connect), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__binding() { return PyModule_Create(&module); }
