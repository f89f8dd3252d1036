// Argument marshalling of the layer operators' Python functions: checks the
// tensors, allocates outputs, fills the descriptor and makes one call of the
// C ABI. A step of one token takes about 3 us on the GPU; the same work in
// Python with ctypes took 13 us on the host, and takes 5.6 here. Nothing is
// computed here, and nothing is kept from one call to the next.
//
// The library is not linked: bind() takes the addresses of its functions, so
// the extension follows whichever build binding.py has loaded.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/ssd.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

struct Library {
  decltype(&ssd_selective_scan_workspace_bytes) workspace_bytes;
  decltype(&ssd_selective_scan) scan;
  decltype(&ssd_selective_scan_varlen) scan_varlen;
  decltype(&ssd_selective_step) step;
  decltype(&ssd_conv1d) conv;
  decltype(&ssd_conv1d_step) conv_step;
  decltype(&ssd_group_norm) norm;
  PyObject* error;  // SSDError
};
Library lib{};

using Dims = c10::SmallVector<int64_t, 4>;

std::string text(IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}
std::string text(ScalarType t) {
  if (t == at::kFloat) return "torch.float32";
  if (t == at::kBFloat16) return "torch.bfloat16";
  if (t == at::kInt) return "torch.int32";
  return c10::toString(t);
}

[[noreturn]] void bad_value(const std::string& s) {
  PyErr_SetString(PyExc_ValueError, s.c_str());
  throw python_error();
}
[[noreturn]] void bad_type(const std::string& s) {
  PyErr_SetString(PyExc_TypeError, s.c_str());
  throw python_error();
}

// A tensor argument; null for None.
const Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const Tensor& device_tensor(PyObject* o, const char* name, int64_t dims) {
  const Tensor* t = tensor(o, name);
  if (t == nullptr) bad_value(std::string(name) + " is required");
  if (!t->is_cuda()) bad_value(std::string(name) + " must be a device tensor");
  if (dims >= 0 && t->dim() != dims)
    bad_value(std::string(name) + " must have " + std::to_string(dims) + " dimensions, got " + std::to_string(t->dim()));
  return *t;
}

// Type, device and shape as they have to be.
void check(const Tensor& t, const char* name, ScalarType type, c10::Device device, IntArrayRef shape) {
  if (t.scalar_type() != type)
    bad_type(std::string(name) + " must be " + text(type) + ", got " + text(t.scalar_type()));
  if (t.device() != device) bad_value(std::string(name) + " is on " + t.device().str() + ", expected " + device.str());
  if (t.sizes() != shape) bad_value(std::string(name) + " must have shape " + text(shape) + ", got " + text(t.sizes()));
}

// Strides of [batch, tokens, channels..] (lead 2) or [batch, channels..]
// (lead 1); 0 stands for dense.
ssd_stride_t strides(const Tensor& t, const char* name, int64_t lead) {
  if (t.is_contiguous()) return {0, 0};
  const IntArrayRef shape = t.sizes(), st = t.strides();
  int64_t width = 1;
  for (int64_t i = t.dim() - 1; i >= lead; --i) {
    if (shape[i] != 1 && st[i] != width) bad_value(std::string(name) + ": the channels of a token must be contiguous");
    width *= shape[i];
  }
  const int64_t rows = lead == 2 ? shape[1] : 1;
  const int64_t token = rows > 1 ? st[1] : width;
  const int64_t batch = shape[0] > 1 ? st[0] : (rows - 1) * token + width;
  if (token < width || batch < width)
    bad_value(std::string(name) + ": tokens must not overlap (an expanded dimension needs a copy)");
  return {token, batch};
}
ssd_stride_t strided(const Tensor& t, const char* name, ScalarType type, c10::Device device, IntArrayRef shape,
                     int64_t lead) {
  check(t, name, type, device, shape);
  return strides(t, name, lead);
}

// Address of a dense argument; null for None.
void* dense(PyObject* o, const char* name, ScalarType type, c10::Device device, IntArrayRef shape) {
  const Tensor* t = tensor(o, name);
  if (t == nullptr) return nullptr;
  check(*t, name, type, device, shape);
  if (!t->is_contiguous()) bad_value(std::string(name) + " must be contiguous");
  return t->data_ptr();
}
const float* floats(PyObject* o, const char* name, c10::Device device, IntArrayRef shape) {
  return static_cast<const float*>(dense(o, name, at::kFloat, device, shape));
}

// The output given, or a new dense one.
Tensor output(PyObject* o, const char* name, ScalarType type, const Tensor& like, IntArrayRef shape) {
  if (o == Py_None) return at::empty(shape, like.options().dtype(type));
  dense(o, name, type, like.device(), shape);
  return THPVariable_Unpack(o);
}

int32_t io_code(const Tensor& t, const char* name) {
  if (t.scalar_type() == at::kFloat) return SSD_DTYPE_F32;
  if (t.scalar_type() == at::kBFloat16) return SSD_DTYPE_BF16;
  bad_type(std::string(name) + ": unsupported io dtype " + text(t.scalar_type()));
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}
void* handle(PyObject* o) {
  const unsigned long long v = PyLong_AsUnsignedLongLongMask(o);
  if (v == ~0ull && PyErr_Occurred()) throw python_error();
  return reinterpret_cast<void*>(static_cast<uintptr_t>(v));
}

// The interpreter's lock, given up while this lives.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// Makes the call without the interpreter's lock and raises for its status. F
// is the call of the library and nothing else: what asks Python or a tensor
// for something (an address, a stream's handle) needs the lock and may throw,
// so it is taken before.
template <typename F> void call(const char* where, F&& f) {
  ssd_status_t status;
  {
    Unlocked unlocked;
    status = f();
  }
  if (status == SSD_OK) return;
  PyObject* e = PyObject_CallFunction(lib.error, "is", (int)status, where);
  if (e != nullptr) {
    PyErr_SetObject(lib.error, e);
    Py_DECREF(e);
  }
  throw python_error();
}

void need_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) bad_type("expected " + std::to_string(want) + " arguments, got " + std::to_string(n));
}

// (x, dt, A, B, C, z) and the dt preprocessing (bias, softplus, limit).
ssd_selective_desc_t selective_desc(const Tensor& x, PyObject* const* a, PyObject* pre_bias, PyObject* pre_softplus,
                                    PyObject* pre_limit, int64_t lead) {
  const Tensor& dt = device_tensor(a[1], "dt", lead + 1);
  const Tensor& A = device_tensor(a[2], "A", 2);
  const Tensor& B = device_tensor(a[3], "B", lead + 2);
  const Tensor& C = device_tensor(a[4], "C", lead + 2);
  const Tensor* z = tensor(a[6], "z");
  const auto dev = x.device();
  const auto io = x.scalar_type();
  const IntArrayRef shape = x.sizes();
  ssd_selective_desc_t d{};
  d.batch = shape[0];
  d.seqlen = lead == 2 ? shape[1] : 1;
  d.channels = shape[lead];
  d.dstate = A.size(1);
  d.ngroups = B.size(lead);
  d.io_dtype = io_code(x, "x");
  if (dt.scalar_type() != at::kFloat && dt.scalar_type() != io)
    bad_type("dt must be torch.float32 or " + text(io) + ", got " + text(dt.scalar_type()));
  d.dt_dtype = io_code(dt, "dt");
  d.dt_bias = floats(pre_bias, "dt bias", dev, {d.channels});
  d.dt_softplus = truth(pre_softplus);
  if (pre_limit != Py_None) {
    PyObject* lo = PySequence_GetItem(pre_limit, 0);
    PyObject* hi = lo == nullptr ? nullptr : PySequence_GetItem(pre_limit, 1);
    if (hi != nullptr) {
      d.dt_clamp = 1;
      d.dt_min = (float)PyFloat_AsDouble(lo);
      d.dt_max = (float)PyFloat_AsDouble(hi);
    }
    Py_XDECREF(lo);
    Py_XDECREF(hi);
    if (PyErr_Occurred()) throw python_error();
  }
  Dims bc(shape.begin(), shape.begin() + lead);
  bc.push_back(d.ngroups);
  bc.push_back(d.dstate);
  d.x_stride = strides(x, "x", lead);
  d.dt_stride = strided(dt, "dt", dt.scalar_type(), dev, shape, lead);
  if (z != nullptr) d.z_stride = strided(*z, "z", io, dev, shape, lead);
  d.B_stride = strided(B, "B", io, dev, bc, lead);
  d.C_stride = strided(C, "C", io, dev, bc, lead);
  return d;
}

const void* data(PyObject* o) { return o == Py_None ? nullptr : THPVariable_Unpack(o).data_ptr(); }

// Offsets of packed sequences, and their number.
const int32_t* offsets(PyObject* o, c10::Device device, int64_t* num_seqs) {
  *num_seqs = 0;
  const Tensor* t = tensor(o, "cu_seqlens");
  if (t == nullptr) return nullptr;
  if (t->dim() != 1 || t->numel() < 2) bad_value("cu_seqlens must hold num_seqs + 1 offsets, num_seqs >= 1");
  *num_seqs = t->numel() - 1;
  return static_cast<const int32_t*>(dense(o, "cu_seqlens", at::kInt, device, t->sizes()));
}

// x dt A B C D z cu_seqlens init y final want_final workspace bias softplus limit stream -> (y, final, workspace)
PyObject* selective_prompts(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need_args(n, 17);
  const Tensor& x = device_tensor(a[0], "x", 3);
  const auto dev = x.device();
  ssd_selective_desc_t d = selective_desc(x, a, a[13], a[14], a[15], 2);
  int64_t S;
  const int32_t* cu = offsets(a[7], dev, &S);
  if (S > 0 && d.batch != 1) bad_value("packed sequences: x must be [1, T, channels]");
  const int64_t states[] = {S > 0 ? S : d.batch, d.channels, d.dstate};
  const float* A = floats(a[2], "A", dev, {d.channels, d.dstate});
  const float* D = floats(a[5], "D", dev, {d.channels});
  const float* init = floats(a[8], S > 0 ? "init_states" : "init_state", dev, states);
  Tensor y = output(a[9], "y", x.scalar_type(), x, x.sizes());
  Tensor final_state, workspace;
  if (a[10] != Py_None || truth(a[11]))
    final_state = output(a[10], S > 0 ? "final_states" : "final_state", at::kFloat, x, states);
  size_t need = 0;
  call("ssd_selective_scan_workspace_bytes", [&] { return lib.workspace_bytes(&d, S, &need); });
  const Tensor* given = tensor(a[12], "workspace");
  if (given != nullptr) {
    if (!given->is_contiguous() || given->device() != dev || given->nbytes() < need)
      bad_value("workspace needs " + std::to_string(need) + " contiguous bytes on " + dev.str());
    workspace = *given;
  } else if (need > 0) {
    workspace = at::empty({(int64_t)need}, x.options().dtype(at::kByte));
  }
  const void *xp = x.data_ptr(), *dt = data(a[1]), *B = data(a[3]), *C = data(a[4]), *z = data(a[6]);
  void *yp = y.data_ptr(), *stream = handle(a[16]);
  void* ws = workspace.defined() ? workspace.data_ptr() : nullptr;
  const size_t ws_bytes = workspace.defined() ? workspace.nbytes() : 0;
  float* fin = final_state.defined() ? final_state.data_ptr<float>() : nullptr;
  if (S > 0)
    call("ssd_selective_scan_varlen", [&] {
      return lib.scan_varlen(&d, cu, S, xp, dt, A, B, C, D, z, init, yp, fin, ws, ws_bytes, stream);
    });
  else
    call("ssd_selective_scan", [&] {
      return lib.scan(&d, xp, dt, A, B, C, D, z, init, yp, fin, ws, ws_bytes, stream);
    });
  PyObject* r = PyTuple_New(3);
  if (r == nullptr) throw python_error();
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(y));
  if (!final_state.defined()) Py_INCREF(Py_None);
  PyTuple_SET_ITEM(r, 1, final_state.defined() ? THPVariable_Wrap(final_state) : Py_None);
  if (!workspace.defined()) Py_INCREF(Py_None);
  PyTuple_SET_ITEM(r, 2, workspace.defined() ? THPVariable_Wrap(workspace) : Py_None);
  return r;
  END_HANDLE_TH_ERRORS
}

// x dt A B C D z state slots y bias softplus limit stream -> y
PyObject* selective_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need_args(n, 14);
  const Tensor& x = device_tensor(a[0], "x", 2);
  const auto dev = x.device();
  const ssd_selective_desc_t d = selective_desc(x, a, a[10], a[11], a[12], 1);
  const int64_t slots = device_tensor(a[7], "state", 3).size(0);
  const float* A = floats(a[2], "A", dev, {d.channels, d.dstate});
  const float* D = floats(a[5], "D", dev, {d.channels});
  float* state = static_cast<float*>(dense(a[7], "state", at::kFloat, dev, {slots, d.channels, d.dstate}));
  const int32_t* map = static_cast<const int32_t*>(dense(a[8], "state_slots", at::kInt, dev, {d.batch}));
  Tensor y = output(a[9], "y", x.scalar_type(), x, x.sizes());
  const void *xp = x.data_ptr(), *dt = data(a[1]), *B = data(a[3]), *C = data(a[4]), *z = data(a[6]);
  void *yp = y.data_ptr(), *stream = handle(a[13]);
  call("ssd_selective_step", [&] { return lib.step(&d, xp, dt, A, B, C, D, z, state, map, slots, yp, stream); });
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

// The descriptor of a convolution of x, and its outputs: one of all channels
// (y or a new one), or, with split = (nheads, headdim, ngroups, dstate), new
// x, B and C.
struct Conv {
  ssd_conv1d_desc_t d;
  const float *w, *bias;
  Tensor out[3];
  int outs;
  void* ptr[3];  // their addresses, null for none
  PyObject* wrap() const {
    if (outs == 1) return THPVariable_Wrap(out[0]);
    PyObject* r = PyTuple_New(3);
    if (r == nullptr) throw python_error();
    for (int i = 0; i < 3; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(out[i]));
    return r;
  }
};
Conv conv_of(const Tensor& x, PyObject* weight, PyObject* bias, PyObject* split, PyObject* silu, PyObject* y,
             int64_t lead) {
  Conv c{};
  const Tensor& w = device_tensor(weight, "weight", 2);
  const IntArrayRef shape = x.sizes();
  const int64_t CH = shape[lead], K = w.size(1);
  c.w = floats(weight, "weight", x.device(), {CH, K});
  c.bias = floats(bias, "bias", x.device(), {CH});
  c.d.batch = shape[0];
  c.d.seqlen = lead == 2 ? shape[1] : 1;
  c.d.channels = CH;
  c.d.conv_width = K < 100 ? (int32_t)K : 100;  // the library refuses what it does not support
  c.d.silu = truth(silu);
  c.d.io_dtype = io_code(x, "x");
  c.d.x_stride = strides(x, "x", lead);
  if (split == Py_None) {
    c.outs = 1;
    c.d.out_channels[0] = CH;
    c.out[0] = output(y, "y", x.scalar_type(), x, shape);
    c.ptr[0] = c.out[0].data_ptr();
    return c;
  }
  int64_t h[4];
  for (int i = 0; i < 4; ++i) {
    h[i] = integer(PyTuple_GET_ITEM(split, i));
    if (h[i] < 1 || h[i] > CH) bad_value("xbc channels must be H*P + 2*G*N");
  }
  if (CH != h[0] * h[1] + 2 * h[2] * h[3]) bad_value("xbc channels must be H*P + 2*G*N");
  c.outs = 3;
  for (int i = 0; i < 3; ++i) {
    Dims s(shape.begin(), shape.begin() + lead);
    s.push_back(h[i == 0 ? 0 : 2]);
    s.push_back(h[i == 0 ? 1 : 3]);
    c.d.out_channels[i] = s[lead] * s[lead + 1];
    c.out[i] = at::empty(s, x.options());
    c.ptr[i] = c.out[i].data_ptr();
  }
  return c;
}

// x weight bias split silu cu_seqlens state_in state_out y stream -> y or (x, B, C)
PyObject* conv_prompts(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need_args(n, 10);
  const Tensor& x = device_tensor(a[0], "x", 3);
  const auto dev = x.device();
  int64_t S;
  const int32_t* cu = offsets(a[5], dev, &S);
  if (S > 0 && x.size(0) != 1) bad_value("packed sequences: x must be [1, T, channels]");
  Conv c = conv_of(x, a[1], a[2], a[3], a[4], a[8], 2);
  const int64_t states[] = {S > 0 ? S : c.d.batch, c.d.channels, (int64_t)THPVariable_Unpack(a[1]).size(1) - 1};
  const float* in = floats(a[6], S > 0 ? "conv_states_in" : "conv_state_in", dev, states);
  float* last = const_cast<float*>(floats(a[7], S > 0 ? "conv_states_out" : "conv_state_out", dev, states));
  const void* xp = x.data_ptr();
  void* stream = handle(a[9]);
  call("ssd_conv1d", [&] {
    return lib.conv(&c.d, cu, S, xp, c.w, c.bias, in, last, c.ptr[0], c.ptr[1], c.ptr[2], stream);
  });
  return c.wrap();
  END_HANDLE_TH_ERRORS
}

// x weight bias split silu state slots y stream -> y or (x, B, C)
PyObject* conv_token(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need_args(n, 9);
  const Tensor& x = device_tensor(a[0], "x", 2);
  const auto dev = x.device();
  const int64_t slots = device_tensor(a[5], "conv_state", 3).size(0);
  Conv c = conv_of(x, a[1], a[2], a[3], a[4], a[7], 1);
  float* state = static_cast<float*>(dense(a[5], "conv_state", at::kFloat, dev,
                                           {slots, c.d.channels, (int64_t)THPVariable_Unpack(a[1]).size(1) - 1}));
  const int32_t* map = static_cast<const int32_t*>(dense(a[6], "state_slots", at::kInt, dev, {c.d.batch}));
  const void* xp = x.data_ptr();
  void* stream = handle(a[8]);
  call("ssd_conv1d_step", [&] {
    return lib.conv_step(&c.d, xp, c.w, c.bias, state, map, slots, c.ptr[0], c.ptr[1], c.ptr[2], stream);
  });
  return c.wrap();
  END_HANDLE_TH_ERRORS
}

// x weight bias z ngroups eps center gate_first silu out stream -> out
PyObject* group_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need_args(n, 11);
  const Tensor* given = tensor(a[0], "x");
  if (given != nullptr && (given->dim() < 1 || given->dim() > 3)) bad_value("x must have 1 to 3 dimensions");
  const Tensor& x = device_tensor(a[0], "x", -1);
  const auto dev = x.device();
  const Tensor* z = tensor(a[3], "z");
  if (z != nullptr) check(*z, "z", x.scalar_type(), dev, x.sizes());
  // as [batch, rows, channels]
  auto in3 = [](const Tensor& t) { return t.dim() == 3 ? t : t.dim() == 2 ? t.unsqueeze(0) : t.unsqueeze(0).unsqueeze(0); };
  const Tensor x3 = in3(x);
  ssd_group_norm_desc_t d{};
  d.batch = x3.size(0);
  d.rows = x3.size(1);
  d.channels = x3.size(2);
  d.ngroups = integer(a[4]);
  d.eps = (float)number(a[5]);
  d.center = truth(a[6]);
  d.gate_first = truth(a[7]);
  d.silu = truth(a[8]);
  d.io_dtype = io_code(x, "x");
  d.x_stride = strides(x3, "x", 2);
  if (z != nullptr) d.z_stride = strides(in3(*z), "z", 2);
  const float* w = floats(a[1], "weight", dev, {d.channels});
  const float* bias = floats(a[2], "bias", dev, {d.channels});
  Tensor out = output(a[9], "out", x.scalar_type(), x, x.sizes());
  const void *xp = x.data_ptr(), *zp = data(a[3]);
  void *op = out.data_ptr(), *stream = handle(a[10]);
  call("ssd_group_norm", [&] { return lib.norm(&d, xp, w, bias, zp, op, stream); });
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// strides(t, lead) -> (token, batch), 0 for dense
PyObject* strides_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need_args(n, 2);
  const Tensor* t = tensor(a[0], "t");
  if (t == nullptr) bad_value("t is required");
  const ssd_stride_t s = strides(*t, "t", integer(a[1]));
  return Py_BuildValue("LL", (long long)s.token, (long long)s.batch);
  END_HANDLE_TH_ERRORS
}

// bind(addresses in the order of Library, error class)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need_args(n, 8);
  int i = 0;
  auto take = [&](auto& f) {
    f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(handle(a[i++]));
    if (f == nullptr) bad_value("bind: a null address");
  };
  take(lib.workspace_bytes);
  take(lib.scan);
  take(lib.scan_varlen);
  take(lib.step);
  take(lib.conv);
  take(lib.conv_step);
  take(lib.norm);
  Py_INCREF(a[i]);
  Py_XDECREF(lib.error);
  lib.error = a[i];
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define FAST(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST("bind", bind),
                         FAST("strides", strides_py),
                         FAST("selective_prompts", selective_prompts),
                         FAST("selective_step", selective_step),
                         FAST("conv_prompts", conv_prompts),
                         FAST("conv_token", conv_token),
                         FAST("group_norm", group_norm),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
