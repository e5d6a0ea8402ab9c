// _pycall: the tensor calls of rotary.py and clip.py.
//
// A Python module that checks the tensors of a call, makes its outputs and
// workspace, and calls tp_rope.h / tp_grad.h.  It computes nothing.  These
// operators take a few microseconds on the GPU for a few tokens, and the same
// steps in Python and ctypes took 21 us around a library call of 4.1 us (32
// tokens of 16 + 16 heads, Grace host): here they take 1.6.
//
// The library's functions come by address from the ctypes binding (bind), so
// that whichever build of libtpmlp the binding loaded is the one called.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <string>
#include <vector>

#include "tp_grad.h"
#include "tp_rope.h"

namespace {

struct Library {
  decltype(&tp_rope_apply) rope_apply = nullptr;
  decltype(&tp_qk_norm_forward) norm_forward = nullptr;
  decltype(&tp_qk_norm_workspace_bytes) norm_workspace_bytes = nullptr;
  decltype(&tp_qk_norm_backward) norm_backward = nullptr;
  decltype(&tp_grad_workspace_bytes) grad_workspace_bytes = nullptr;
  decltype(&tp_grad_norm) grad_norm = nullptr;
  decltype(&tp_grad_clip) grad_clip = nullptr;
  PyObject* check = nullptr;   // binding._check(status, what)
} lib;

struct Refused {   // a ValueError
  std::string msg;
};
struct Raised {};  // a Python error is set

std::string shown(const at::Tensor& t) {
  std::ostringstream s;
  s << t.sizes() << " " << t.dtype().name() << " on " << t.device();
  return s.str();
}

const at::Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o))
    throw Refused{std::string(name) + " must be a torch tensor"};
  return THPVariable_Unpack(o);
}

// A tensor argument that may be None.
const at::Tensor* maybe(const char* name, PyObject* o) {
  return o == Py_None ? nullptr : &tensor(name, o);
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

int dtype_code(const char* name, const at::Tensor& t) {
  if (t.is_cuda()) {
    if (t.scalar_type() == at::kBFloat16) return TPMLP_BF16;
    if (t.scalar_type() == at::kFloat) return TPMLP_FP32;
  }
  throw Refused{std::string(name) + " must be a bf16 or fp32 CUDA tensor, got " +
                shown(t)};
}

// The device of a call's tensors made current, and its stream (a
// torch.cuda.Stream, a raw handle, or None for the device's current one) the
// one that new tensors belong to.
struct Place {
  c10::cuda::OptionalCUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard guard;
  void* stream;

  Place(const at::Device& d, PyObject* s) {
    if (d.index() != c10::cuda::current_device()) device.set_device(d);
    if (s == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(d.index()).stream();
      return;
    }
    long long raw = 0;
    if (PyLong_Check(s)) {
      raw = integer(s);
    } else {
      PyObject* i = PyObject_GetAttrString(s, "device_index");
      if (i == nullptr) throw Raised{};
      const long long index = PyLong_AsLongLong(i);
      Py_DECREF(i);
      if (index == -1 && PyErr_Occurred()) throw Raised{};
      if (index != d.index())
        throw Refused{"the stream belongs to another device than the tensors"};
      PyObject* h = PyObject_GetAttrString(s, "cuda_stream");
      if (h == nullptr) throw Raised{};
      raw = PyLong_AsLongLong(h);
      Py_DECREF(h);
      if (raw == -1 && PyErr_Occurred()) throw Raised{};
    }
    const auto handle = reinterpret_cast<cudaStream_t>(raw);
    guard.reset_stream(handle == nullptr
                           ? c10::cuda::getDefaultCUDAStream(d.index())
                           : c10::cuda::getStreamFromExternal(handle, d.index()));
    stream = handle;
  }
};

template <class F>
int without_gil(F&& f) {
  PyThreadState* s = PyEval_SaveThread();
  const int rc = f();
  PyEval_RestoreThread(s);
  return rc;
}

void check(int status, const char* what) {
  if (status == TPMLP_OK) return;
  PyObject* r = PyObject_CallFunction(lib.check, "is", status, what);
  Py_XDECREF(r);
  if (r != nullptr) PyErr_SetString(PyExc_RuntimeError, what);
  throw Raised{};
}

// A new contiguous tensor on the current device and stream (at::empty without
// its dispatch).
at::Tensor make(at::IntArrayRef size, at::ScalarType type, const at::Device& d) {
  return at::Tensor(at::detail::empty_cuda(size, type, d, std::nullopt));
}

// Row i of a new contiguous [n, d] tensor, as a tensor of its own.
at::Tensor row_of(const at::Tensor& all, int64_t i) {
  auto t = c10::make_intrusive<c10::TensorImpl>(c10::Storage(all.storage()),
                                                all.key_set(), all.dtype());
  const int64_t d = all.size(1);
  t->set_storage_offset(i * d);
  t->set_sizes_contiguous(d);
  return at::Tensor(std::move(t));
}

// ---------------------------------------------------------------- heads --

tp_heads heads_of(const char* name, const at::Tensor& x, long long d,
                  const at::Tensor* like = nullptr) {
  if (like != nullptr &&
      (x.sizes() != like->sizes() || x.scalar_type() != like->scalar_type() ||
       x.device() != like->device()))
    throw Refused{std::string(name) + ": expected " + shown(*like) + ", got " +
                  shown(x)};
  const auto size = x.sizes();
  const auto stride = x.strides();
  const auto n = size.size();
  if ((n != 3 && n != 4) || size[n - 1] != d || (stride[n - 1] != 1 && d != 1))
    throw Refused{std::string(name) + ": expected [T, heads, " +
                  std::to_string(d) + "] or [T, shards, heads, " +
                  std::to_string(d) + "] with consecutive head elements, got " +
                  shown(x)};
  const long long heads = n == 3 ? size[1] : size[1] * size[2];
  if (heads < 1 || heads > 65535 || size[0] > (1 << 28))
    throw Refused{std::string(name) + ": expected 1 to 65535 heads and at most "
                  "2^28 tokens, got " + shown(x)};
  tp_heads v;
  v.data = x.numel() == 0 ? nullptr : const_cast<void*>(x.const_data_ptr());
  v.token_stride = stride[0];
  v.group_stride = n == 3 ? 0 : stride[1];
  v.head_stride = stride[n - 2];
  v.heads = static_cast<int>(heads);
  v.group = static_cast<int>(size[n - 2]);
  return v;
}

// q and k of a call (k may be absent), as inputs and outputs.
struct Heads {
  const at::Tensor* in[2];
  at::Tensor out[2];
  tp_heads vin[2], vout[2];
  int dtype;

  const tp_heads* i(int s) const { return in[s] ? &vin[s] : nullptr; }
  const tp_heads* o(int s) const { return in[s] ? &vout[s] : nullptr; }

  Heads(const char* nq, const char* nk, PyObject* q, PyObject* k, long long d) {
    in[0] = &tensor(nq, q);
    in[1] = maybe(nk, k);
    dtype = dtype_code(nq, *in[0]);
    vin[0] = heads_of(nq, *in[0], d);
    if (in[1] == nullptr) return;
    vin[1] = heads_of(nk, *in[1], d);
    if (in[1]->size(0) != in[0]->size(0) ||
        in[1]->scalar_type() != in[0]->scalar_type() ||
        in[1]->device() != in[0]->device())
      throw Refused{std::string(nq) + " and " + nk +
                    " differ in tokens, type or device"};
  }
  // The outputs: as given, or new.  (The device and stream are current.)
  void outputs(PyObject* q_out, PyObject* k_out, long long d) {
    PyObject* given[2] = {q_out, k_out};
    const char* names[2] = {"q_out", "k_out"};
    for (int s = 0; s < 2; ++s) {
      if (in[s] == nullptr) {
        if (given[s] != Py_None) throw Refused{"k_out without k"};
        continue;
      }
      if (given[s] != Py_None) {
        out[s] = tensor(names[s], given[s]);
        heads_of(names[s], out[s], d, in[s]);
        // a lazy copy has memory of its own from here on; then its address
        out[s].data_ptr();
        vout[s] = heads_of(names[s], out[s], d, in[s]);
        continue;
      }
      out[s] = make(in[s]->sizes(), in[s]->scalar_type(), in[s]->device());
      vout[s] = heads_of(names[s], out[s], d);
    }
  }
  int tokens() const { return static_cast<int>(in[0]->size(0)); }
};

tp_positions positions_of(PyObject* o, PyObject* offset, PyObject* seq_len,
                          const at::Tensor& q) {
  tp_positions p;
  p.data = nullptr;
  p.is_int64 = 0;
  p.offset = integer(offset);
  p.seq_len = integer(seq_len);
  const at::Tensor* t = maybe("positions", o);
  if (t == nullptr) return p;
  const auto type = t->scalar_type();
  if (t->dim() != 1 || t->size(0) != q.size(0) || t->device() != q.device() ||
      (type != at::kInt && type != at::kLong) || !t->is_contiguous())
    throw Refused{"positions: expected a contiguous int32 or int64 tensor [" +
                  std::to_string(q.size(0)) + "] on the device of q, got " +
                  shown(*t)};
  p.data = t->const_data_ptr();
  p.is_int64 = type == at::kLong;
  return p;
}

float* param_of(const char* name, PyObject* o, long long d,
                const at::Tensor& q) {
  const at::Tensor* t = maybe(name, o);
  if (t == nullptr) return nullptr;
  if (t->scalar_type() != at::kFloat || t->dim() != 1 || t->size(0) != d ||
      t->device() != q.device() || !t->is_contiguous())
    throw Refused{std::string(name) + ": expected a contiguous fp32 tensor [" +
                  std::to_string(d) + "] on the device of q, got " + shown(*t)};
  return static_cast<float*>(const_cast<void*>(t->const_data_ptr()));
}

PyObject* wrapped(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  PyObject* o = THPVariable_Wrap(t);
  if (o == nullptr) throw Raised{};
  return o;
}

// New references into a tuple; null entries are None.
PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
  PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (t == nullptr) throw Raised{};
  Py_ssize_t i = 0;
  try {
    for (const at::Tensor& x : ts) PyTuple_SET_ITEM(t, i++, wrapped(x));
  } catch (...) {
    Py_DECREF(t);
    throw;
  }
  return t;
}

tp_rope_handle* rope_handle(PyObject* o) {
  return o == Py_None ? nullptr
                      : reinterpret_cast<tp_rope_handle*>(integer(o));
}

// rope(handle, d, inverse, q, k, positions, offset, seq_len, q_out, k_out,
//      stream) -> (q, k)
PyObject* rope(PyObject* const* a) {
  const long long d = integer(a[1]);
  Heads h("q", "k", a[3], a[4], d);
  const tp_positions pos = positions_of(a[5], a[6], a[7], *h.in[0]);
  Place place(h.in[0]->device(), a[10]);
  h.outputs(a[8], a[9], d);
  tp_rope_handle* handle = rope_handle(a[0]);
  const int inverse = static_cast<int>(integer(a[2]));
  check(without_gil([&] {
          return lib.rope_apply(handle, h.tokens(), h.dtype, inverse, h.i(0),
                                h.o(0), h.i(1), h.o(1), &pos, place.stream);
        }),
        "tp_rope_apply");
  return tuple_of({h.out[0], h.out[1]});
}

// norm_forward(handle, d, norm, eps, q, k, q_gamma, q_beta, k_gamma, k_beta,
//              positions, offset, seq_len, q_out, k_out, stream) -> (q, k)
PyObject* norm_forward(PyObject* const* a) {
  const long long d = integer(a[1]);
  Heads h("q", "k", a[4], a[5], d);
  const at::Tensor& q = *h.in[0];
  const tp_qk_norm n = {static_cast<int>(integer(a[2])),
                        static_cast<float>(real(a[3])),
                        param_of("q_gamma", a[6], d, q),
                        param_of("q_beta", a[7], d, q),
                        param_of("k_gamma", a[8], d, q),
                        param_of("k_beta", a[9], d, q)};
  const tp_positions pos = positions_of(a[10], a[11], a[12], q);
  Place place(q.device(), a[15]);
  h.outputs(a[13], a[14], d);
  tp_rope_handle* handle = rope_handle(a[0]);
  check(without_gil([&] {
          return lib.norm_forward(handle, h.tokens(), h.dtype, &n, h.i(0),
                                  h.o(0), h.i(1), h.o(1), &pos, place.stream);
        }),
        "tp_qk_norm_forward");
  return tuple_of({h.out[0], h.out[1]});
}

// norm_backward(handle, d, norm, eps, dq, dk, q, k, q_gamma, k_gamma,
//               positions, offset, seq_len, dq_out, dk_out, param_grads,
//               q_gamma_out, q_beta_out, k_gamma_out, k_beta_out, stream)
//   -> (dq, dk, dq_gamma, dq_beta, dk_gamma, dk_beta)
PyObject* norm_backward(PyObject* const* a) {
  const long long d = integer(a[1]);
  Heads h("dq", "dk", a[4], a[5], d);
  const at::Tensor& dq = *h.in[0];
  if ((a[5] == Py_None) != (a[7] == Py_None))
    throw Refused{"dk and k must be given together"};
  const tp_heads xq = heads_of("q", tensor("q", a[6]), d, h.in[0]);
  tp_heads xk;
  if (h.in[1] != nullptr) xk = heads_of("k", tensor("k", a[7]), d, h.in[1]);
  const tp_qk_norm n = {static_cast<int>(integer(a[2])),
                        static_cast<float>(real(a[3])),
                        param_of("q_gamma", a[8], d, dq), nullptr,
                        param_of("k_gamma", a[9], d, dq), nullptr};
  const tp_positions pos = positions_of(a[10], a[11], a[12], dq);
  Place place(dq.device(), a[20]);
  h.outputs(a[13], a[14], d);
  tp_rope_handle* handle = rope_handle(a[0]);
  at::Tensor grad[4], ws;
  float* gp[4] = {nullptr, nullptr, nullptr, nullptr};
  size_t bytes = 0;
  const int params = PyObject_IsTrue(a[15]);
  if (params < 0) throw Raised{};
  at::Tensor all;   // parameter gradients that are made new: one allocation
  const char* names[4] = {"dq_gamma", "dq_beta", "dk_gamma", "dk_beta"};
  for (int i = 0; i < 4; ++i) {
    PyObject* given = a[16 + i];
    if (!params || (i % 2 == 1 && n.norm != TPQK_LAYERNORM) ||
        (i >= 2 && h.in[1] == nullptr)) {
      if (given != Py_None)
        throw Refused{std::string("out: this call has no ") + names[i]};
      continue;
    }
    if (given == Py_None) {
      if (!all.defined()) all = make({4, d}, at::kFloat, dq.device());
      grad[i] = row_of(all, i);
      gp[i] = grad[i].data_ptr<float>();
    } else {
      param_of(names[i], given, d, dq);
      grad[i] = tensor(names[i], given);
      gp[i] = grad[i].data_ptr<float>();   // (as the heads' outputs)
    }
  }
  if (params) {
    // a workspace of this call alone: calls on several streams, and captured
    // graphs, share no partial sums
    bytes = lib.norm_workspace_bytes(handle);
    ws = make({static_cast<int64_t>(bytes)}, at::kByte, dq.device());
  }
  const tp_qk_norm_grads g = {gp[0], gp[1], gp[2], gp[3]};
  void* wp = ws.defined() ? ws.data_ptr() : nullptr;
  check(without_gil([&] {
          return lib.norm_backward(
              handle, h.tokens(), h.dtype, &n, h.i(0), &xq, h.o(0), h.i(1),
              h.in[1] != nullptr ? &xk : nullptr, h.o(1), &pos, &g, wp, bytes,
              place.stream);
        }),
        "tp_qk_norm_backward");
  return tuple_of({h.out[0], h.out[1], grad[0], grad[1], grad[2], grad[3]});
}

// ------------------------------------------------------------ gradients --

// grads(tensors, outs or None, clip, max_norm, eps, stream) -> norm
PyObject* grads(PyObject* const* a) {
  struct List {
    PyObject* seq;
    explicit List(PyObject* o)
        : seq(o == Py_None ? nullptr : PySequence_Fast(o, "expected a list")) {
      if (o != Py_None && seq == nullptr) throw Raised{};
    }
    ~List() { Py_XDECREF(seq); }
    Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(seq); }
    PyObject* at(Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq, i); }
  };
  const List in(a[0]), out(a[1]);
  const Py_ssize_t n = in.size();
  if (n == 0 || n > (1 << 24)) throw Refused{"expected 1 to 2^24 gradients"};
  if (out.seq != nullptr && out.size() != n)
    throw Refused{"out: expected " + std::to_string(n) + " tensors, got " +
                  std::to_string(out.size())};
  const bool clip = integer(a[2]) != 0;
  const double max_norm = real(a[3]), eps = real(a[4]);
  std::vector<tp_grad_tensor> table(static_cast<size_t>(n));
  const at::Device dev = tensor("gradient", in.at(0)).device();
  dtype_code("a gradient", tensor("gradient", in.at(0)));
  // (an output that is a lazy copy is copied below, on the call's stream)
  const Place place(dev, a[5]);
  for (Py_ssize_t i = 0; i < n; ++i) {
    const at::Tensor& g = tensor("gradient", in.at(i));
    tp_grad_tensor& t = table[static_cast<size_t>(i)];
    t.dtype = dtype_code("a gradient", g);
    if (g.device() != dev || !g.is_contiguous())
      throw Refused{"gradient " + std::to_string(i) + ": expected a contiguous "
                    "tensor on the device of the first, got " + shown(g)};
    t.numel = g.numel();
    if (out.seq == nullptr) {
      t.grad = clip ? g.data_ptr() : const_cast<void*>(g.const_data_ptr());
      t.out = const_cast<void*>(t.grad);
      continue;
    }
    const at::Tensor& o = tensor("out", out.at(i));
    if (o.sizes() != g.sizes() || o.scalar_type() != g.scalar_type() ||
        o.device() != dev || !o.is_contiguous())
      throw Refused{"out " + std::to_string(i) + ": expected a contiguous " +
                    shown(g) + " tensor, got " + shown(o)};
    t.grad = g.const_data_ptr();
    t.out = o.data_ptr();
  }
  const at::Tensor norm = make({}, at::kFloat, dev);
  const int count = static_cast<int>(n);
  const size_t bytes = lib.grad_workspace_bytes(count);
  // of this call alone, as above
  const at::Tensor ws = make({static_cast<int64_t>(bytes)}, at::kByte, dev);
  float* np = norm.data_ptr<float>();
  void* wp = ws.data_ptr();
  check(without_gil([&] {
          return clip ? lib.grad_clip(count, table.data(), max_norm, eps, np, wp,
                                      bytes, place.stream)
                      : lib.grad_norm(count, table.data(), np, wp, bytes,
                                      place.stream);
        }),
        clip ? "tp_grad_clip" : "tp_grad_norm");
  return wrapped(norm);
}

// --------------------------------------------------------------- module --

// bind(check, addresses of Library's functions in its order)
PyObject* bind(PyObject* const* a) {
  auto at = [&](int i) { return reinterpret_cast<void*>(integer(a[i])); };
  Library l;
  l.rope_apply = reinterpret_cast<decltype(l.rope_apply)>(at(1));
  l.norm_forward = reinterpret_cast<decltype(l.norm_forward)>(at(2));
  l.norm_workspace_bytes =
      reinterpret_cast<decltype(l.norm_workspace_bytes)>(at(3));
  l.norm_backward = reinterpret_cast<decltype(l.norm_backward)>(at(4));
  l.grad_workspace_bytes =
      reinterpret_cast<decltype(l.grad_workspace_bytes)>(at(5));
  l.grad_norm = reinterpret_cast<decltype(l.grad_norm)>(at(6));
  l.grad_clip = reinterpret_cast<decltype(l.grad_clip)>(at(7));
  Py_INCREF(a[0]);
  l.check = a[0];
  Py_XDECREF(lib.check);
  lib = l;
  Py_RETURN_NONE;
}

// A function of N positional arguments; no C++ exception leaves it.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  if (lib.check == nullptr && F != bind) {
    PyErr_SetString(PyExc_RuntimeError, "_pycall is not bound to the library");
    return nullptr;
  }
  HANDLE_TH_ERRORS   // torch's own exceptions, as torch raises them
  try {
    return F(a);
  } catch (const Raised&) {
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.msg.c_str());
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"bind", nullptr, 0, nullptr},
    {"rope", nullptr, 0, nullptr},
    {"norm_forward", nullptr, 0, nullptr},
    {"norm_backward", nullptr, 0, nullptr},
    {"grads", nullptr, 0, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycall",
                      "Tensor calls of libtpmlp's query/key and gradient "
                      "operators.",
                      -1, methods, nullptr, nullptr, nullptr, nullptr};

template <PyObject* (*F)(PyObject* const*), int N>
void set(int i) {
  methods[i].ml_meth = reinterpret_cast<PyCFunction>(
      reinterpret_cast<void (*)()>(entry<F, N>));
  methods[i].ml_flags = METH_FASTCALL;
}

}  // namespace

PyMODINIT_FUNC PyInit__pycall() {
  set<bind, 8>(0);
  set<rope, 11>(1);
  set<norm_forward, 16>(2);
  set<norm_backward, 21>(3);
  set<grads, 6>(4);
  return PyModule_Create(&module);
}
