// The block operators' Python binding (module _blocks): argument checks, new result tensors and
// the C call, in one native call each.  A small call's time is its host time; through ctypes,
// with torch.empty for the results, a layer norm of 64 x 768 took 21 us of it.
//
// Functions take every argument by position (blocks.py gives them names, defaults and their
// documentation); None stands for an absent tensor.  A refused argument raises ValueError, a
// status from the library MuonBankError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <optional>
#include <string>
#include <utility>
#include <vector>

#include "muonbank.h"

namespace {

using at::Tensor;
using c10::ScalarType;

PyObject* g_check;           // _binding.check(name, status): raises MuonBankError
PyObject* g_out_of_memory;   // torch.OutOfMemoryError

struct Refused {
  std::string text;
};
struct Raised {};     // a Python exception is set

std::string str(c10::IntArrayRef v) {
  std::string s = "(";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + ")";
}
std::string str(const Tensor& t) {
  return str(t.sizes()) + " " + c10::toString(t.scalar_type()) + " on " + t.device().str();
}

// ---------------------------------------------------------------- arguments

// A tensor argument, or null for None.
const Tensor* tensor_or_none(PyObject* o, const char* what) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw Refused{std::string(what) + " must be a tensor"};
  const Tensor& t = THPVariable_Unpack(o);
  // such a view's memory holds other values than the tensor
  if (t.is_neg()) throw Refused{std::string(what) + " is a negated view: call resolve_neg() first"};
  return &t;
}
const Tensor& tensor(PyObject* o, const char* what) {
  const Tensor* t = tensor_or_none(o, what);
  if (!t) throw Refused{std::string(what) + " must be a tensor"};
  return *t;
}
// The tensor that a call's device comes from.
const Tensor& cuda_tensor(PyObject* o, const char* what) {
  const Tensor& t = tensor(o, what);
  if (!t.is_cuda()) throw Refused{std::string(what) + " must be a CUDA tensor"};
  return t;
}

long long integer(PyObject* o, const char* what) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    if (PyErr_ExceptionMatches(PyExc_OverflowError)) {
      PyErr_Clear();
      throw Refused{std::string(what) + " is out of range"};
    }
    throw Raised{};
  }
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}
float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return static_cast<float>(v);
}

int type_of(const Tensor& t, const char* what) {
  switch (t.scalar_type()) {
    case ScalarType::Float: return MB_F32;
    case ScalarType::BFloat16: return MB_BF16;
    case ScalarType::Half: return MB_F16;
    default:
      throw Refused{std::string(what) + " has dtype " + c10::toString(t.scalar_type()) +
                    ", expected float32, bfloat16 or float16"};
  }
}

void like(const Tensor& t, const char* what, c10::IntArrayRef shape, ScalarType dtype, c10::Device device) {
  if (t.sizes() != shape || t.scalar_type() != dtype || t.device() != device)
    throw Refused{std::string(what) + " is " + str(t) + ", expected " + str(shape) + " " + c10::toString(dtype) +
                  " on " + device.str()};
}

// Address of a contiguous tensor of this shape and type (null: no tensor).
void* dense(const Tensor* t, const char* what, c10::IntArrayRef shape, ScalarType dtype, c10::Device device) {
  if (!t) return nullptr;
  like(*t, what, shape, dtype, device);
  if (!t->is_contiguous()) throw Refused{std::string(what) + " must be contiguous"};
  return t->data_ptr();
}

// Elements from row to row of t taken as [rows, its last dimension].
int64_t row_stride(const Tensor& t, const char* what) {
  const auto n = t.sizes(), s = t.strides();
  const size_t d = n.size();
  if (t.is_contiguous()) return n[d - 1];
  if (n[d - 1] > 1 && s[d - 1] != 1) throw Refused{std::string(what) + " must be contiguous in its last dimension"};
  int64_t stride = -1, rows = 1;   // dimensions of one element do not matter; the others must fold into one
  for (size_t i = d - 1; i-- > 0;) {
    if (n[i] == 1) continue;
    if (stride < 0) stride = s[i];
    else if (s[i] != stride * rows) throw Refused{"the rows of " + std::string(what) + " must be evenly spaced"};
    rows *= n[i];
  }
  return stride < 0 ? n[d - 1] : stride;
}

Tensor make(c10::IntArrayRef shape, ScalarType dtype, c10::Device device) {
  return at::detail::empty_cuda(shape, dtype, device, std::nullopt);
}

// The given result tensor, or a new one.
Tensor result(PyObject* o, const char* what, c10::IntArrayRef shape, ScalarType dtype, c10::Device device) {
  const Tensor* t = tensor_or_none(o, what);
  if (!t) return make(shape, dtype, device);
  like(*t, what, shape, dtype, device);
  return *t;
}

// New results of one call that live equally long in one allocation, 256 bytes apart: an allocation costs 0.7 us of a
// call, a tensor on a ready one 0.2.
struct Together {
  c10::Device device;
  size_t bytes = 0;
  c10::Storage storage;
  explicit Together(c10::Device d) : device(d) {}
  // reserves room for a result that the caller did not pass; its place
  size_t room(PyObject* given, int64_t elements) {
    const size_t at = bytes;
    if (given == Py_None) bytes += (static_cast<size_t>(elements) * 4 + 255) / 256 * 256;
    return at;
  }
  void allocate() {
    if (bytes > 0) storage = make({static_cast<int64_t>(bytes)}, ScalarType::Byte, device).storage();
  }
  // the given tensor, or the one at `at` (of a 4-byte type)
  Tensor take(PyObject* given, const char* what, c10::IntArrayRef shape, ScalarType dtype, size_t at) {
    if (given != Py_None || bytes == 0) return result(given, what, shape, dtype, device);
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(storage), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                        c10::scalarTypeToTypeMeta(dtype));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    t.unsafeGetTensorImpl()->set_storage_offset(static_cast<int64_t>(at / 4));
    return t;
  }
};

struct Workspace {
  Tensor own;
  void* ptr = nullptr;
  size_t bytes = 0;
  Workspace(PyObject* given, size_t need, c10::Device device) {
    const Tensor* t = tensor_or_none(given, "workspace");
    if (!t) {
      if (need == 0) return;
      own = make({static_cast<int64_t>(need)}, ScalarType::Byte, device);
      t = &own;
    } else if (t->device() != device || !t->is_contiguous()) {
      throw Refused{"workspace must be a contiguous tensor on " + device.str()};
    } else if (t->nbytes() < need) {
      throw Refused{"workspace holds " + std::to_string(t->nbytes()) + " bytes, needs " + std::to_string(need)};
    }
    ptr = t->data_ptr();
    bytes = t->nbytes();
  }
};

// The call's device and stream made current.  With a stream given, the call's tensors are
// marked as used on it and new ones belong to it; the caller orders the streams.
struct Where {
  c10::cuda::CUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard on;
  cudaStream_t stream;
  Where(const Tensor& t, PyObject* given, PyObject* const* args, Py_ssize_t nargs) : device(t.device()) {
    if (given == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
      return;
    }
    PyObject* handle = PyObject_HasAttrString(given, "cuda_stream") ? PyObject_GetAttrString(given, "cuda_stream")
                                                                    : Py_NewRef(given);
    if (!handle) throw Raised{};
    void* raw = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (PyErr_Occurred()) throw Raised{};
    stream = static_cast<cudaStream_t>(raw);
    const auto s = c10::cuda::getStreamFromExternal(stream, t.device().index());
    on.reset_stream(s);
    for (Py_ssize_t i = 0; i < nargs; ++i)
      if (THPVariable_Check(args[i]) && THPVariable_Unpack(args[i]).is_cuda())
        THPVariable_Unpack(args[i]).record_stream(s.unwrap());
  }
};

void checked(const char* name, int status) {
  if (status == MB_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "si", name, status);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s: status %d", name, status);
  throw Raised{};
}

// A call of the library, its arguments ready, while other threads may run: a launch waits where the stream's
// queue is full.
template <typename CALL>
int unlocked(CALL&& call) {
  PyThreadState* state = PyEval_SaveThread();
  const int status = call();
  PyEval_RestoreThread(state);
  return status;
}

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
// The given tensor's own object, or a new one; called once the kernels are launched.  A given tensor counts as
// modified in place, so that a backward pass that has saved it notices (one of inference mode has no version).
PyObject* give(PyObject* given, const Tensor& t) {
  if (given == Py_None) return wrap(t);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  return Py_NewRef(given);
}

template <typename... O>
PyObject* tuple(O... o) {
  PyObject* const items[] = {o...};
  constexpr Py_ssize_t n = sizeof...(o);
  PyObject* t = PyTuple_New(n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (t && items[i]) PyTuple_SET_ITEM(t, i, items[i]);
    else Py_XDECREF(items[i]);
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (!items[i]) {
      Py_XDECREF(t);
      return nullptr;
    }
  }
  return t;
}

// ---------------------------------------------------------------- layer norm

struct NormShape {
  int64_t rows, cols;
  int type, w_type;
};

// w: a weight, bias or gradient of one, whose type the others share.
NormShape norm_shape(const Tensor& x, const Tensor* w, const char* what) {
  if (x.dim() < 1) throw Refused{"x must have at least one dimension"};
  NormShape s{};
  s.cols = x.sizes().back();
  if (s.cols == 0) throw Refused{"x has rows of no elements"};
  s.rows = x.numel() / s.cols;
  s.type = type_of(x, "x");
  s.w_type = MB_F32;
  if (w) {
    if (w->scalar_type() != x.scalar_type() && w->scalar_type() != ScalarType::Float)
      throw Refused{std::string(what) + " has dtype " + c10::toString(w->scalar_type()) + ", expected x's or float32"};
    s.w_type = type_of(*w, what);
  }
  return s;
}

// x, weight, bias, eps, y, mean, rstd, stream
PyObject* layer_norm(PyObject* const* a, Py_ssize_t n) {
  const Tensor& x = cuda_tensor(a[0], "x");
  const auto device = x.device();
  Where where(x, a[7], a, n);
  const Tensor *w = tensor_or_none(a[1], "weight"), *b = tensor_or_none(a[2], "bias");
  const Tensor* param = w ? w : b;
  const NormShape s = norm_shape(x, param, w ? "weight" : "bias");
  const auto wt = param ? param->scalar_type() : ScalarType::Float;
  const void *wp = dense(w, "weight", {s.cols}, wt, device), *bp = dense(b, "bias", {s.cols}, wt, device);
  const auto lead = x.sizes().slice(0, x.dim() - 1);
  const float eps = number(a[3]);
  const Tensor y = result(a[4], "y", x.sizes(), x.scalar_type(), device);
  Together stats(device);
  const size_t mean_at = stats.room(a[5], s.rows), rstd_at = stats.room(a[6], s.rows);
  stats.allocate();
  const Tensor mean = stats.take(a[5], "mean", lead, ScalarType::Float, mean_at);
  const Tensor rstd = stats.take(a[6], "rstd", lead, ScalarType::Float, rstd_at);
  const void* xp = x.data_ptr();
  void* yp = y.data_ptr();
  auto* mp = static_cast<float*>(dense(&mean, "mean", lead, ScalarType::Float, device));
  auto* rp = static_cast<float*>(dense(&rstd, "rstd", lead, ScalarType::Float, device));
  const int64_t x_stride = row_stride(x, "x"), y_stride = row_stride(y, "y");
  checked("mb_layer_norm", unlocked([&] {
            return mb_layer_norm(xp, x_stride, s.type, wp, bp, s.w_type, yp, y_stride, mp, rp, s.rows, s.cols, eps,
                                 where.stream);
          }));
  return tuple(give(a[4], y), give(a[5], mean), give(a[6], rstd));
}

// dy, x, mean, rstd, weight, bias (whether its gradient is wanted), dx, dweight, dbias, workspace, stream, weight_grad
// (whether the weight's is)
PyObject* layer_norm_backward(PyObject* const* a, Py_ssize_t n) {
  const Tensor &x = cuda_tensor(a[1], "x"), &dy = tensor(a[0], "dy");
  const auto device = x.device();
  Where where(x, a[10], a, n);
  const Tensor *w = tensor_or_none(a[4], "weight"), *given_db = tensor_or_none(a[8], "dbias");
  if (!w && a[7] != Py_None) throw Refused{"dweight needs a weight"};
  const Tensor* param = w ? w : given_db;
  const NormShape s = norm_shape(x, param, w ? "weight" : "dbias");
  like(dy, "dy", x.sizes(), x.scalar_type(), device);
  const auto lead = x.sizes().slice(0, x.dim() - 1);
  const auto* mean = static_cast<float*>(dense(&tensor(a[2], "mean"), "mean", lead, ScalarType::Float, device));
  const auto* rstd = static_cast<float*>(dense(&tensor(a[3], "rstd"), "rstd", lead, ScalarType::Float, device));
  const Tensor dx = result(a[6], "dx", x.sizes(), x.scalar_type(), device);
  const auto wt = param ? param->scalar_type() : ScalarType::Float;
  const void* wp = dense(w, "weight", {s.cols}, wt, device);
  Tensor dw, db;
  void *dwp = nullptr, *dbp = nullptr;
  if (a[7] != Py_None || (w && truth(a[11]))) {
    dw = result(a[7], "dweight", {s.cols}, wt, device);
    dwp = dense(&dw, "dweight", {s.cols}, wt, device);
  }
  if (given_db || (w && truth(a[5]))) {
    db = result(a[8], "dbias", {s.cols}, wt, device);
    dbp = dense(&db, "dbias", {s.cols}, wt, device);
  }
  std::optional<Workspace> ws;
  if (dwp || dbp) {
    size_t need = 0;
    checked("mb_layer_norm_workspace_bytes", mb_layer_norm_workspace_bytes(s.rows, s.cols, &need));
    ws.emplace(a[9], need, device);
  }
  const void *dyp = dy.data_ptr(), *xp = x.data_ptr();
  void* dxp = dx.data_ptr();
  const int64_t dy_stride = row_stride(dy, "dy"), x_stride = row_stride(x, "x"), dx_stride = row_stride(dx, "dx");
  checked("mb_layer_norm_backward", unlocked([&] {
            return mb_layer_norm_backward(dyp, dy_stride, xp, x_stride, s.type, wp, s.w_type, mean, rstd, dxp, dx_stride,
                                          dwp, dbp, s.rows, s.cols, ws ? ws->ptr : nullptr, ws ? ws->bytes : 0,
                                          where.stream);
          }));
  return tuple(give(a[6], dx), give(a[7], dw), give(a[8], db));
}

// ---------------------------------------------------------------- rotary

void head_tensor(const Tensor& src, const Tensor& dst, const char* what, mb_head_tensor* h) {
  const int64_t d = src.dim();
  h->src = src.data_ptr();
  h->dst = dst.data_ptr();
  h->heads = src.size(d - 2);
  for (const Tensor* t : {&src, &dst})
    if (t->size(d - 1) > 1 && t->stride(d - 1) != 1)
      throw Refused{std::string(what) + " must be contiguous in its last dimension"};
  h->src_batch = d == 4 ? src.stride(0) : 0;
  h->src_token = src.stride(d - 3);
  h->src_head = src.stride(d - 2);
  h->dst_batch = d == 4 ? dst.stride(0) : 0;
  h->dst_token = dst.stride(d - 3);
  h->dst_head = dst.stride(d - 2);
}

// q, k, positions, inv_freq, sections, interleaved, q_out, k_out, stream
template <int (*CALL)(const mb_rotary_desc*, void*)>
PyObject* rotary(PyObject* const* a, Py_ssize_t n, const char* name) {
  const Tensor& q = cuda_tensor(a[0], "q");
  const auto device = q.device();
  Where where(q, a[8], a, n);
  if (q.dim() != 3 && q.dim() != 4)
    throw Refused{"q must be [batch, tokens, heads, dim] or [tokens, heads, dim]"};
  const int64_t d = q.dim();
  mb_rotary_desc r{};
  r.type = type_of(q, "q");
  r.batch = d == 4 ? q.size(0) : 1;
  r.tokens = q.size(d - 3);
  const int64_t dim = q.size(d - 1);
  if (dim > (1 << 30)) throw Refused{"a head of q has too many elements"};
  r.dim = static_cast<int32_t>(dim);
  r.interleaved = truth(a[5]);
  const Tensor qo = result(a[6], "q_out", q.sizes(), q.scalar_type(), device);
  head_tensor(q, qo, "q", &r.q);
  Tensor ko;
  if (const Tensor* k = tensor_or_none(a[1], "k")) {
    c10::DimVector shape(q.sizes().begin(), q.sizes().end());
    shape[d - 2] = k->dim() == d ? k->size(d - 2) : 0;
    like(*k, "k", shape, q.scalar_type(), device);
    ko = result(a[7], "k_out", shape, q.scalar_type(), device);
    head_tensor(*k, ko, "k", &r.k);
  } else if (a[7] != Py_None) {
    throw Refused{"k_out needs a k"};
  }
  PyObject* sections = PySequence_Fast(a[4], "sections must be a sequence of integers");
  if (!sections) throw Raised{};
  const Py_ssize_t axes = PySequence_Fast_GET_SIZE(sections);
  long long pairs = 0;
  try {
    if (axes < 1 || axes > MB_ROTARY_MAX_AXES)
      throw Refused{"sections has " + std::to_string(axes) + " axes, expected 1 to " +
                    std::to_string(MB_ROTARY_MAX_AXES)};
    for (Py_ssize_t i = 0; i < axes; ++i) {
      const long long v = integer(PySequence_Fast_GET_ITEM(sections, i), "a section");
      if (v < -(1 << 30) || v > (1 << 30)) throw Refused{"a section is out of range"};
      r.sections[i] = static_cast<int32_t>(v);
      pairs += v;
    }
  } catch (...) {
    Py_DECREF(sections);
    throw;
  }
  Py_DECREF(sections);
  r.axes = static_cast<int32_t>(axes);
  const Tensor& freq = tensor(a[3], "inv_freq");
  if (pairs != freq.numel())
    throw Refused{"sections add up to " + std::to_string(pairs) + " pairs, inv_freq has " +
                  std::to_string(freq.numel())};
  r.pairs = static_cast<int32_t>(pairs);
  r.inv_freq = static_cast<const float*>(dense(&freq, "inv_freq", {pairs}, ScalarType::Float, device));
  const Tensor& pos = tensor(a[2], "positions");
  switch (pos.scalar_type()) {
    case ScalarType::Int: r.position_type = MB_I32; break;
    case ScalarType::Long: r.position_type = MB_I64; break;
    case ScalarType::Float: r.position_type = MB_F32; break;
    default:
      throw Refused{std::string("positions has dtype ") + c10::toString(pos.scalar_type()) +
                    ", expected int32, int64 or float32"};
  }
  if (pos.dim() == 2) {   // the same positions in every sequence
    like(pos, "positions", {axes, r.tokens}, pos.scalar_type(), device);
    r.pos_token = pos.stride(1);
  } else {
    like(pos, "positions", {axes, r.batch, r.tokens}, pos.scalar_type(), device);
    r.pos_batch = pos.stride(1);
    r.pos_token = pos.stride(2);
  }
  r.pos_axis = pos.stride(0);
  r.positions = pos.data_ptr();
  checked(name, unlocked([&] { return CALL(&r, where.stream); }));
  return tuple(give(a[6], qo), give(a[7], ko));
}

// ---------------------------------------------------------------- router

const uint8_t* valid_of(PyObject* o, int64_t tokens, c10::Device device) {
  const Tensor* v = tensor_or_none(o, "valid");
  if (!v) return nullptr;
  if (v->scalar_type() != ScalarType::Bool && v->scalar_type() != ScalarType::Byte)
    throw Refused{std::string("valid has dtype ") + c10::toString(v->scalar_type()) + ", expected bool or uint8"};
  return static_cast<const uint8_t*>(dense(v, "valid", {tokens}, v->scalar_type(), device));
}

// logits, top_k, valid, normalize, index, gate, counts, loss, used, workspace, stream
PyObject* router(PyObject* const* a, Py_ssize_t n) {
  const Tensor& l = cuda_tensor(a[0], "logits");
  const auto device = l.device();
  Where where(l, a[10], a, n);
  const int type = type_of(l, "logits");
  if (l.dim() != 2) throw Refused{"logits must be [tokens, experts]"};
  const int64_t tokens = l.size(0), experts = l.size(1);
  const long long k = integer(a[1], "top_k");
  if (k < 1 || k > experts || k > 1 << 20) checked("mb_router", MB_ERR_SHAPE);
  const uint8_t* valid = valid_of(a[2], tokens, device);
  const int normalize = truth(a[3]);
  size_t need = 0;
  checked("mb_router_workspace_bytes", mb_router_workspace_bytes(tokens, experts, &need));
  const Workspace ws(a[9], need, device);
  // what belongs to tokens apart from the rest: a loss that is kept must not keep the tokens' results
  Together each(device), all(device);
  const size_t index_at = each.room(a[4], tokens * k), gate_at = each.room(a[5], tokens * k);
  const size_t counts_at = all.room(a[6], experts), loss_at = all.room(a[7], 1), used_at = all.room(a[8], 1);
  each.allocate();
  all.allocate();
  const Tensor index = each.take(a[4], "index", {tokens, k}, ScalarType::Int, index_at);
  const Tensor gate = each.take(a[5], "gate", {tokens, k}, ScalarType::Float, gate_at);
  const Tensor counts = all.take(a[6], "counts", {experts}, ScalarType::Int, counts_at);
  const Tensor loss = all.take(a[7], "loss", {1}, ScalarType::Float, loss_at);
  const Tensor used = all.take(a[8], "used", {1}, ScalarType::Int, used_at);
  auto* ip = static_cast<int32_t*>(dense(&index, "index", {tokens, k}, ScalarType::Int, device));
  auto* gp = static_cast<float*>(dense(&gate, "gate", {tokens, k}, ScalarType::Float, device));
  auto* cp = static_cast<int32_t*>(dense(&counts, "counts", {experts}, ScalarType::Int, device));
  auto* lossp = static_cast<float*>(dense(&loss, "loss", {1}, ScalarType::Float, device));
  auto* usedp = static_cast<int32_t*>(dense(&used, "used", {1}, ScalarType::Int, device));
  const void* lp = l.data_ptr();
  const int64_t stride = row_stride(l, "logits");
  checked("mb_router", unlocked([&] {
            return mb_router(lp, stride, type, valid, tokens, experts, static_cast<int>(k), normalize, ip, gp, cp, lossp,
                             usedp, ws.ptr, ws.bytes, where.stream);
          }));
  return tuple(give(a[4], index), give(a[5], gate), give(a[6], counts), give(a[7], loss), give(a[8], used));
}

// dloss, dgate, logits, index, gate, counts, used, valid, normalize, dlogits, stream
PyObject* router_backward(PyObject* const* a, Py_ssize_t n) {
  const Tensor& l = cuda_tensor(a[2], "logits");
  const auto device = l.device();
  Where where(l, a[10], a, n);
  const int type = type_of(l, "logits");
  const Tensor& index = tensor(a[3], "index");
  if (l.dim() != 2) throw Refused{"logits must be [tokens, experts]"};
  if (index.dim() != 2) throw Refused{"index must be [tokens, top_k]"};
  const int64_t tokens = l.size(0), experts = l.size(1), k = index.size(1);
  if (k < 1 || k > experts) checked("mb_router_backward", MB_ERR_SHAPE);
  const Tensor dl = result(a[9], "dlogits", l.sizes(), l.scalar_type(), device);
  const auto f32 = ScalarType::Float, i32 = ScalarType::Int;
  const auto* dlossp = static_cast<const float*>(dense(tensor_or_none(a[0], "dloss"), "dloss", {1}, f32, device));
  const auto* dgatep = static_cast<const float*>(dense(tensor_or_none(a[1], "dgate"), "dgate", {tokens, k}, f32, device));
  const uint8_t* valid = valid_of(a[7], tokens, device);
  const int normalize = truth(a[8]);
  const auto* ip = static_cast<const int32_t*>(dense(&index, "index", {tokens, k}, i32, device));
  const auto* gp = static_cast<const float*>(dense(&tensor(a[4], "gate"), "gate", {tokens, k}, f32, device));
  const auto* cp = static_cast<const int32_t*>(dense(&tensor(a[5], "counts"), "counts", {experts}, i32, device));
  const auto* usedp = static_cast<const int32_t*>(dense(&tensor(a[6], "used"), "used", {1}, i32, device));
  const void* lp = l.data_ptr();
  void* dlp = dl.data_ptr();
  const int64_t stride = row_stride(l, "logits"), dl_stride = row_stride(dl, "dlogits");
  checked("mb_router_backward", unlocked([&] {
            return mb_router_backward(dlossp, dgatep, lp, stride, type, valid, tokens, experts, static_cast<int>(k),
                                      normalize, ip, gp, cp, usedp, dlp, dl_stride, where.stream);
          }));
  return give(a[9], dl);
}

// ---------------------------------------------------------------- linear

int activation_of(PyObject* o) {
  const char* names[] = {"none", "relu", "relu2", "silu", "gelu"};
  if (PyUnicode_Check(o))
    for (int i = 0; i < 5; ++i)
      if (PyUnicode_CompareWithASCIIString(o, names[i]) == 0) return i;
  throw Refused{"activation must be 'none', 'relu', 'relu2', 'silu' or 'gelu'"};
}

struct LinearShape {
  int64_t rows, in, out, groups;
  int type;
  const int32_t* ends;
  c10::DimVector lead;        // of x, without its last dimension
  c10::DimVector param;       // of a bias
};

// Of x and w; in a backward call one of them may be absent, and dy stands in for what it would say.
LinearShape linear_shape(const Tensor* x, const Tensor* w, PyObject* ends, const Tensor* dy = nullptr) {
  LinearShape s{};
  const Tensor& rows = x ? *x : *dy;
  const char* const rows_name = x ? "x" : "dy";
  if (rows.dim() < 1) throw Refused{std::string(rows_name) + " must have at least one dimension"};
  if (w && w->dim() != 2 && w->dim() != 3) throw Refused{"weight must be [out, in], or [groups, out, in] with ends"};
  if (rows.scalar_type() != ScalarType::BFloat16 && rows.scalar_type() != ScalarType::Half)
    throw Refused{std::string(rows_name) + " has dtype " + c10::toString(rows.scalar_type()) + ", expected bfloat16 or float16"};
  s.type = type_of(rows, rows_name);
  const Tensor* e = tensor_or_none(ends, "ends");
  if (w) {
    const auto wn = w->sizes();
    s.in = wn[w->dim() - 1];
    s.out = wn[w->dim() - 2];
    s.groups = w->dim() == 3 ? wn[0] : 1;
    if (s.in == 0 || s.out == 0 || s.groups == 0) throw Refused{"weight has no elements"};
    s.param.assign(wn.begin(), wn.end() - 1);
  } else {
    if (dy->dim() < 1) throw Refused{"dy must have at least one dimension"};
    s.in = x ? x->sizes().back() : 1;
    s.out = dy->sizes().back();
    s.groups = e ? e->numel() : 1;
    if (s.in == 0 || s.out == 0 || s.groups == 0) throw Refused{"the weight would have no elements"};
    if (e) s.param.push_back(s.groups);
    s.param.push_back(s.out);
  }
  if (s.in > 1 << 20 || s.out > 1 << 20 || s.groups > 1024) checked("mb_linear", MB_ERR_SHAPE);
  const int64_t last = x ? s.in : s.out;
  if (rows.sizes().back() != last)
    throw Refused{std::string(rows_name) + " is " + str(rows) + ", its last dimension must be the weight's " + std::to_string(last)};
  if (w) dense(w, "weight", w->sizes(), rows.scalar_type(), rows.device());
  s.rows = rows.numel() / last;
  if (s.rows > 1ll << 30) checked("mb_linear", MB_ERR_SHAPE);
  s.lead.assign(rows.sizes().begin(), rows.sizes().end() - 1);
  if (w && (e != nullptr) != (w->dim() == 3))
    throw Refused{e ? "ends needs a weight of [groups, out, in]" : "a weight of [groups, out, in] needs ends"};
  if (e) s.ends = static_cast<const int32_t*>(dense(e, "ends", {s.groups}, ScalarType::Int, rows.device()));
  return s;
}

c10::DimVector with(const c10::DimVector& lead, int64_t last) {
  c10::DimVector d(lead);
  d.push_back(last);
  return d;
}

// Where a tensor of a call lies: rows of `width` bytes, `step` bytes apart.
struct Place {
  const char* name;
  const void* at;          // or null: there is none
  int64_t rows, width, step;
  uintptr_t begin() const { return reinterpret_cast<uintptr_t>(at); }
  uintptr_t end() const { return begin() + static_cast<uintptr_t>((rows - 1) * step + width); }
};
Place place_of(const char* name, const void* at, int64_t rows, int64_t cols, int64_t stride, int64_t size = 2) {
  return {name, rows > 0 && cols > 0 ? at : nullptr, stride == 0 ? 1 : rows, cols * size, stride * size};   // (one row for all)
}
Place bytes_at(const char* name, const void* at, size_t bytes) {
  return {name, bytes > 0 ? at : nullptr, 1, static_cast<int64_t>(bytes), static_cast<int64_t>(bytes)};
}

// Whether any byte of one is a byte of the other.  Views of one buffer side by side are apart.
bool overlap(const Place& a, const Place& b) {
  if (!a.at || !b.at || a.begin() >= b.end() || b.begin() >= a.end()) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  const Place &few = a.rows <= b.rows ? a : b, &many = a.rows <= b.rows ? b : a;
  if (a.step == b.step && a.step >= a.width && a.step >= b.width) {
    // columns of rows of one width: a's begin at 0, b's at d, and wrap around
    const int64_t apart = static_cast<int64_t>(b.begin()) - static_cast<int64_t>(a.begin());
    const int64_t d = (apart % a.step + a.step) % a.step;
    return d < a.width || d + b.width > a.step;
  }
  for (int64_t i = 0; i < few.rows; ++i) {       // each row of one: the rows of the other that end past its begin
    const auto lo = static_cast<int64_t>(few.begin() + i * few.step), hi = lo + few.width, at = static_cast<int64_t>(many.begin());
    int64_t first = 0;
    if (many.step > 0 && lo >= at + many.width) first = (lo - at - many.width) / many.step + 1;
    if (first < many.rows && at + first * many.step < hi && at + first * many.step + many.width > lo) return true;
  }
  return false;
}

// Results that share memory with an input of the call, or with another result.
void apart(std::initializer_list<Place> results, std::initializer_list<Place> inputs) {
  for (auto r = results.begin(); r != results.end(); ++r) {
    if (!r->at) continue;
    for (const auto& i : inputs)
      if (overlap(*r, i)) throw Refused{std::string(r->name) + " may not be written over " + i.name};
    for (auto o = results.begin(); o != r; ++o)
      if (overlap(*r, *o)) throw Refused{std::string(r->name) + " may not be written over " + o->name};
  }
}

// x, weight, bias, residual, activation, ends, keep, y, z, workspace, stream
PyObject* linear(PyObject* const* a, Py_ssize_t n) {
  const Tensor &x = cuda_tensor(a[0], "x"), &w = tensor(a[1], "weight");
  const auto device = x.device();
  const auto dtype = x.scalar_type();
  Where where(x, a[10], a, n);
  const LinearShape s = linear_shape(&x, &w, a[5]);
  const auto shape = with(s.lead, s.out);
  mb_linear_desc d{};
  d.activation = activation_of(a[4]);
  const Tensor* bias = tensor_or_none(a[2], "bias");
  d.bias_type = MB_F32;
  if (bias) {
    if (bias->scalar_type() != dtype && bias->scalar_type() != ScalarType::Float)
      throw Refused{std::string("bias has dtype ") + c10::toString(bias->scalar_type()) + ", expected x's or float32"};
    d.bias_type = type_of(*bias, "bias");
    d.bias = dense(bias, "bias", s.param, bias->scalar_type(), device);
  }
  const Tensor* residual = tensor_or_none(a[3], "residual");
  if (residual) {
    like(*residual, "residual", shape, dtype, device);
    d.residual = residual->data_ptr();
    d.residual_stride = row_stride(*residual, "residual");
  }
  const Tensor y = result(a[7], "y", shape, dtype, device);
  Tensor z;
  if (a[8] != Py_None || truth(a[6])) {
    z = result(a[8], "z", shape, dtype, device);
    d.z = z.data_ptr();
    d.z_stride = row_stride(z, "z");
  }
  d.x = x.data_ptr();
  d.x_stride = row_stride(x, "x");
  d.weight = w.data_ptr();
  d.ends = s.ends;
  d.y = y.data_ptr();
  d.y_stride = row_stride(y, "y");
  d.rows = s.rows;
  d.in = static_cast<int32_t>(s.in);
  d.out = static_cast<int32_t>(s.out);
  d.groups = static_cast<int32_t>(s.groups);
  d.type = s.type;
  size_t need = 0;
  checked("mb_linear_workspace_bytes", mb_linear_workspace_bytes(&d, &need));
  const Workspace ws(a[9], need, device);
  const Place residual_at = place_of("residual", d.residual, s.rows, s.out, d.residual_stride);
  const Place z_at = place_of("z", d.z, s.rows, s.out, d.z_stride), scratch = bytes_at("workspace", ws.ptr, need);
  const bool over = d.y == d.residual && (d.y_stride == d.residual_stride || s.rows <= 1);      // each element over its own
  apart({place_of("y", d.y, s.rows, s.out, d.y_stride), z_at, scratch},
        {place_of("x", d.x, s.rows, s.in, d.x_stride), bytes_at("weight", d.weight, w.nbytes()),
         bytes_at("bias", d.bias, bias ? bias->nbytes() : 0), bytes_at("ends", d.ends, s.groups * 4), over ? Place{} : residual_at});
  if (over) apart({z_at, scratch}, {residual_at});
  checked("mb_linear", unlocked([&] { return mb_linear(&d, ws.ptr, ws.bytes, where.stream); }));
  return tuple(give(a[7], y), give(a[8], z));
}

// dy, x, weight, z, activation, ends, input_grad, weight_grad, bias (whether its gradient is wanted), dx, dweight, dbias,
// workspace, stream
PyObject* linear_backward(PyObject* const* a, Py_ssize_t n) {
  const Tensor& dy = cuda_tensor(a[0], "dy");
  const Tensor *x = tensor_or_none(a[1], "x"), *w = tensor_or_none(a[2], "weight");
  const auto device = dy.device();
  const auto dtype = dy.scalar_type();
  Where where(dy, a[13], a, n);
  const bool want_dx = a[9] != Py_None || truth(a[6]), want_dw = a[10] != Py_None || truth(a[7]);
  if (want_dx && !w) throw Refused{"the gradient of x needs the weight"};
  if (want_dw && !x) throw Refused{"the gradient of the weight needs x"};
  const LinearShape s = linear_shape(x, w, a[5], &dy);
  const auto shape = with(s.lead, s.out);
  if (x && (x->device() != device || x->scalar_type() != dtype))
    throw Refused{"x is " + str(*x) + ", dy " + str(dy) + ": expected one type and device"};
  mb_linear_backward_desc d{};
  d.activation = activation_of(a[4]);
  like(dy, "dy", shape, dtype, device);
  d.dy = dy.data_ptr();
  d.dy_stride = row_stride(dy, "dy");
  if (d.activation != MB_ACT_NONE) {
    const Tensor* z = tensor_or_none(a[3], "z");
    if (!z) throw Refused{"the gradient of an activation needs z (keep=True in the forward call)"};
    like(*z, "z", shape, dtype, device);
    d.z = z->data_ptr();
    d.z_stride = row_stride(*z, "z");
  }
  Tensor dx, dw, db;
  if (want_dx) {
    dx = result(a[9], "dx", with(s.lead, s.in), dtype, device);
    d.dx = dx.data_ptr();
    d.dx_stride = row_stride(dx, "dx");
  }
  if (want_dw) {
    const auto matrices = with(s.param, s.in);
    dw = result(a[10], "dweight", matrices, dtype, device);
    d.dweight = dense(&dw, "dweight", matrices, dtype, device);
    d.x = x->data_ptr();
    d.x_stride = row_stride(*x, "x");
  }
  d.bias_type = s.type;
  if (a[11] != Py_None || truth(a[8])) {
    const Tensor* given = tensor_or_none(a[11], "dbias");
    auto type = dtype;
    if (given && given->scalar_type() == ScalarType::Float) {
      type = ScalarType::Float;
      d.bias_type = MB_F32;
    }
    db = result(a[11], "dbias", s.param, type, device);
    d.dbias = dense(&db, "dbias", s.param, type, device);
  }
  if (want_dx) d.weight = w->data_ptr();
  d.ends = s.ends;
  d.rows = s.rows;
  d.in = static_cast<int32_t>(s.in);
  d.out = static_cast<int32_t>(s.out);
  d.groups = static_cast<int32_t>(s.groups);
  d.type = s.type;
  size_t need = 0;
  checked("mb_linear_backward_workspace_bytes", mb_linear_backward_workspace_bytes(&d, &need));
  const Workspace ws(a[12], need, device);
  apart({place_of("dx", d.dx, s.rows, s.in, d.dx_stride), bytes_at("dweight", d.dweight, dw.defined() ? dw.nbytes() : 0),
         bytes_at("dbias", d.dbias, db.defined() ? db.nbytes() : 0), bytes_at("workspace", ws.ptr, need)},
        {place_of("dy", d.dy, s.rows, s.out, d.dy_stride), place_of("x", d.x, s.rows, s.in, d.x_stride),
         bytes_at("weight", d.weight, want_dx ? w->nbytes() : 0), place_of("z", d.z, s.rows, s.out, d.z_stride),
         bytes_at("ends", d.ends, s.groups * 4)});
  checked("mb_linear_backward", unlocked([&] { return mb_linear_backward(&d, ws.ptr, ws.bytes, where.stream); }));
  return tuple(give(a[9], dx), give(a[10], dw), give(a[11], db));
}

// ---------------------------------------------------------------- AdamW

// The tensors of a call as descriptors, and the ones that it writes.
struct AdamwList {
  static constexpr const char* NAMES[7] = {"param", "grad", "exp_avg", "exp_avg_sq", "mantissa", "avg_scale", "sq_scale"};
  std::vector<mb_adamw_tensor> descs;
  std::vector<const Tensor*> written;      // held by the call's list, which `seq` and `items` hold
  std::vector<PyObject*> held;
  Tensor first;
  c10::Device device = c10::Device(c10::kCPU);

  // The memory of every tensor of the list, field by field; an empty one has none.
  struct Range {
    uintptr_t begin = 0, end = 0;
  };
  std::vector<Range> memory;
  bool present[7] = {};

  static std::string name(int field, Py_ssize_t at) { return std::string(NAMES[field]) + " of tensor " + std::to_string(at); }

  void* place(const Tensor& t, int field, Py_ssize_t at, int64_t n, ScalarType dtype, ScalarType also) {
    if (t.scalar_type() != dtype && t.scalar_type() != also)
      throw Refused{name(field, at) + " has dtype " + c10::toString(t.scalar_type()) + ", expected " + c10::toString(dtype)};
    if (t.numel() != n)
      throw Refused{name(field, at) + " has " + std::to_string(t.numel()) + " elements, expected " + std::to_string(n)};
    if (t.device() != device) throw Refused{name(field, at) + " is on " + t.device().str() + ", expected " + device.str()};
    if (!t.is_contiguous()) throw Refused{name(field, at) + " must be contiguous"};
    if (field != 1) written.push_back(&t);
    void* p = t.data_ptr();
    if (n > 0) {
      const auto at_byte = reinterpret_cast<uintptr_t>(p);
      memory[field * (memory.size() / 7) + at] = {at_byte, at_byte + static_cast<size_t>(n) * t.element_size()};
      present[field] = true;
    }
    return p;
  }

  void add(PyObject* const* f, Py_ssize_t at) {
    mb_adamw_tensor d{};
    const Tensor &param = cuda_tensor(f[0], NAMES[0]), &grad = tensor(f[1], NAMES[1]);
    const Tensor &avg = tensor(f[2], NAMES[2]), &sq = tensor(f[3], NAMES[3]);
    const Tensor *low = tensor_or_none(f[4], NAMES[4]);
    const Tensor* scale[2] = {tensor_or_none(f[5], NAMES[5]), tensor_or_none(f[6], NAMES[6])};
    if (at == 0) {
      first = param;
      device = param.device();
    }
    d.n = param.numel();
    d.param_type = type_of(param, NAMES[0]);
    d.grad_type = type_of(grad, NAMES[1]);
    const auto none = ScalarType::Undefined;
    d.param = place(param, 0, at, d.n, param.scalar_type(), none);
    if (grad.sizes() != param.sizes()) throw Refused{name(1, at) + " is " + str(grad) + ", its parameter " + str(param)};
    d.grad = place(grad, 1, at, d.n, grad.scalar_type(), none);
    const bool eight = avg.scalar_type() == ScalarType::Float8_e4m3fn;
    const auto state = eight ? ScalarType::Float8_e4m3fn : ScalarType::Float;
    d.state_type = eight ? MB_E4M3 : MB_F32;
    d.exp_avg = place(avg, 2, at, d.n, state, none);
    d.exp_avg_sq = place(sq, 3, at, d.n, state, none);
    if (low) {
      if (param.scalar_type() != ScalarType::BFloat16) throw Refused{name(4, at) + " needs a bfloat16 parameter"};
      d.mantissa = static_cast<uint16_t*>(place(*low, 4, at, d.n, ScalarType::Short, ScalarType::UInt16));
    }
    for (int i = 0; i < 2; ++i) {
      if (eight != (scale[i] != nullptr))
        throw Refused{name(5 + i, at) + (eight ? " is missing: 8-bit moments need it" : " is for 8-bit moments only")};
      if (eight)
        (i == 0 ? d.avg_scale : d.sq_scale) =
            static_cast<float*>(place(*scale[i], 5 + i, at, (d.n + 255) / 256, ScalarType::Float, none));
    }
    d.lr_mul = number(f[7]);
    d.wd_mul = number(f[8]);
    descs.push_back(d);
  }

  static Range range_of(const void* p, size_t bytes) {
    const auto begin = reinterpret_cast<uintptr_t>(p);
    return p ? Range{begin, begin + bytes} : Range{};
  }

  // What the call reads or writes beside the list.
  struct Beside {
    const char* name;
    Range range;
    bool written;
  };

  // One field's memory over the list: from the first byte to the last, and whether the tensors ascend (or descend) apart.
  struct Field {
    const Range* at;
    Range whole;
    bool up = true, down = true;
    explicit Field(const Range* at_, size_t n) : at(at_) {
      Range last;
      for (size_t i = 0; i < n; ++i) {
        const Range& r = at[i];
        if (r.end == 0) continue;
        if (last.end > 0) {
          up &= r.begin >= last.end;
          down &= r.end <= last.begin;
        }
        last = r;
        whole.begin = whole.end == 0 ? r.begin : std::min(whole.begin, r.begin);
        whole.end = std::max(whole.end, r.end);
      }
    }
    // Whether two fields, each in order, share a byte.
    bool meets(const Field& o, size_t n) const {
      for (size_t i = 0, j = 0; i < n && j < n;) {
        const Range &a = at[up ? i : n - 1 - i], &b = o.at[o.up ? j : n - 1 - j];
        if (a.end <= b.begin || a.end == 0) ++i;
        else if (b.end <= a.begin) ++j;
        else return true;
      }
      return false;
    }
  };

  // Nothing that the call writes may be in two places of it: two CTAs would step it at once.  (What is only read may.)  Where each
  // field's tensors are in the order of their memory, as allocated in turn or cut from one buffer, the fields are compared
  // side by side; else all are sorted (50 tensors of four fields: 1 and 2 us).
  void check_memory(std::initializer_list<Beside> beside) const {
    const size_t n = descs.size();
    std::optional<Field> fields[7];
    bool apart = true;
    const auto clear = [](const Range& a, const Range& b) { return a.begin >= b.end || b.begin >= a.end; };
    for (int f = 0; f < 7 && apart; ++f) {
      if (!present[f]) continue;
      const Field& w = fields[f].emplace(&memory[f * n], n);
      apart = w.up || w.down;
      for (int g = 0; g < f && apart; ++g)
        if (fields[g] && !clear(fields[g]->whole, w.whole)) apart = !fields[g]->meets(w, n);
      for (const Beside& b : beside)
        if (!clear(b.range, w.whole))
          for (size_t i = 0; i < n && apart; ++i) apart = clear(b.range, w.at[i]);
    }
    for (auto b = beside.begin(); b != beside.end(); ++b)
      for (auto o = beside.begin(); o != b; ++o) apart = apart && clear(b->range, o->range);
    if (apart) return;
    // by first byte: what is written begins behind all before it, what is read behind all that is written
    std::vector<std::pair<uintptr_t, size_t>> order;
    order.reserve(memory.size() + beside.size());
    const auto range = [&](size_t i) { return i < memory.size() ? memory[i] : beside.begin()[i - memory.size()].range; };
    for (size_t i = 0; i < memory.size() + beside.size(); ++i)
      if (range(i).end > 0) order.emplace_back(range(i).begin, i);
    std::sort(order.begin(), order.end());
    size_t last = 0, last_written = 0;     // of those so far, the ones that end last, as places in `order`
    uintptr_t end = 0, end_written = 0;
    const auto title = [&](size_t k) {
      const size_t i = order[k].second;
      return i < memory.size() ? name(static_cast<int>(i / n), static_cast<Py_ssize_t>(i % n))
                               : std::string(beside.begin()[i - memory.size()].name);
    };
    for (size_t k = 0; k < order.size(); ++k) {
      const size_t i = order[k].second;
      const bool writes = i < memory.size() ? i / n != 1 : beside.begin()[i - memory.size()].written;
      if (order[k].first < (writes ? end : end_written))
        throw Refused{"memory that the call writes overlaps: " + title(writes ? last : last_written) + " and " + title(k)};
      const uintptr_t e = range(i).end;
      if (e > end) end = e, last = k;
      if (writes) end_written = e, last_written = k;
    }
  }

  explicit AdamwList(PyObject* list) {
    try {
      PyObject* seq = PySequence_Fast(list, "tensors must be a sequence of AdamState");
      if (!seq) throw Raised{};
      held.push_back(seq);
      const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
      if (n == 0) throw Refused{"no tensors"};
      if (n > MB_ADAMW_MAX_TENSORS) checked("adamw_multi_step", MB_ERR_TOO_MANY);
      descs.reserve(n);
      written.reserve(5 * n);
      memory.resize(7 * n);
      held.reserve(n + 1);
      for (Py_ssize_t i = 0; i < n; ++i) {
        PyObject* item = PySequence_Fast_GET_ITEM(seq, i);
        if (!PyTuple_Check(item) || PyTuple_GET_SIZE(item) != 9) throw Refused{"each tensor of the call is an AdamState"};
        held.push_back(Py_NewRef(item));       // other threads may change the list while the call launches
        PyObject* f[9];
        for (int k = 0; k < 9; ++k) f[k] = PyTuple_GET_ITEM(item, k);
        add(f, i);
      }
    } catch (...) {
      release();
      throw;
    }
  }
  AdamwList(const AdamwList&) = delete;
  ~AdamwList() { release(); }
  void release() {
    for (PyObject* o : held) Py_DECREF(o);
    held.clear();
  }

  // Marks the tensors as used on the stream that the call was given.
  void record(cudaStream_t stream) const {
    const auto s = c10::cuda::getStreamFromExternal(stream, device.index()).unwrap();
    for (size_t i = 1; i < held.size(); ++i)
      for (int k = 0; k < 7; ++k) {
        PyObject* t = PyTuple_GET_ITEM(held[i], k);
        if (t != Py_None) THPVariable_Unpack(t).record_stream(s);
      }
  }
  void stepped() const {
    for (const Tensor* t : written)
      if (!t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
  }
};

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

// The seed of stochastic rounding (None: to the nearest).
uint32_t seed_of(PyObject* o, int* stochastic) {
  *stochastic = o != Py_None;
  if (!*stochastic) return 0;
  const long long v = integer(o, "seed");
  if (v < 0 || v >= (1ll << 32)) throw Refused{"seed is out of range: 0 to 2^32 - 1"};
  return static_cast<uint32_t>(v);
}

// A clipping factor: one fp32 value, as a scalar tensor (what a norm gives) or of one dimension.
const float* factor(PyObject* o, c10::Device device) {
  const Tensor* t = tensor_or_none(o, "grad_scale");
  const int64_t one = 1;
  const c10::IntArrayRef shape(&one, t && t->dim() == 0 ? 0 : 1);
  return static_cast<const float*>(dense(t, "grad_scale", shape, ScalarType::Float, device));
}

// tensors, lr, wd, beta1, beta2, eps, step, grad_scale, seed, stream
PyObject* adamw(PyObject* const* a, Py_ssize_t n) {
  const AdamwList list(a[0]);
  Where where(list.first, a[9], a, n);
  if (a[9] != Py_None) list.record(where.stream);
  const double lr = real(a[1]), wd = real(a[2]), beta1 = real(a[3]), beta2 = real(a[4]), eps = real(a[5]);
  const long long step = integer(a[6], "step");
  const float* scale = factor(a[7], list.device);
  int stochastic = 0;
  const uint32_t seed = seed_of(a[8], &stochastic);
  list.check_memory({{"grad_scale", AdamwList::range_of(scale, 4), false}});
  checked("adamw_multi_step", unlocked([&] {
            return adamw_multi_step(list.descs.data(), static_cast<int>(list.descs.size()), lr, wd, beta1, beta2, eps, step,
                                    scale, stochastic, seed, where.stream);
          }));
  list.stepped();
  Py_RETURN_NONE;
}

// tensors, scalars, grad_scale, seed, workspace, stream
PyObject* adamw_dev(PyObject* const* a, Py_ssize_t n) {
  const AdamwList list(a[0]);
  Where where(list.first, a[5], a, n);
  if (a[5] != Py_None) list.record(where.stream);
  const auto* scalars =
      static_cast<const double*>(dense(&tensor(a[1], "scalars"), "scalars", {6}, ScalarType::Double, list.device));
  const float* scale = factor(a[2], list.device);
  int stochastic = 0;
  const uint32_t seed = seed_of(a[3], &stochastic);
  const int count = static_cast<int>(list.descs.size());
  size_t need = 0;
  checked("adamw_multi_step_dev_workspace_bytes", adamw_multi_step_dev_workspace_bytes(count, &need));
  const Workspace ws(a[4], need, list.device);
  list.check_memory({{"grad_scale", AdamwList::range_of(scale, 4), false},
                     {"scalars", AdamwList::range_of(scalars, 48), false},
                     {"workspace", AdamwList::range_of(ws.ptr, need), true}});
  checked("adamw_multi_step_dev", unlocked([&] {
            return adamw_multi_step_dev(list.descs.data(), count, scalars, scale, stochastic, seed, ws.ptr, ws.bytes,
                                        where.stream);
          }));
  list.stepped();
  return a[4] == Py_None ? wrap(ws.own) : Py_NewRef(a[4]);
}

// ---------------------------------------------------------------- the module

PyObject* rotary_forward(PyObject* const* a, Py_ssize_t n) { return rotary<mb_rotary>(a, n, "mb_rotary"); }
PyObject* rotary_backward(PyObject* const* a, Py_ssize_t n) {
  return rotary<mb_rotary_backward>(a, n, "mb_rotary_backward");
}

// No C++ exception leaves a call: each becomes the Python exception it stands for.
template <PyObject* (*CALL)(PyObject* const*, Py_ssize_t), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != N) return PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, nargs);
  try {
    return CALL(args, nargs);
  } catch (const Raised&) {
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.text.c_str());
  } catch (const std::bad_alloc&) {
    PyErr_NoMemory();
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_out_of_memory, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <PyObject* (*CALL)(PyObject* const*, Py_ssize_t), Py_ssize_t N>
constexpr PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<CALL, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<layer_norm, 8>("mb_layer_norm"),
                           method<layer_norm_backward, 12>("mb_layer_norm_backward"),
                           method<rotary_forward, 9>("mb_rotary"),
                           method<rotary_backward, 9>("mb_rotary_backward"),
                           method<router, 11>("mb_router"),
                           method<router_backward, 11>("mb_router_backward"),
                           method<linear, 11>("mb_linear"),
                           method<linear_backward, 14>("mb_linear_backward"),
                           method<adamw, 10>("adamw_multi_step"),
                           method<adamw_dev, 6>("adamw_multi_step_dev"),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_blocks", "Native calls of the block operators.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__blocks() {
  PyObject* binding = PyImport_ImportModule("newton_schulz_stacked_gb300._binding");
  PyObject* torch = binding ? PyImport_ImportModule("torch") : nullptr;
  if (torch) {
    g_check = PyObject_GetAttrString(binding, "check");
    g_out_of_memory = PyObject_GetAttrString(torch, "OutOfMemoryError");
  }
  Py_XDECREF(binding);
  Py_XDECREF(torch);
  return g_check && g_out_of_memory ? PyModule_Create(&g_module) : nullptr;
}
