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

#include <optional>
#include <string>

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
