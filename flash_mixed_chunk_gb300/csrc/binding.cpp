// binding.cpp -- the allocating Python wrappers of the training operators
// (layer_norm, layer_norm_backward, gau_project_backward, gau_output_backward,
// vocab_loss, vocab_loss_backward) as a CPython module.
//
// A call is checks, up to four tensors from torch's allocator and one call of
// the C ABI (include/flash_mca.h): at one token the device work is 3 us and the
// same steps taken in Python cost 18 us a call.  Every check raises before
// anything is queued.  The tensors are allocated for, and the work queued on,
// torch's current stream of the operands' device.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "flash_mca.h"

namespace {

PyObject *g_error = nullptr;  // the package's FmcaError(status, what)

[[noreturn]] void fail(PyObject *type, const std::string &msg) {
  PyErr_SetString(type, msg.c_str());
  throw python_error();
}

void check(fmca_status st, const char *what) {
  if (st == FMCA_OK) return;
  PyObject *e = PyObject_CallFunction(g_error, "is", (int)st, what);
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw python_error();
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

const at::Tensor &tensor(const char *name, PyObject *o) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

const at::Tensor &cuda_tensor(const char *name, PyObject *o) {
  const at::Tensor &t = tensor(name, o);
  if (!t.is_cuda()) fail(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
  return t;
}

// The device address of a contiguous tensor of this type and shape on `dev`.
void *on(const char *name, const at::Tensor &t, at::ScalarType type, at::IntArrayRef shape,
         const at::Device &dev) {
  if (t.scalar_type() != type || t.sizes() != shape || t.device() != dev || !t.is_contiguous())
    fail(PyExc_ValueError, std::string(name) + " must be a contiguous " + at::toString(type) +
                               " tensor of shape " + shape_text(shape) + " on " + dev.str() +
                               ", got " + at::toString(t.scalar_type()) + " " +
                               shape_text(t.sizes()) + " on " + t.device().str() +
                               (t.is_contiguous() ? "" : ", not contiguous"));
  return t.data_ptr();
}
void *on(const char *name, PyObject *o, at::ScalarType type, at::IntArrayRef shape,
         const at::Device &dev) {
  return on(name, tensor(name, o), type, shape, dev);
}
const at::Tensor &matrix(const char *name, PyObject *o) {
  const at::Tensor &t = tensor(name, o);
  if (t.dim() != 2) fail(PyExc_ValueError, std::string(name) + " must be 2-D");
  return t;
}
// A size that the C ABI takes as an int.
int size_of(const char *what, int64_t v) {
  if (v > INT32_MAX) fail(PyExc_ValueError, std::string(what) + " does not fit 32 bits");
  return (int)v;
}

// torch.empty without its dispatcher
at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Device &dev) {
  return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}
// Other threads run while a call allocates (which may wait for the device) and
// queues its kernels (which waits while the stream's queue is full).
class WithoutGil {
 public:
  WithoutGil() : state_(PyEval_SaveThread()) {}
  ~WithoutGil() { PyEval_RestoreThread(state_); }
  WithoutGil(const WithoutGil &) = delete;

 private:
  PyThreadState *state_;
};
// The tensors of one call.  While they are small together they are parts of one
// allocation: an allocation and its release are 0.8 us, of a call of 5 for one
// token.  One result that is kept keeps the others' memory with it, which is of
// its own order; a workspace of more than 16 KB, which no caller knows of, and
// anything large are allocations of their own.
class Results {
 public:
  explicit Results(const at::Device &dev) : dev_(dev) {}
  int add(at::IntArrayRef shape, at::ScalarType type) {
    Item &it = items_[n_];
    it.shape = shape;
    it.type = type;
    place(it, c10::multiply_integers(shape) * (int64_t)c10::elementSize(type), kShared);
    return n_++;
  }
  // `bytes` as a ..._workspace_bytes function gave them
  int add_workspace(size_t bytes, const char *what) {
    if (bytes == 0) check(FMCA_ERR_UNSUPPORTED, what);
    Item &it = items_[n_];
    it.bytes = (int64_t)bytes;
    it.shape = at::IntArrayRef(&it.bytes, 1);
    it.type = at::kByte;
    place(it, it.bytes, kSharedWorkspace);
    return n_++;
  }
  // makes the tensors and queues the call that writes them
  template <typename F>
  fmca_status queue(const F &call) {
    const WithoutGil other_threads_run;
    make();
    return call();
  }
  const at::Tensor &operator[](int i) const { return t_[i]; }
  template <typename T = void>
  T *ptr(int i) const {
    return static_cast<T *>(t_[i].data_ptr());
  }

 private:
  void make() {
    const bool shared = total_ > 0 && total_ <= kShared;
    const at::Tensor all = shared ? ::make({total_}, at::kByte, dev_) : at::Tensor();
    for (int i = 0; i < n_; ++i) {
      if (!shared || items_[i].at < 0) {
        t_[i] = ::make(items_[i].shape, items_[i].type, dev_);
        continue;
      }
      t_[i] = at::detail::make_tensor<c10::TensorImpl>(
          c10::Storage(all.storage()), all.key_set(), c10::scalarTypeToTypeMeta(items_[i].type));
      t_[i].unsafeGetTensorImpl()->set_storage_offset(
          items_[i].at / (int64_t)c10::elementSize(items_[i].type));
      t_[i].unsafeGetTensorImpl()->set_sizes_contiguous(items_[i].shape);
    }
  }
  static constexpr int64_t kShared = 256 << 10, kSharedWorkspace = 16 << 10;
  struct Item {
    at::IntArrayRef shape;  // of an operand, or of `bytes`
    int64_t bytes, at;      // at < 0: an allocation of its own
    at::ScalarType type;
  };
  void place(Item &it, int64_t bytes, int64_t limit) {
    it.at = -1;
    if (bytes > limit) return;
    it.at = total_;
    total_ += (bytes + 255) / 256 * 256;
  }
  at::Device dev_;
  Item items_[4];
  at::Tensor t_[4];
  int n_ = 0;
  int64_t total_ = 0;
};
fmca_stream_t stream_of(const at::Device &dev) {
  return reinterpret_cast<fmca_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
}
fmca_dtype dtype_of(const at::Tensor &t) {
  if (t.scalar_type() == at::kBFloat16) return FMCA_BF16;
  if (t.scalar_type() == at::kFloat) return FMCA_F32;
  fail(PyExc_TypeError, std::string("unsupported dtype ") + at::toString(t.scalar_type()) +
                            ": use torch.bfloat16 or torch.float32");
}

void arguments(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) fail(PyExc_TypeError, "expected " + std::to_string(want) + " arguments");
}
template <typename... T>
PyObject *pack(const T &...t) {
  PyObject *r = PyTuple_New(sizeof...(t));
  if (r == nullptr) throw python_error();
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t)), ...);
  for (i = 0; i < (Py_ssize_t)sizeof...(t); ++i)
    if (PyTuple_GET_ITEM(r, i) == nullptr) {
      Py_DECREF(r);
      throw python_error();
    }
  return r;
}

// (x, weight, bias, eps, residual or None) -> (y, h, mean, rstd)
PyObject *layer_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 5);
  const at::Tensor &x = cuda_tensor("x", a[0]);
  const double eps = PyFloat_AsDouble(a[3]);
  if (eps == -1.0 && PyErr_Occurred()) throw python_error();
  if (x.dim() < 1 || x.numel() == 0)
    fail(PyExc_ValueError, "x must be [..., d] with at least one row");
  const at::Device dev = x.device();
  const fmca_dtype dt = dtype_of(x);
  const int64_t d = x.size(-1);
  const at::ScalarType type = x.scalar_type();
  const auto rows = x.sizes().slice(0, x.dim() - 1);
  const void *px = on("x", x, type, x.sizes(), dev);
  const bool has = a[4] != Py_None;
  const void *pr = has ? on("residual", a[4], type, x.sizes(), dev) : nullptr;
  const float *pw = (const float *)on("weight", a[1], at::kFloat, {d}, dev);
  const float *pb = (const float *)on("bias", a[2], at::kFloat, {d}, dev);
  const int M = size_of("the number of rows", x.numel() / d), di = size_of("d", d);
  c10::cuda::CUDAGuard guard(dev);
  Results t(dev);
  const int y = t.add(x.sizes(), type), mean = t.add(rows, at::kFloat);
  const int rstd = t.add(rows, at::kFloat), h = has ? t.add(x.sizes(), type) : y;
  check(t.queue([&] {
          return flash_mca_layer_norm(px, pr, pw, pb, has ? t.ptr(h) : nullptr, t.ptr(y),
                                      t.ptr<float>(mean), t.ptr<float>(rstd), M, di, (float)eps,
                                      dt, stream_of(dev));
        }),
        "flash_mca_layer_norm");
  if (has) return pack(t[y], t[h], t[mean], t[rstd]);
  PyObject *r = pack(t[y], t[y], t[mean], t[rstd]);  // h is the caller's x itself
  Py_DECREF(PyTuple_GET_ITEM(r, 1));
  Py_INCREF(a[0]);
  PyTuple_SET_ITEM(r, 1, a[0]);
  return r;
  END_HANDLE_TH_ERRORS
}

// (dy, h, weight, mean, rstd, dh or None) -> (dx, dweight, dbias)
PyObject *layer_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 6);
  const at::Tensor &dy = cuda_tensor("dy", a[0]);
  if (dy.dim() < 1 || dy.numel() == 0)
    fail(PyExc_ValueError, "dy must be [..., d] with at least one row");
  const at::Device dev = dy.device();
  const fmca_dtype dt = dtype_of(dy);
  const int64_t d = dy.size(-1);
  const at::ScalarType type = dy.scalar_type();
  const auto rows = dy.sizes().slice(0, dy.dim() - 1);
  const void *py = on("dy", dy, type, dy.sizes(), dev);
  const void *ph = on("h", a[1], type, dy.sizes(), dev);
  const float *pw = (const float *)on("weight", a[2], at::kFloat, {d}, dev);
  const float *pm = (const float *)on("mean", a[3], at::kFloat, rows, dev);
  const float *pr = (const float *)on("rstd", a[4], at::kFloat, rows, dev);
  const void *pd = a[5] != Py_None ? on("dh", a[5], type, dy.sizes(), dev) : nullptr;
  const int M = size_of("the number of rows", dy.numel() / d), di = size_of("d", d);
  c10::cuda::CUDAGuard guard(dev);
  Results t(dev);
  const int ws = t.add_workspace(flash_mca_layer_norm_backward_workspace_bytes(M, di),
                                 "flash_mca_layer_norm_backward_workspace_bytes");
  const int64_t vec[1] = {d};
  const int dx = t.add(dy.sizes(), type), dw = t.add(vec, at::kFloat), db = t.add(vec, at::kFloat);
  check(t.queue([&] {
          return flash_mca_layer_norm_backward(py, ph, pw, pm, pr, pd, t.ptr(dx), t.ptr<float>(dw),
                                               t.ptr<float>(db), M, di, dt, t.ptr(ws),
                                               (size_t)t[ws].numel(), stream_of(dev));
        }),
        "flash_mca_layer_norm_backward");
  return pack(t[dx], t[dw], t[db]);
  END_HANDLE_TH_ERRORS
}

// (X, Wt, dU, dV, dZ) -> (dX, dWt)
PyObject *gau_project_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 5);
  const at::Tensor &X = cuda_tensor("X", a[0]);
  matrix("X", a[0]);
  const int64_t M = X.size(0), d = X.size(1);
  const int64_t e = matrix("dU", a[2]).size(1), s = matrix("dZ", a[4]).size(1);
  const int64_t N = 2 * e + s;
  const at::Device dev = X.device();
  const auto bf = at::kBFloat16;
  const void *px = on("X", X, bf, {M, d}, dev), *pw = on("Wt", a[1], bf, {N, d}, dev);
  const void *pu = on("dU", a[2], bf, {M, e}, dev), *pv = on("dV", a[3], bf, {M, e}, dev);
  const void *pz = on("dZ", a[4], bf, {M, s}, dev);
  const int Mi = size_of("M", M), di = size_of("d", d), ei = size_of("e", e), si = size_of("s", s);
  c10::cuda::CUDAGuard guard(dev);
  const int64_t wshape[2] = {N, d};
  Results t(dev);
  const int ws = t.add_workspace(flash_mca_gau_project_backward_workspace_bytes(Mi, di, ei, si),
                                 "flash_mca_gau_project_backward_workspace_bytes");
  const int dX = t.add(X.sizes(), bf), dWt = t.add(wshape, bf);
  check(t.queue([&] {
          return flash_mca_gau_project_backward(px, pw, pu, pv, pz, t.ptr(dX), t.ptr(dWt), Mi, di,
                                                ei, si, t.ptr(ws), (size_t)t[ws].numel(),
                                                stream_of(dev));
        }),
        "flash_mca_gau_project_backward");
  return pack(t[dX], t[dWt]);
  END_HANDLE_TH_ERRORS
}

// (Y, Wo_t, dOut) -> (dY, dWo_t)
PyObject *gau_output_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 3);
  const at::Tensor &Y = cuda_tensor("Y", a[0]);
  matrix("Y", a[0]);
  const int64_t M = Y.size(0), e = Y.size(1), d = matrix("dOut", a[2]).size(1);
  const at::Device dev = Y.device();
  const auto bf = at::kBFloat16;
  const void *py = on("Y", Y, bf, {M, e}, dev), *pw = on("Wo_t", a[1], bf, {d, e}, dev);
  const void *po = on("dOut", a[2], bf, {M, d}, dev);
  const int Mi = size_of("M", M), ei = size_of("e", e), di = size_of("d", d);
  c10::cuda::CUDAGuard guard(dev);
  const int64_t wshape[2] = {d, e};
  Results t(dev);
  const int ws = t.add_workspace(flash_mca_gau_output_backward_workspace_bytes(Mi, ei, di),
                                 "flash_mca_gau_output_backward_workspace_bytes");
  const int dY = t.add(Y.sizes(), bf), dW = t.add(wshape, bf);
  check(t.queue([&] {
          return flash_mca_gau_output_backward(py, pw, po, t.ptr(dY), t.ptr(dW), Mi, ei, di,
                                               t.ptr(ws), (size_t)t[ws].numel(), stream_of(dev));
        }),
        "flash_mca_gau_output_backward");
  return pack(t[dY], t[dW]);
  END_HANDLE_TH_ERRORS
}

// (X, W, target) -> (loss, lse)
PyObject *vocab_loss(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 3);
  const at::Tensor &X = cuda_tensor("X", a[0]);
  matrix("X", a[0]);
  const int64_t M = X.size(0), d = X.size(1), V = matrix("W", a[1]).size(0);
  const at::Device dev = X.device();
  const void *px = on("X", X, at::kBFloat16, {M, d}, dev);
  const void *pw = on("W", a[1], at::kBFloat16, {V, d}, dev);
  const int64_t *pt = (const int64_t *)on("target", a[2], at::kLong, {M}, dev);
  const int Mi = size_of("M", M), Vi = size_of("V", V), di = size_of("d", d);
  c10::cuda::CUDAGuard guard(dev);
  const int64_t rows[1] = {M};
  Results t(dev);
  const int ws = t.add_workspace(flash_mca_vocab_loss_workspace_bytes(Mi, Vi, di),
                                 "flash_mca_vocab_loss_workspace_bytes");
  const int loss = t.add(rows, at::kFloat), lse = t.add(rows, at::kFloat);
  check(t.queue([&] {
          return flash_mca_vocab_loss(px, pw, pt, t.ptr<float>(loss), t.ptr<float>(lse), Mi, Vi, di,
                                      t.ptr(ws), (size_t)t[ws].numel(), stream_of(dev));
        }),
        "flash_mca_vocab_loss");
  return pack(t[loss], t[lse]);
  END_HANDLE_TH_ERRORS
}

// (X, W, target, lse, dloss) -> (dX, dW)
PyObject *vocab_loss_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 5);
  const at::Tensor &X = cuda_tensor("X", a[0]);
  matrix("X", a[0]);
  const int64_t M = X.size(0), d = X.size(1), V = matrix("W", a[1]).size(0);
  const at::Device dev = X.device();
  const void *px = on("X", X, at::kBFloat16, {M, d}, dev);
  const void *pw = on("W", a[1], at::kBFloat16, {V, d}, dev);
  const int64_t *pt = (const int64_t *)on("target", a[2], at::kLong, {M}, dev);
  const float *pl = (const float *)on("lse", a[3], at::kFloat, {M}, dev);
  const float *pg = (const float *)on("dloss", a[4], at::kFloat, {M}, dev);
  const int Mi = size_of("M", M), Vi = size_of("V", V), di = size_of("d", d);
  c10::cuda::CUDAGuard guard(dev);
  const int64_t wshape[2] = {V, d};
  Results t(dev);
  const int ws = t.add_workspace(flash_mca_vocab_loss_backward_workspace_bytes(Mi, Vi, di),
                                 "flash_mca_vocab_loss_backward_workspace_bytes");
  const int dX = t.add(X.sizes(), at::kBFloat16), dW = t.add(wshape, at::kBFloat16);
  check(t.queue([&] {
          return flash_mca_vocab_loss_backward(px, pw, pt, pl, pg, t.ptr(dX), t.ptr(dW), Mi, Vi, di,
                                               t.ptr(ws), (size_t)t[ws].numel(), stream_of(dev));
        }),
        "flash_mca_vocab_loss_backward");
  return pack(t[dX], t[dW]);
  END_HANDLE_TH_ERRORS
}

// (FmcaError): the class that a refused call raises
PyObject *set_error(PyObject *, PyObject *type) {
  Py_XINCREF(type);
  Py_XSETREF(g_error, type);
  Py_RETURN_NONE;
}

#define FMCA_FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {
    FMCA_FAST(layer_norm),          FMCA_FAST(layer_norm_backward),
    FMCA_FAST(gau_project_backward), FMCA_FAST(gau_output_backward),
    FMCA_FAST(vocab_loss),          FMCA_FAST(vocab_loss_backward),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding",
                       "Allocating wrappers of the training operators.", -1, kMethods};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__binding(void) {
  return PyModule_Create(&kModule);
}
