// Python binding of the calls on an f8 cache, the normed append, the windowed and the shared-prefix attention
// (include/td.h) as a CPython extension on torch tensors: argument checks, outputs and workspaces made
// when the caller passes none, then the C call.
//
// The other calls are bound through ctypes (api.py). These are bound natively because a token's
// append or a short decode takes the GPU 2 to 7 us, and marshalling twenty arguments and checking
// ten tensors from Python took the host 9 to 13 us a call; here it takes 3 us, most of it the launch.
//
// Shapes and types are checked before devices, so every refusal but the library's own can be met
// without a GPU. Errors are ValueError, TypeError, or the library's TDError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/FunctionRef.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <cmath>
#include <list>
#include <mutex>
#include <optional>
#include <stdexcept>
#include <string>

#include "td.h"

namespace {

PyObject *g_check = nullptr;  // _lib.check(name, status): raises TDError

struct Refused : std::runtime_error {
  PyObject *type;
  Refused(PyObject *t, const char *what) : std::runtime_error(what), type(t) {}
};
struct Raised {};  // a Python error is set

void want(bool ok, PyObject *type, const char *what) {
  if (!ok) throw Refused(type, what);
}

const at::Tensor *tensor_or_null(PyObject *o) {
  if (o == Py_None) return nullptr;
  want(THPVariable_Check(o), PyExc_TypeError, "td calls take torch tensors");
  return &THPVariable_Unpack(o);
}
const at::Tensor &tensor(PyObject *o) {
  const at::Tensor *t = tensor_or_null(o);
  want(t != nullptr, PyExc_TypeError, "td calls take torch tensors");
  return *t;
}
long long integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
int small(PyObject *o) {
  const long long v = integer(o);
  want(v >= -2147483647LL && v <= 2147483647LL, PyExc_ValueError, "size out of range");
  return (int)v;
}
int extent(const at::Tensor &t, int64_t d) {
  const int64_t v = t.size(d);
  want(v <= 2147483647LL, PyExc_ValueError, "size out of range");
  return (int)v;
}
double real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}
bool same_shape(const at::Tensor &a, const at::Tensor &b) { return a.sizes() == b.sizes(); }
bool shaped(const at::Tensor &t, std::initializer_list<int64_t> s) { return t.sizes() == c10::IntArrayRef(s); }

td_dtype code(at::ScalarType t) {
  want(t == at::kFloat || t == at::kBFloat16, PyExc_TypeError, "td supports float32 and bfloat16 tensors");
  return t == at::kFloat ? TD_F32 : TD_BF16;
}

template <typename T>
T *ptr(const at::Tensor &t) {
  return static_cast<T *>(t.data_ptr());
}
template <typename T>
T *ptr(const at::Tensor *t) {
  return t == nullptr ? nullptr : static_cast<T *>(t->data_ptr());
}

// The one CUDA device the given tensors are on; all contiguous (null: not given).
int device_of(std::initializer_list<const at::Tensor *> ts) {
  int dev = -1;
  for (const at::Tensor *t : ts) {
    if (t == nullptr) continue;
    want(t->is_cuda(), PyExc_ValueError, "td kernels take CUDA tensors");
    want(t->is_contiguous(), PyExc_ValueError, "td kernels take contiguous tensors");
    if (dev < 0) dev = t->get_device();
    want(t->get_device() == dev, PyExc_ValueError, "all tensors must be on one CUDA device");
  }
  return dev;
}

// Makes `dev` current for the call (if it is not) and, with a stream of the caller's, that stream
// for the allocations the call makes.
class Place {
 public:
  Place(int dev, PyObject *stream) {
    if (c10::cuda::current_device() != dev) device_.emplace((c10::DeviceIndex)dev);
    if (stream == Py_None) {
      stream_ = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
      return;
    }
    long long raw;
    if (PyObject *attr = PyObject_GetAttrString(stream, "cuda_stream")) {
      raw = PyLong_AsLongLong(attr);
      Py_DECREF(attr);
    } else {
      PyErr_Clear();
      PyObject *num = PyNumber_Long(stream);
      if (num == nullptr) throw Raised{};
      raw = PyLong_AsLongLong(num);
      Py_DECREF(num);
    }
    if (raw == -1 && PyErr_Occurred()) throw Raised{};
    stream_ = reinterpret_cast<cudaStream_t>((intptr_t)raw);
    guard_.emplace(stream_ == nullptr ? c10::cuda::getDefaultCUDAStream((c10::DeviceIndex)dev)
                                      : c10::cuda::getStreamFromExternal(stream_, (c10::DeviceIndex)dev));
  }
  cudaStream_t stream() const { return stream_; }

 private:
  std::optional<c10::cuda::CUDAGuard> device_;
  std::optional<c10::cuda::CUDAStreamGuard> guard_;
  cudaStream_t stream_ = nullptr;
};

PyObject *done(const char *name, td_status st) {
  if (st == TD_OK) Py_RETURN_NONE;
  return PyObject_CallFunction(g_check, "si", name, (int)st);  // raises
}
void checked(const char *name, td_status st) {
  PyObject *r = done(name, st);
  if (r == nullptr) throw Raised{};
  Py_DECREF(r);
}

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }

template <typename F>
PyObject *guarded(F &&f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refused &r) {
    PyErr_SetString(r.type, r.what());
    return nullptr;
  } catch (const Raised &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// A block-scaled cache and its lengths, checked against one another.
struct Cache {
  const at::Tensor &kc, &ks, &vc, &vs, &lens;
  int block, B, Hkv, Smax, D;

  explicit Cache(PyObject *const *a)
      : kc(tensor(a[0])), ks(tensor(a[1])), vc(tensor(a[2])), vs(tensor(a[3])), lens(tensor(a[4])), block(small(a[5])) {
    want(kc.scalar_type() == at::kFloat8_e4m3fn && vc.scalar_type() == at::kFloat8_e4m3fn, PyExc_TypeError,
         "codes must be float8_e4m3fn [B, Hkv, Smax, D]");
    want(kc.dim() == 4 && same_shape(vc, kc), PyExc_ValueError, "codes must be [B, Hkv, Smax, D], K and V alike");
    want(block == 16 || block == 32 || block == 64 || block == 128, PyExc_ValueError, "block must be 16, 32, 64 or 128");
    B = extent(kc, 0), Hkv = extent(kc, 1), Smax = extent(kc, 2), D = extent(kc, 3);
    want(ks.scalar_type() == at::kFloat && vs.scalar_type() == at::kFloat, PyExc_TypeError, "scales must be float32");
    want(shaped(ks, {B, Hkv, (Smax + (int64_t)block - 1) / block}) && same_shape(vs, ks), PyExc_ValueError,
         "scales must be [B, Hkv, ceil(Smax / block)]");
    want(lens.scalar_type() == at::kInt && shaped(lens, {B}), PyExc_TypeError, "seq_lens must be int32 [B]");
  }
};
constexpr int kCache = 6;  // Python arguments of a Cache

const at::Tensor *status_word(PyObject *o) {
  const at::Tensor *t = tensor_or_null(o);
  want(t == nullptr || (t->scalar_type() == at::kInt && t->numel() >= 1), PyExc_TypeError,
       "dev_status must be an int32 tensor");
  return t;
}

int new_rows(const at::Tensor &k, const at::Tensor &v, const Cache &c) {
  want(k.dim() == 4 && same_shape(v, k), PyExc_ValueError, "new rows must be [B, Hkv, T, D], K and V alike");
  const int T = extent(k, 2);
  want(shaped(k, {c.B, c.Hkv, T, c.D}), PyExc_ValueError, "shape mismatch between new rows and caches");
  want(v.scalar_type() == k.scalar_type(), PyExc_TypeError, "new rows must share a dtype");
  code(k.scalar_type());
  return T;
}

// Rotation tables [rows, D/2] with positions [B, T, axes] and axes [D/2] or neither, checked; the axes' count.
int turns(const at::Tensor &cos, const at::Tensor &sin, const at::Tensor *pos, const at::Tensor *axes, int B, int T,
          int Smax, int D) {
  want(cos.scalar_type() == at::kFloat && sin.scalar_type() == at::kFloat && cos.dim() == 2 && cos.size(1) == D / 2 &&
           same_shape(sin, cos),
       PyExc_TypeError, "rope tables must be float32 [rows, D/2], alike");
  if (pos == nullptr) {
    want(axes == nullptr, PyExc_ValueError, "axes need positions");
    want(cos.size(0) >= Smax, PyExc_TypeError, "rope tables must have a row for every cache row");
    return 0;
  }
  want(pos->scalar_type() == at::kInt && pos->dim() == 3 && pos->size(0) == B && pos->size(1) == T, PyExc_TypeError,
       "positions must be int32 [B, T, axes]");
  want(axes == nullptr || (axes->scalar_type() == at::kInt && shaped(*axes, {D / 2})), PyExc_TypeError,
       "axes must be int32 [D/2]");
  return extent(*pos, 2);
}

// append(k_new, v_new, <cache>, advance, dev_status, stream)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t) {
  return guarded([&]() -> PyObject * {
    const at::Tensor &k = tensor(a[0]), &v = tensor(a[1]);
    const Cache c(a + 2);
    a += 2 + kCache;
    const int T = new_rows(k, v, c);
    const bool advance = truth(a[0]);
    const at::Tensor *st = status_word(a[1]);
    const Place place(device_of({&k, &v, &c.kc, &c.ks, &c.vc, &c.vs, &c.lens, st}), a[2]);
    return done("td_kv_append_f8",
                td_kv_append_f8(code(k.scalar_type()), ptr<void>(k), ptr<void>(v), ptr<void>(c.kc), ptr<float>(c.ks),
                                ptr<void>(c.vc), ptr<float>(c.vs), ptr<int32_t>(c.lens), c.B, c.Hkv, T, c.Smax, c.D,
                                c.block, advance, ptr<uint32_t>(st), place.stream()));
  });
}

// rope_append(k_new, v_new, <cache>, cos_t, sin_t, positions, axes, q, q_out, advance, dev_status, stream)
PyObject *rope_append(PyObject *, PyObject *const *a, Py_ssize_t) {
  return guarded([&]() -> PyObject * {
    const at::Tensor &k = tensor(a[0]), &v = tensor(a[1]);
    const Cache c(a + 2);
    a += 2 + kCache;
    const int T = new_rows(k, v, c);
    const at::Tensor &cos = tensor(a[0]), &sin = tensor(a[1]);
    const at::Tensor *pos = tensor_or_null(a[2]), *axes = tensor_or_null(a[3]), *q = tensor_or_null(a[4]);
    const at::Tensor *q_out = tensor_or_null(a[5]);
    const bool advance = truth(a[6]);
    const at::Tensor *st = status_word(a[7]);
    const int rows = extent(cos, 0);
    const int A = turns(cos, sin, pos, axes, c.B, T, c.Smax, c.D);
    int Hq = 0;
    if (q != nullptr) {
      want(q->dim() == 4 && q->size(0) == c.B && q->size(2) == T && q->size(3) == c.D &&
               q->scalar_type() == k.scalar_type(),
           PyExc_ValueError, "q must be [B, Hq, T, D] in the new rows' dtype");
      Hq = extent(*q, 1);
      want(q_out == nullptr || (same_shape(*q_out, *q) && q_out->scalar_type() == q->scalar_type()), PyExc_TypeError,
           "q_out must match q");
    } else {
      want(q_out == nullptr, PyExc_ValueError, "q_out needs q");
    }
    const int dev = device_of({&k, &v, &c.kc, &c.ks, &c.vc, &c.vs, &c.lens, &cos, &sin, pos, axes, q, q_out, st});
    const Place place(dev, a[8]);
    at::Tensor made;
    if (q != nullptr && q_out == nullptr) {
      made = at::empty_like(*q);
      q_out = &made;
    }
    checked("td_rope_kv_append_f8",
            td_rope_kv_append_f8(code(k.scalar_type()), ptr<void>(q), ptr<void>(q_out), Hq, ptr<void>(k), ptr<void>(v),
                                 ptr<float>(cos), ptr<float>(sin), rows, ptr<int32_t>(pos), ptr<int32_t>(axes), A,
                                 ptr<void>(c.kc), ptr<float>(c.ks), ptr<void>(c.vc), ptr<float>(c.vs),
                                 ptr<int32_t>(c.lens), c.B, c.Hkv, T, c.Smax, c.D, c.block, advance, ptr<uint32_t>(st),
                                 place.stream()));
    if (q_out == nullptr) Py_RETURN_NONE;
    if (!made.defined()) return Py_NewRef(a[5]);
    return wrap(made);
  });
}

// norm_append(k_new, v_new, k_cache, v_cache, seq_lens, k_weight, cos_t, sin_t, eps, positions, axes, q, q_weight,
// q_out, advance, dev_status, stream)
PyObject *norm_append(PyObject *, PyObject *const *a, Py_ssize_t) {
  return guarded([&]() -> PyObject * {
    const at::Tensor &k = tensor(a[0]), &v = tensor(a[1]), &kc = tensor(a[2]), &vc = tensor(a[3]), &lens = tensor(a[4]);
    const at::Tensor &kw = tensor(a[5]), &cos = tensor(a[6]), &sin = tensor(a[7]);
    const double eps = real(a[8]);
    const at::Tensor *pos = tensor_or_null(a[9]), *axes = tensor_or_null(a[10]), *q = tensor_or_null(a[11]);
    const at::Tensor *qw = tensor_or_null(a[12]), *q_out = tensor_or_null(a[13]);
    const bool advance = truth(a[14]);
    const at::Tensor *st = status_word(a[15]);
    want(k.dim() == 4 && same_shape(v, k) && kc.dim() == 4 && same_shape(vc, kc), PyExc_ValueError,
         "new rows must be [B, Hkv, T, D] and caches [B, Hkv, Smax, D], K and V alike");
    const int B = extent(k, 0), Hkv = extent(k, 1), T = extent(k, 2), D = extent(k, 3), Smax = extent(kc, 2);
    want(shaped(kc, {B, Hkv, Smax, D}), PyExc_ValueError, "shape mismatch between new rows and caches");
    const at::ScalarType type = k.scalar_type();
    want(v.scalar_type() == type && kc.scalar_type() == type && vc.scalar_type() == type, PyExc_TypeError,
         "new rows and caches must share a dtype");
    const td_dtype dt = code(type);
    want(lens.scalar_type() == at::kInt && shaped(lens, {B}), PyExc_TypeError, "seq_lens must be int32 [B]");
    want(kw.scalar_type() == at::kFloat && shaped(kw, {D}), PyExc_TypeError, "k_weight must be float32 [D]");
    const int A = turns(cos, sin, pos, axes, B, T, Smax, D);
    int Hq = 0;
    if (q != nullptr) {
      want(q->dim() == 4 && q->size(0) == B && q->size(2) == T && q->size(3) == D && q->scalar_type() == type,
           PyExc_ValueError, "q must be [B, Hq, T, D] in the new rows' dtype");
      Hq = extent(*q, 1);
      want(qw != nullptr && qw->scalar_type() == at::kFloat && shaped(*qw, {D}), PyExc_TypeError,
           "q_weight must be float32 [D]");
      want(q_out == nullptr || (same_shape(*q_out, *q) && q_out->scalar_type() == type), PyExc_TypeError,
           "q_out must match q");
    } else {
      want(q_out == nullptr && qw == nullptr, PyExc_ValueError, "q_weight and q_out need q");
    }
    const Place place(device_of({&k, &v, &kc, &vc, &lens, &kw, &cos, &sin, pos, axes, q, qw, q_out, st}), a[16]);
    at::Tensor made;
    if (q != nullptr && q_out == nullptr) {
      made = at::empty_like(*q);
      q_out = &made;
    }
    checked("td_norm_rope_kv_append",
            td_norm_rope_kv_append(dt, ptr<void>(q), ptr<void>(q_out), Hq, ptr<float>(qw), ptr<void>(k), ptr<void>(v),
                                   ptr<float>(kw), (float)eps, ptr<float>(cos), ptr<float>(sin), extent(cos, 0),
                                   ptr<int32_t>(pos), ptr<int32_t>(axes), A, ptr<void>(kc), ptr<void>(vc),
                                   ptr<int32_t>(lens), B, Hkv, T, Smax, D, advance, ptr<uint32_t>(st), place.stream()));
    if (q_out == nullptr) Py_RETURN_NONE;
    if (!made.defined()) return Py_NewRef(a[13]);
    return wrap(made);
  });
}

// read(<cache>, rows, start, dtype, k_out, v_out, dev_status, stream)
PyObject *read(PyObject *, PyObject *const *a, Py_ssize_t) {
  return guarded([&]() -> PyObject * {
    const Cache c(a);
    a += kCache;
    const at::Tensor *start = tensor_or_null(a[1]), *k = tensor_or_null(a[3]), *v = tensor_or_null(a[4]);
    const at::Tensor *st = status_word(a[5]);
    want(THPDtype_Check(a[2]), PyExc_TypeError, "dtype must be a torch dtype");
    want((k == nullptr) == (v == nullptr), PyExc_ValueError, "give both outputs or neither");
    want(start == nullptr || (start->scalar_type() == at::kInt && shaped(*start, {c.B})), PyExc_TypeError,
         "start must be int32 [B]");
    const at::ScalarType type =
        k != nullptr ? k->scalar_type() : reinterpret_cast<THPDtype *>(a[2])->scalar_type;
    const td_dtype dt = code(type);
    int N = a[0] == Py_None ? c.Smax : small(a[0]);
    if (k != nullptr) {
      want(k->dim() == 4 && same_shape(*v, *k) && v->scalar_type() == type, PyExc_ValueError,
           "outputs must be [B, Hkv, rows, D], alike");
      want(a[0] == Py_None || k->size(2) == N, PyExc_ValueError, "rows and the outputs disagree");
      N = extent(*k, 2);
      want(shaped(*k, {c.B, c.Hkv, N, c.D}), PyExc_ValueError, "outputs must be [B, Hkv, rows, D], alike");
    }
    want(N > 0, PyExc_ValueError, "rows must be positive");
    const Place place(device_of({&c.kc, &c.ks, &c.vc, &c.vs, &c.lens, start, k, v, st}), a[6]);
    at::Tensor made[2];
    if (k == nullptr) {
      for (at::Tensor &m : made) m = at::zeros({c.B, c.Hkv, N, c.D}, c.kc.options().dtype(type));
      k = &made[0], v = &made[1];
    }
    checked("td_kv_read_f8",
            td_kv_read_f8(dt, ptr<void>(c.kc), ptr<float>(c.ks), ptr<void>(c.vc), ptr<float>(c.vs), ptr<int32_t>(c.lens),
                          ptr<int32_t>(start), c.B, c.Hkv, N, c.Smax, c.D, c.block, ptr<void>(k), ptr<void>(v),
                          ptr<uint32_t>(st), place.stream()));
    return made[0].defined() ? Py_BuildValue("(NN)", wrap(made[0]), wrap(made[1])) : PyTuple_Pack(2, a[3], a[4]);
  });
}

// Workspaces kept for calls that bring none: one per (device, stream, call shape), zero-filled when
// made, most recently used first, kMost of them and kMostBytes in all at most (a caller's split can ask
// for gigabytes; the one in use stays whatever its size). One that is dropped goes back to the
// allocator of the stream whose calls alone used it. Never destroyed at exit, which they may outlive.
using Key = std::array<long long, 13>;  // which call, device, stream, its shape arguments
enum : long long { kWsF8, kWsWindow, kWsPrefix };
at::Tensor kept_workspace(const Key &key, const at::Tensor &like, c10::function_ref<size_t()> bytes_of) {
  static std::mutex mu;
  static auto *kept = new std::list<std::pair<Key, at::Tensor>>();
  constexpr size_t kMost = 32, kMostBytes = size_t(256) << 20;
  want(c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None, PyExc_ValueError,
       "pass a workspace of its own to a call that is captured in a graph");
  {
    std::lock_guard<std::mutex> lock(mu);
    for (auto it = kept->begin(); it != kept->end(); ++it)
      if (it->first == key) {
        if (it != kept->begin()) kept->splice(kept->begin(), *kept, it);
        return it->second;
      }
  }
  const size_t need = bytes_of();
  at::Tensor ws = at::zeros({(int64_t)(need < 256 ? 256 : need)}, like.options().dtype(at::kByte));
  std::lock_guard<std::mutex> lock(mu);
  kept->emplace_front(key, ws);
  size_t bytes = 0;
  for (const auto &w : *kept) bytes += (size_t)w.second.numel();
  while (kept->size() > 1 && (kept->size() > kMost || bytes > kMostBytes)) {
    bytes -= (size_t)kept->back().second.numel();
    kept->pop_back();
  }
  return ws;
}

long long stream_key(const Place &place) { return (long long)reinterpret_cast<intptr_t>(place.stream()); }

// The results of an attention call: what the caller passed, or tensors made here.
struct Results {
  const at::Tensor *out, *lse;
  at::Tensor made_out, made_lse;
  PyObject *given_out, *given_lse;
  bool want_lse;

  Results(PyObject *o, PyObject *l, PyObject *return_lse, const at::Tensor &q)
      : out(tensor_or_null(o)), lse(tensor_or_null(l)), given_out(o), given_lse(l) {
    want(out == nullptr || (same_shape(*out, q) && out->scalar_type() == q.scalar_type()), PyExc_TypeError,
         "out must match q");
    want(lse == nullptr || (lse->scalar_type() == at::kFloat && lse->sizes() == rows(q)), PyExc_TypeError,
         "lse must be float32 in q's shape without D");
    want_lse = lse != nullptr || truth(return_lse);
  }
  static c10::IntArrayRef rows(const at::Tensor &q) { return q.sizes().slice(0, q.dim() - 1); }
  void make(const at::Tensor &q) {
    if (out == nullptr) {
      made_out = at::empty_like(q);
      out = &made_out;
    }
    if (want_lse && lse == nullptr) {
      made_lse = at::empty(rows(q), q.options().dtype(at::kFloat));
      lse = &made_lse;
    }
  }
  PyObject *give() const {
    PyObject *o = made_out.defined() ? wrap(made_out) : Py_NewRef(given_out);
    if (!want_lse) return o;
    return Py_BuildValue("(NN)", o, made_lse.defined() ? wrap(made_lse) : Py_NewRef(given_lse));
  }
};

double scale_of(PyObject *o, int D) { return o == Py_None ? 1.0 / std::sqrt((double)D) : real(o); }

// attn(q, <cache>, scale, split, out, lse, workspace, dev_status, stream, return_lse): decode for a
// 3-D q, else verify
PyObject *attn(PyObject *, PyObject *const *a, Py_ssize_t) {
  return guarded([&]() -> PyObject * {
    const at::Tensor &q = tensor(a[0]);
    const Cache c(a + 1);
    a += 1 + kCache;
    const bool decode = q.dim() == 3;
    const char *name = decode ? "td_decode_attn_f8" : "td_verify_attn_f8";
    const double scale = scale_of(a[0], c.D);
    const int split = small(a[1]);
    want(q.scalar_type() == at::kBFloat16, PyExc_TypeError, "q must be bfloat16");
    want(q.size(0) == c.B && q.size(-1) == c.D, PyExc_ValueError, "q and cache shapes disagree");
    Results r(a[2], a[3], a[7], q);
    const at::Tensor *ws = tensor_or_null(a[4]);
    const at::Tensor *st = status_word(a[5]);
    want(ws == nullptr || ws->scalar_type() == at::kByte, PyExc_TypeError, "workspace must be a uint8 tensor");
    const int Hq = extent(q, 1), T = decode ? 1 : extent(q, 2);
    const int dev = device_of({&q, &c.kc, &c.ks, &c.vc, &c.vs, &c.lens, r.out, r.lse, ws, st});
    const Place place(dev, a[6]);
    r.make(q);
    at::Tensor kept;
    if (ws == nullptr) {
      kept = kept_workspace({kWsF8, dev, stream_key(place), c.B, Hq, c.Hkv, c.Smax, c.D, T, split}, q,
                            [&] { return td_f8_workspace_bytes(c.B, Hq, c.Hkv, c.Smax, c.D, T, split); });
      ws = &kept;
    }
    checked(name, td_verify_attn_f8(ptr<void>(q), ptr<void>(c.kc), ptr<float>(c.ks), ptr<void>(c.vc), ptr<float>(c.vs),
                                    ptr<int32_t>(c.lens), c.B, Hq, c.Hkv, T, c.Smax, c.D, c.block, (float)scale, split,
                                    ptr<void>(r.out), ptr<float>(r.lse), ptr<void>(ws), (size_t)ws->numel(),
                                    ptr<uint32_t>(st), place.stream()));
    return r.give();
  });
}

// A cache of rows, its lengths and the queries over it, checked against one another (T is 1 for a 3-D q).
struct Rows {
  const at::Tensor &q, &k, &v, &lens;
  bool decode;
  int B, Hq, Hkv, T, Smax, D;
  td_dtype dt;

  explicit Rows(PyObject *const *a) : q(tensor(a[0])), k(tensor(a[1])), v(tensor(a[2])), lens(tensor(a[3])) {
    want((q.dim() == 3 || q.dim() == 4) && k.dim() == 4 && same_shape(v, k) && q.size(0) == k.size(0) &&
             q.size(-1) == k.size(3),
         PyExc_ValueError, "q and cache shapes disagree");
    want(k.scalar_type() == q.scalar_type() && v.scalar_type() == q.scalar_type(), PyExc_TypeError,
         "q and caches must share a dtype");
    dt = code(q.scalar_type());
    decode = q.dim() == 3;
    B = extent(q, 0), Hq = extent(q, 1), T = decode ? 1 : extent(q, 2), D = extent(q, -1);
    Hkv = extent(k, 1), Smax = extent(k, 2);
    want(lens.scalar_type() == at::kInt && shaped(lens, {B}), PyExc_TypeError, "seq_lens must be int32 [B]");
  }
};

// window_attn(q, k_cache, v_cache, seq_lens, window, sinks, scale, split, out, lse, workspace, dev_status, stream,
// return_lse): decode for a 3-D q, else verify
PyObject *window_attn(PyObject *, PyObject *const *a, Py_ssize_t) {
  return guarded([&]() -> PyObject * {
    const Rows c(a);
    const int window = small(a[4]), sinks = small(a[5]), split = small(a[7]);
    const double scale = scale_of(a[6], c.D);
    Results r(a[8], a[9], a[13], c.q);
    const at::Tensor *ws = tensor_or_null(a[10]), *st = status_word(a[11]);
    want(ws == nullptr || ws->scalar_type() == at::kByte, PyExc_TypeError, "workspace must be a uint8 tensor");
    const int dev = device_of({&c.q, &c.k, &c.v, &c.lens, r.out, r.lse, ws, st});
    const Place place(dev, a[12]);
    r.make(c.q);
    at::Tensor kept;
    if (ws == nullptr) {
      kept = kept_workspace(
          {kWsWindow, dev, stream_key(place), c.B, c.Hq, c.Hkv, c.Smax, c.D, c.T, split, window, sinks,
           c.dt}, c.q,
          [&] { return td_window_workspace_bytes(c.B, c.Hq, c.Hkv, c.Smax, c.D, c.T, window, sinks, split); });
      ws = &kept;
    }
    checked(c.decode ? "td_decode_attn_window" : "td_verify_attn_window",
            td_verify_attn_window(c.dt, ptr<void>(c.q), ptr<void>(c.k), ptr<void>(c.v), ptr<int32_t>(c.lens), c.B, c.Hq,
                                  c.Hkv, c.T, c.Smax, c.D, (float)scale, window, sinks, split, ptr<void>(r.out),
                                  ptr<float>(r.lse), ptr<void>(ws), (size_t)ws->numel(), ptr<uint32_t>(st),
                                  place.stream()));
    return r.give();
  });
}

// window_prefill(q, k_cache, v_cache, seq_lens, window, sinks, scale, out, lse, dev_status, stream, return_lse)
PyObject *window_prefill(PyObject *, PyObject *const *a, Py_ssize_t) {
  return guarded([&]() -> PyObject * {
    const Rows c(a);
    want(c.dt == TD_BF16, PyExc_TypeError, "prefill takes bfloat16 q and caches");
    const int window = small(a[4]), sinks = small(a[5]);
    const double scale = scale_of(a[6], c.D);
    Results r(a[7], a[8], a[11], c.q);
    const at::Tensor *st = status_word(a[9]);
    const Place place(device_of({&c.q, &c.k, &c.v, &c.lens, r.out, r.lse, st}), a[10]);
    r.make(c.q);
    checked("td_prefill_attn_window",
            td_prefill_attn_window(ptr<void>(c.q), ptr<void>(c.k), ptr<void>(c.v), ptr<int32_t>(c.lens), c.B, c.Hq, c.Hkv,
                                   c.T, c.Smax, c.D, (float)scale, window, sinks, ptr<void>(r.out), ptr<float>(r.lse),
                                   ptr<uint32_t>(st), place.stream()));
    return r.give();
  });
}

// prefix_attn(q, k_cache, v_cache, seq_lens, k_prefix, v_prefix, prefix_len, scale, out, lse, workspace, dev_status,
// stream, return_lse): decode for a 3-D q, else verify
PyObject *prefix_attn(PyObject *, PyObject *const *a, Py_ssize_t) {
  return guarded([&]() -> PyObject * {
    const Rows c(a);
    want(c.dt == TD_BF16, PyExc_TypeError, "attention over a prefix takes bfloat16 q and caches");
    const at::Tensor &kp = tensor(a[4]), &vp = tensor(a[5]), &plen = tensor(a[6]);
    want(kp.dim() == 3 && same_shape(vp, kp) && kp.size(0) == c.Hkv && kp.size(2) == c.D, PyExc_ValueError,
         "the prefix must be [Hkv, Pmax, D], K and V alike");
    want(kp.scalar_type() == at::kBFloat16 && vp.scalar_type() == at::kBFloat16, PyExc_TypeError,
         "the prefix must be bfloat16");
    want(plen.scalar_type() == at::kInt && plen.numel() == 1, PyExc_TypeError, "prefix_len must be one int32");
    const int Pmax = extent(kp, 1);
    const double scale = scale_of(a[7], c.D);
    Results r(a[8], a[9], a[13], c.q);
    const at::Tensor *ws = tensor_or_null(a[10]), *st = status_word(a[11]);
    want(ws == nullptr || ws->scalar_type() == at::kByte, PyExc_TypeError, "workspace must be a uint8 tensor");
    const int dev = device_of({&c.q, &c.k, &c.v, &c.lens, &kp, &vp, &plen, r.out, r.lse, ws, st});
    const Place place(dev, a[12]);
    r.make(c.q);
    at::Tensor kept;
    if (ws == nullptr) {
      kept = kept_workspace({kWsPrefix, dev, stream_key(place), c.B, c.Hq, c.Hkv, c.Smax, c.D, c.T, Pmax}, c.q, [&] {
        return td_prefix_workspace_bytes(c.B, c.Hq, c.Hkv, Pmax, c.Smax, c.D, c.T);
      });
      ws = &kept;
    }
    checked(c.decode ? "td_decode_attn_prefix" : "td_verify_attn_prefix",
            td_verify_attn_prefix(ptr<void>(c.q), ptr<void>(kp), ptr<void>(vp), ptr<int32_t>(plen), ptr<void>(c.k),
                                  ptr<void>(c.v), ptr<int32_t>(c.lens), c.B, c.Hq, c.Hkv, c.T, Pmax, c.Smax, c.D,
                                  (float)scale, ptr<void>(r.out), ptr<float>(r.lse), ptr<void>(ws), (size_t)ws->numel(),
                                  ptr<uint32_t>(st), place.stream()));
    return r.give();
  });
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t), int N>
PyObject *counted(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  return F(self, a, n);
}

#define TD_METHOD(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&counted<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {TD_METHOD(append, 2 + kCache + 3), TD_METHOD(rope_append, 2 + kCache + 9), TD_METHOD(norm_append, 17),
                         TD_METHOD(read, kCache + 7), TD_METHOD(attn, 1 + kCache + 8),
                         TD_METHOD(window_attn, 14), TD_METHOD(window_prefill, 12), TD_METHOD(prefix_attn, 14), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_td_torch", "Native binding of some of the calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__td_torch() {
  PyObject *lib = PyImport_ImportModule("decode_attention_split_gb300._lib");
  if (lib == nullptr) return nullptr;
  g_check = PyObject_GetAttrString(lib, "check");
  Py_DECREF(lib);
  return g_check == nullptr ? nullptr : PyModule_Create(&module);
}
