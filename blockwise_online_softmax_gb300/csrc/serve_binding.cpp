// The argument marshalling of the serving and training calls around the
// attention kernels, as a CPython extension (module _serve): checks of the
// tensors, output allocation, and the call of the C ABI in libra.so.  No
// arithmetic.  The Python functions of the same names in binding.py hold the
// documentation and hand their arguments through in order.
//
// Each of these calls is one or two short kernels, made once or more per layer
// of a serving step.  Checked in Python and called through ctypes they took 15
// to 45 us of host time each, which was the time of a small step.
#include <cstdarg>
#include <cstdio>
#include <exception>
#include <optional>
#include <string>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "ra.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* g_on_status = nullptr;  // Python callable: raises for a status

struct Refused : std::exception {
  PyObject* type;
  std::string text;
  Refused(PyObject* t, std::string s) : type(t), text(std::move(s)) {}
  const char* what() const noexcept override { return text.c_str(); }
};
struct PythonError : std::exception {};  // the error is set already

[[noreturn]] __attribute__((format(printf, 2, 3))) void refuse(PyObject* type, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  throw Refused(type, buf);
}

const char* type_name(ScalarType t) {
  switch (t) {
    case ScalarType::Float: return "torch.float32";
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Int: return "torch.int32";
    case ScalarType::Long: return "torch.int64";
    default: return c10::toString(t);
  }
}

std::string shape_of(const Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + (t.dim() == 1 ? ",)" : ")");
}

// ------------------------------------------------------------------ arguments
const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch tensor", name);
  return THPVariable_Unpack(o);
}
const Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

long long integer(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw PythonError();
  return x;
}
int small(PyObject* o, const char* name) {
  const long long x = integer(o);
  if (x < INT32_MIN || x > INT32_MAX) refuse(PyExc_ValueError, "%s=%lld does not fit 32 bits", name, x);
  return static_cast<int>(x);
}
float real(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw PythonError();
  return static_cast<float>(x);
}
int truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw PythonError();
  return x;
}

int device_of(const Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", name);
  return static_cast<int>(t.get_device());
}

void placed(const Tensor& t, const char* name, int dev, ScalarType type) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", name);
  if (t.get_device() != dev)
    refuse(PyExc_ValueError, "%s is on cuda:%d, not on cuda:%d", name, static_cast<int>(t.get_device()), dev);
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, "%s must be %s, got %s", name, type_name(type), type_name(t.scalar_type()));
}

// A dense tensor.
void* dense(const Tensor& t, const char* name, int dev, ScalarType type) {
  placed(t, name, dev, type);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
  return t.data_ptr();
}
// A dense 1-D tensor of n entries.
template <typename T = void>
T* vec(const Tensor& t, const char* name, int64_t n, int dev, ScalarType type) {
  void* p = dense(t, name, dev, type);
  if (t.dim() != 1 || t.size(0) != n)
    refuse(PyExc_ValueError, "%s must have shape (%lld,), got %s", name, static_cast<long long>(n), shape_of(t).c_str());
  return static_cast<T*>(p);
}
int* ints(const Tensor& t, const char* name, int64_t n, int dev) { return vec<int>(t, name, n, dev, ScalarType::Int); }

// A [T, heads, d] tensor whose heads are dense; tokens may lie further apart
// (a view of a packed projection).
struct Rows {
  void* p;
  int64_t stride;
};
Rows rows(const Tensor& t, const char* name, int dev, ScalarType type) {
  placed(t, name, dev, type);
  const int64_t T = t.size(0), heads = t.size(1), d = t.size(2);
  if (T && (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d)))
    refuse(PyExc_ValueError, "%s: the heads of a token must be dense (strides (%lld, %lld, %lld))", name,
           static_cast<long long>(t.stride(0)), static_cast<long long>(t.stride(1)), static_cast<long long>(t.stride(2)));
  return {t.data_ptr(), T > 1 ? t.stride(0) : heads * d};
}

struct Heads {
  int64_t T;
  int heads, kv_heads, d;
  ScalarType type;
};
int to_int(int64_t x, const char* name) {
  if (x > INT32_MAX) refuse(PyExc_ValueError, "%s=%lld does not fit 32 bits", name, static_cast<long long>(x));
  return static_cast<int>(x);
}
Heads qk_shapes(const Tensor& q, const Tensor& k) {
  if (q.dim() != 3 || k.dim() != 3) refuse(PyExc_ValueError, "q: [T, heads, d]; k: [T, kv_heads, d]");
  if (k.size(0) != q.size(0) || k.size(2) != q.size(2) || k.scalar_type() != q.scalar_type())
    refuse(PyExc_ValueError, "q and k must share their tokens, head dim and dtype");
  if (q.scalar_type() != ScalarType::BFloat16 && q.scalar_type() != ScalarType::Float)
    refuse(PyExc_TypeError, "q/k/v must be bfloat16 or float32, got %s", type_name(q.scalar_type()));
  return {q.size(0), to_int(q.size(1), "heads"), to_int(k.size(1), "kv_heads"), to_int(q.size(2), "d"), q.scalar_type()};
}
int type_code(ScalarType t) { return t == ScalarType::BFloat16 ? RA_BF16 : RA_F32; }

struct Weights {
  const void *q = nullptr, *k = nullptr;
  int type = RA_F32;
};
Weights weights(const Tensor* q, const Tensor* k, int d, int dev) {
  Weights w;
  auto one = [&](const Tensor* t, const char* name) -> const void* {
    if (!t) return nullptr;
    if (t->scalar_type() != ScalarType::Float && t->scalar_type() != ScalarType::BFloat16)
      refuse(PyExc_TypeError, "%s must be float32 or bfloat16, got %s", name, type_name(t->scalar_type()));
    w.type = type_code(t->scalar_type());
    return vec(*t, name, d, dev, t->scalar_type());
  };
  w.q = one(q, "q_weight");
  w.k = one(k, "k_weight");
  if (q && k && q->scalar_type() != k->scalar_type())
    refuse(PyExc_TypeError, "q_weight and k_weight must share a dtype");
  return w;
}

struct Phases {
  const void* p = nullptr;
  int rot = 0;
};
Phases phase_table(const Tensor* t, int dev) {
  if (!t) return {};
  return {vec(*t, "phases", t->numel(), dev, ScalarType::Long), to_int(2 * t->numel(), "rot_dim")};
}

struct Table {
  int* p;
  int n_req, width;
};
Table block_table(const Tensor& t, int64_t n_req, int dev) {
  if (t.dim() != 2 || t.size(0) != n_req)
    refuse(PyExc_ValueError, "block_table must be [n_req=%lld, max_pages], got %s", static_cast<long long>(n_req),
           shape_of(t).c_str());
  if (dev < 0) return {nullptr, 0, 0};  // the shape alone
  return {static_cast<int*>(dense(t, "block_table", dev, ScalarType::Int)), to_int(n_req, "n_req"),
          to_int(t.size(1), "max_pages")};
}

struct Cache {
  void* p;
  int pages, page_size;
  int64_t stride;
};
Cache cache(const Tensor& t, const char* name, int kv_heads, int d, int dev) {
  placed(t, name, dev, ScalarType::BFloat16);
  if (t.dim() != 4 || t.size(2) != kv_heads || t.size(3) != d)
    refuse(PyExc_ValueError, "%s must be [n_pages, page_size, %d, %d], got %s", name, kv_heads, d, shape_of(t).c_str());
  const int64_t n = t.size(0), ps = t.size(1), row = static_cast<int64_t>(kv_heads) * d;
  if (n && ((d > 1 && t.stride(3) != 1) || (kv_heads > 1 && t.stride(2) != d) || (ps > 1 && t.stride(1) != row)))
    refuse(PyExc_ValueError, "%s: a page must be dense (strides (%lld, %lld, %lld, %lld))", name,
           static_cast<long long>(t.stride(0)), static_cast<long long>(t.stride(1)),
           static_cast<long long>(t.stride(2)), static_cast<long long>(t.stride(3)));
  return {t.data_ptr(), to_int(n, "n_pages"), to_int(ps, "page_size"), n > 1 ? t.stride(0) : ps * row};
}
void same_pages(const Cache& k, const Cache& v) {
  if (k.pages != v.pages || k.page_size != v.page_size)
    refuse(PyExc_ValueError, "k_cache and v_cache must match in pages and page size");
}

// ------------------------------------------------------------------ outputs
// Device and stream of a call.  Outputs that the caller left out are made with
// that stream current: what work on another stream still holds is not handed
// out, and a result that is dropped goes back in the stream's order.  The
// current stream, which may read them too, is recorded as their user.
struct Place {
  int dev;
  void* stream;
  c10::cuda::CUDAStream current;
  std::optional<c10::cuda::CUDAStream> other;  // the stream, if it is not the current one

  Place(int dev_, PyObject* o)
      : dev(dev_), stream(nullptr), current(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev_))) {
    if (o == Py_None) {
      stream = current.stream();
      return;
    }
    PyObject* h = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : PyNumber_Long(o);
    if (!h) throw PythonError();
    stream = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (!stream && PyErr_Occurred()) throw PythonError();
    const auto st = static_cast<cudaStream_t>(stream);
    if (st == current.stream()) return;
    const auto index = static_cast<c10::DeviceIndex>(dev);
    // (The legacy default stream goes by two names, of which torch knows one.)
    other = st && st != cudaStreamLegacy ? c10::cuda::getStreamFromExternal(st, index)
                                         : c10::cuda::getDefaultCUDAStream(index);
  }
  Tensor make(at::IntArrayRef sizes, ScalarType type) const {
    const c10::Device d(c10::DeviceType::CUDA, static_cast<c10::DeviceIndex>(dev));
    if (!other) return at::detail::empty_cuda(sizes, type, d, std::nullopt);
    c10::cuda::CUDAStreamGuard guard(*other);
    Tensor t = at::detail::empty_cuda(sizes, type, d, std::nullopt);
    if (t.numel()) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), current);
    return t;
  }
};

// An output the caller gave, or a new one.
struct Out {
  Tensor made;
  const Tensor* t;
  PyObject* given;
  Out(PyObject* o, const char* name) : t(maybe(o, name)), given(o == Py_None ? nullptr : o) {}
  const Tensor& get(at::IntArrayRef sizes, ScalarType type, const Place& at) {
    if (!t) {
      made = at.make(sizes, type);
      t = &made;
    }
    return *t;
  }
  PyObject* release() {
    if (given) {
      Py_INCREF(given);
      return given;
    }
    if (!t) Py_RETURN_NONE;
    return THPVariable_Wrap(std::move(made));
  }
};

// The small outputs that the caller did not give, as views of one allocation: an
// allocation each took 0.7 us of host time, most of a small step's call.
class Block {
 public:
  void add(Out& o, at::IntArrayRef sizes, ScalarType type) {
    if (o.t) return;
    Part& p = parts_[count_++];
    p = {&o, {}, sizes.size(), bytes_, type};
    int64_t n = static_cast<int64_t>(c10::elementSize(type));
    for (size_t i = 0; i < sizes.size(); ++i) n *= p.sizes[i] = sizes[i];
    bytes_ += (n + 255) / 256 * 256;
  }
  void make(const Place& at) {
    if (count_ == 0) return;
    const Tensor all = at.make({bytes_}, ScalarType::Byte);
    for (int i = 0; i < count_; ++i) {
      const Part& p = parts_[i];
      Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                          c10::scalarTypeToTypeMeta(p.type));
      t.unsafeGetTensorImpl()->set_storage_offset(p.at / static_cast<int64_t>(c10::elementSize(p.type)));
      t.unsafeGetTensorImpl()->set_sizes_contiguous(at::IntArrayRef(p.sizes, p.dim));
      p.o->made = std::move(t);
      p.o->t = &p.o->made;
    }
  }

 private:
  struct Part {
    Out* o;
    int64_t sizes[3];
    size_t dim;
    int64_t at;
    ScalarType type;
  };
  Part parts_[6];
  int count_ = 0;
  int64_t bytes_ = 0;
};

PyObject* pack(std::initializer_list<Out*> outs) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(outs.size()));
  if (!r) throw PythonError();
  Py_ssize_t i = 0;
  for (Out* o : outs) {
    PyObject* x = o->release();
    if (!x) {
      Py_DECREF(r);
      throw PythonError();
    }
    PyTuple_SET_ITEM(r, i++, x);
  }
  return r;
}

// Runs f(stream) with the tensors' device current and without the GIL; a
// status other than RA_OK raises.
template <typename F>
void call(const Place& at, F f) {
  c10::cuda::OptionalCUDAGuard guard;
  if (c10::cuda::current_device() != at.dev) guard.set_index(static_cast<c10::DeviceIndex>(at.dev));
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f(at.stream);
  Py_END_ALLOW_THREADS;
  if (rc == RA_OK) return;
  PyObject* r = PyObject_CallFunction(g_on_status, "i", rc);
  Py_XDECREF(r);
  if (r) PyErr_Format(PyExc_RuntimeError, "status %d", rc);
  throw PythonError();
}

template <PyObject* (*F)(PyObject* const*)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n, Py_ssize_t want) {
  if (n != want) return PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  try {
    return F(a);
  } catch (const PythonError&) {
    return nullptr;
  } catch (const Refused& e) {
    PyErr_SetString(e.type, e.what());
    return nullptr;
  } catch (...) {  // torch's own, out of memory among them
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

void same_shape(const Tensor& t, const Tensor& like, const char* text) {
  if (t.sizes() != like.sizes()) refuse(PyExc_ValueError, "%s", text);
}

// ------------------------------------------------------------------ the calls
// q, k, phases, q_weight, k_weight, eps, interleaved, mscale, positions, P,
// layout, q_out, k_out, stream
PyObject* norm_rope(PyObject* const* a) {
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
  const Heads h = qk_shapes(q, k);
  Out qo(a[11], "q_out"), ko(a[12], "k_out");
  if (qo.t) same_shape(*qo.t, q, "q_out and k_out must match q and k in shape");
  if (ko.t) same_shape(*ko.t, k, "q_out and k_out must match q and k in shape");
  const int dev = device_of(q, "q");
  const Rows rq = rows(q, "q", dev, h.type), rk = rows(k, "k", dev, h.type);
  const Phases ph = phase_table(maybe(a[2], "phases"), dev);
  const Weights w = weights(maybe(a[3], "q_weight"), maybe(a[4], "k_weight"), h.d, dev);
  const Tensor* pos = maybe(a[8], "positions");
  const int* pp = pos ? ints(*pos, "positions", h.T, dev) : nullptr;
  const float eps = real(a[5]), ms = real(a[7]);
  const int inter = truth(a[6]), P = small(a[9], "P"), layout = small(a[10], "layout");
  const Place at(dev, a[13]);
  void* po = dense(qo.get(q.sizes(), h.type, at), "q_out", dev, h.type);
  void* pk = dense(ko.get(k.sizes(), h.type, at), "k_out", dev, h.type);
  call(at, [&](void* st) {
    return ra_qk_norm_rope(rq.p, rk.p, po, pk, h.T, h.d, h.heads, h.kv_heads, rq.stride, rk.stride, pp, layout, P,
                           ph.rot, inter, ph.p, ms, w.q, w.k, w.type, eps, type_code(h.type), st);
  });
  return pack({&qo, &ko});
}

// q, k, phases, dq_out, dk_out, q_weight, k_weight, eps, interleaved, mscale,
// positions, P, layout, dq, dk, dq_weight, dk_weight, stream
PyObject* norm_rope_backward(PyObject* const* a) {
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
  const Tensor &gq = tensor(a[3], "dq_out"), &gk = tensor(a[4], "dk_out");
  const Heads h = qk_shapes(q, k);
  same_shape(gq, q, "dq_out and dk_out must match q and k in shape");
  same_shape(gk, k, "dq_out and dk_out must match q and k in shape");
  Out dq(a[13], "dq"), dk(a[14], "dk"), dqw(a[15], "dq_weight"), dkw(a[16], "dk_weight");
  if (dq.t) same_shape(*dq.t, q, "dq and dk must match q and k in shape");
  if (dk.t) same_shape(*dk.t, k, "dq and dk must match q and k in shape");
  const Tensor *qw = maybe(a[5], "q_weight"), *kw = maybe(a[6], "k_weight");
  if (!qw && dqw.t) refuse(PyExc_ValueError, "dq_weight without its weight");
  if (!kw && dkw.t) refuse(PyExc_ValueError, "dk_weight without its weight");
  const int dev = device_of(q, "q");
  const Rows rq = rows(q, "q", dev, h.type), rk = rows(k, "k", dev, h.type);
  const Phases ph = phase_table(maybe(a[2], "phases"), dev);
  const Weights w = weights(qw, kw, h.d, dev);
  const Tensor* pos = maybe(a[10], "positions");
  const int* pp = pos ? ints(*pos, "positions", h.T, dev) : nullptr;
  const float eps = real(a[7]), ms = real(a[9]);
  const int inter = truth(a[8]), P = small(a[11], "P"), layout = small(a[12], "layout");
  const auto f32 = ScalarType::Float;
  const auto* pgq = static_cast<const float*>(dense(gq, "dq_out", dev, f32));
  const auto* pgk = static_cast<const float*>(dense(gk, "dk_out", dev, f32));
  const Place at(dev, a[17]);
  const Rows oq = rows(dq.get(q.sizes(), h.type, at), "dq", dev, h.type);
  const Rows ok = rows(dk.get(k.sizes(), h.type, at), "dk", dev, h.type);
  float* wq = qw ? vec<float>(dqw.get({h.d}, f32, at), "dq_weight", h.d, dev, f32) : nullptr;
  float* wk = kw ? vec<float>(dkw.get({h.d}, f32, at), "dk_weight", h.d, dev, f32) : nullptr;
  call(at, [&](void* st) {
    return ra_qk_norm_rope_backward(rq.p, rk.p, pgq, pgk, oq.p, ok.p, wq, wk, h.T, h.d, h.heads, h.kv_heads,
                                    rq.stride, rk.stride, oq.stride, ok.stride, pp, layout, P, ph.rot, inter, ph.p,
                                    ms, w.q, w.k, w.type, eps, type_code(h.type), st);
  });
  return pack({&dq, &dk, &dqw, &dkw});
}

// lengths, new_tokens, block_table, free_pages, free_count, page_size, tokens,
// lengths_out, free_count_out, slots, positions, cu_tokens, status, stream
PyObject* extend(PyObject* const* a) {
  const Tensor &len = tensor(a[0], "lengths"), &nw = tensor(a[1], "new_tokens"), &tab = tensor(a[2], "block_table");
  const Tensor &fp = tensor(a[3], "free_pages"), &fc = tensor(a[4], "free_count");
  const int64_t n = len.numel();
  const long long tokens = integer(a[6]);
  const int ps = small(a[5], "page_size");
  block_table(tab, n, -1);
  const int dev = device_of(len, "lengths");
  const Table tb = block_table(tab, n, dev);
  Out lo(a[7], "lengths_out"), co(a[8], "free_count_out"), sl(a[9], "slots"), po(a[10], "positions"),
      cu(a[11], "cu_tokens"), stt(a[12], "status");
  if (tokens < 0) refuse(PyExc_ValueError, "tokens=%lld is negative", tokens);
  const auto i32 = ScalarType::Int;
  const int* pl = ints(len, "lengths", n, dev);
  const int* pn = ints(nw, "new_tokens", n, dev);
  const int* pf = ints(fp, "free_pages", fp.numel(), dev);
  const int* pc = ints(fc, "free_count", 1, dev);
  const int pool = to_int(fp.numel(), "free_pages");
  Block made;
  made.add(sl, {tokens}, ScalarType::Long);
  made.add(po, {tokens}, i32);
  made.add(cu, {n + 1}, i32);
  made.add(lo, {n}, i32);
  made.add(co, {1}, i32);
  made.add(stt, {3}, i32);
  const Place at(dev, a[13]);
  made.make(at);
  int* plo = ints(*lo.t, "lengths_out", n, dev);
  int* pco = ints(*co.t, "free_count_out", 1, dev);
  auto* psl = reinterpret_cast<long long*>(vec<int64_t>(*sl.t, "slots", tokens, dev, ScalarType::Long));
  int* ppo = ints(*po.t, "positions", tokens, dev);
  int* pcu = ints(*cu.t, "cu_tokens", n + 1, dev);
  int* pst = ints(*stt.t, "status", 3, dev);
  call(at, [&](void* st) {
    return ra_paged_extend(pl, pn, tb.n_req, tb.p, tb.width, pf, pool, pc, ps, tokens, plo, pco, psl, ppo, pcu, pst,
                           st);
  });
  return pack({&sl, &po, &cu, &lo, &co, &stt});
}

// lengths, finished, block_table, free_pages, free_count, page_size,
// lengths_out, free_count_out, stream
PyObject* release(PyObject* const* a) {
  const Tensor &len = tensor(a[0], "lengths"), &fin = tensor(a[1], "finished"), &tab = tensor(a[2], "block_table");
  const Tensor &fp = tensor(a[3], "free_pages"), &fc = tensor(a[4], "free_count");
  const int64_t n = len.numel();
  const int ps = small(a[5], "page_size"), dev = device_of(len, "lengths");
  const Table tb = block_table(tab, n, dev);
  Out lo(a[6], "lengths_out"), co(a[7], "free_count_out");
  const int* pl = ints(len, "lengths", n, dev);
  const int* pn = ints(fin, "finished", n, dev);
  int* pf = ints(fp, "free_pages", fp.numel(), dev);
  const int* pc = ints(fc, "free_count", 1, dev);
  const int pool = to_int(fp.numel(), "free_pages");
  Block made;
  made.add(lo, {n}, ScalarType::Int);
  made.add(co, {1}, ScalarType::Int);
  const Place at(dev, a[8]);
  made.make(at);
  int* plo = ints(*lo.t, "lengths_out", n, dev);
  int* pco = ints(*co.t, "free_count_out", 1, dev);
  call(at, [&](void* st) {
    return ra_paged_release(pl, pn, tb.n_req, tb.p, tb.width, pf, pool, pc, ps, plo, pco, st);
  });
  return pack({&lo, &co});
}

// q, k, v, phases, k_cache, v_cache, slots, positions, q_weight, k_weight, eps,
// interleaved, mscale, q_out, stream
PyObject* append(PyObject* const* a) {
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  const Tensor &kc = tensor(a[4], "k_cache"), &vc = tensor(a[5], "v_cache");
  const Tensor &sl = tensor(a[6], "slots"), &pos = tensor(a[7], "positions");
  const Heads h = qk_shapes(q, k);
  if (v.sizes() != k.sizes() || v.scalar_type() != q.scalar_type())
    refuse(PyExc_ValueError, "v must match k in shape and dtype");
  Out qo(a[13], "q_out");
  if (qo.t) same_shape(*qo.t, q, "q_out must match q in shape");
  const int dev = device_of(q, "q");
  const Rows rq = rows(q, "q", dev, h.type), rk = rows(k, "k", dev, h.type), rv = rows(v, "v", dev, h.type);
  const Cache ck = cache(kc, "k_cache", h.kv_heads, h.d, dev), cv = cache(vc, "v_cache", h.kv_heads, h.d, dev);
  same_pages(ck, cv);
  const Phases ph = phase_table(maybe(a[3], "phases"), dev);
  const Weights w = weights(maybe(a[8], "q_weight"), maybe(a[9], "k_weight"), h.d, dev);
  const auto* psl = reinterpret_cast<const long long*>(vec<int64_t>(sl, "slots", h.T, dev, ScalarType::Long));
  const int* pp = ints(pos, "positions", h.T, dev);
  const float eps = real(a[10]), ms = real(a[12]);
  const int inter = truth(a[11]);
  const Place at(dev, a[14]);
  void* po = dense(qo.get(q.sizes(), h.type, at), "q_out", dev, h.type);
  call(at, [&](void* st) {
    return ra_paged_append(rq.p, rk.p, rv.p, po, ck.p, cv.p, h.T, h.d, h.heads, h.kv_heads, rq.stride, rk.stride,
                           rv.stride, ck.pages, ck.page_size, ck.stride, cv.stride, psl, pp, ph.rot, inter, ph.p, ms,
                           w.q, w.k, w.type, eps, type_code(h.type), st);
  });
  return qo.release();
}

// q, k_cache, v_cache, block_table, lengths, cu_q, n_q, window, out, lse, stream
PyObject* decode(PyObject* const* a) {
  const Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache");
  const Tensor &tab = tensor(a[3], "block_table"), &len = tensor(a[4], "lengths");
  const Tensor* cu = maybe(a[5], "cu_q");
  const int expect = small(a[6], "n_q");
  const long long window = integer(a[7]);
  Out out(a[8], "out"), lse(a[9], "lse");
  if (q.dim() != 3) refuse(PyExc_ValueError, "q: [T, heads, d]");
  if (kc.dim() != 4) refuse(PyExc_ValueError, "k_cache: [n_pages, page_size, kv_heads, d]");
  const int64_t n = len.numel(), T = q.size(0);
  const int heads = to_int(q.size(1), "heads"), d = to_int(q.size(2), "d"), kv_heads = to_int(kc.size(2), "kv_heads");
  if (!cu && (n ? T % n != 0 : T != 0))
    refuse(PyExc_ValueError, "T=%lld rows are not a multiple of %lld requests (and cu_q is None)",
           static_cast<long long>(T), static_cast<long long>(n));
  if (!cu && expect && expect * n != T)
    refuse(PyExc_ValueError, "n_q=%d rows for each of %lld requests are not the %lld of q (and cu_q is None)", expect,
           static_cast<long long>(n), static_cast<long long>(T));
  if (out.t) {
    if (out.t->sizes() != q.sizes())
      refuse(PyExc_ValueError, "out must have shape %s, got %s", shape_of(q).c_str(), shape_of(*out.t).c_str());
    if (out.t->scalar_type() != ScalarType::Float && out.t->scalar_type() != ScalarType::BFloat16)
      refuse(PyExc_TypeError, "out must be float32 or bfloat16, got %s", type_name(out.t->scalar_type()));
  }
  if (lse.t && (lse.t->dim() != 2 || lse.t->size(0) != T || lse.t->size(1) != heads))
    refuse(PyExc_ValueError, "lse must have shape (%lld, %d), got %s", static_cast<long long>(T), heads,
           shape_of(*lse.t).c_str());
  const int dev = device_of(q, "q");
  const void* pq = dense(q, "q", dev, ScalarType::BFloat16);
  const Cache ck = cache(kc, "k_cache", kv_heads, d, dev), cv = cache(vc, "v_cache", kv_heads, d, dev);
  same_pages(ck, cv);
  const Table tb = block_table(tab, n, dev);
  const int* pc = cu ? ints(*cu, "cu_q", n + 1, dev) : nullptr;
  const int* pl = ints(len, "lengths", n, dev);
  Block made;
  made.add(out, q.sizes(), ScalarType::Float);
  made.add(lse, {T, heads}, ScalarType::Float);
  const Place at(dev, a[10]);
  made.make(at);
  const Tensor& to = *out.t;
  void* po = dense(to, "out", dev, to.scalar_type());
  auto* ps = static_cast<float*>(dense(*lse.t, "lse", dev, ScalarType::Float));
  const int n_q = cu ? expect : !n ? 0 : to_int(T / n, "rows per request"), code = type_code(to.scalar_type());
  call(at, [&](void* st) {
    return ra_paged_decode(pq, ck.p, cv.p, po, ps, T, tb.n_req, n_q, pc, tb.p, tb.width, pl, ck.pages, ck.page_size,
                           ck.stride, cv.stride, window, d, heads, kv_heads, RA_BF16, code, st);
  });
  return pack({&out, &lse});
}

PyObject* on_status(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(g_on_status, f);
  Py_RETURN_NONE;
}

#define RA_ENTRY(name, n)                                                              \
  PyObject* name##_entry(PyObject* m, PyObject* const* a, Py_ssize_t got) {             \
    return entry<name>(m, a, got, n);                                                  \
  }
RA_ENTRY(norm_rope, 14)
RA_ENTRY(norm_rope_backward, 18)
RA_ENTRY(extend, 14)
RA_ENTRY(release, 9)
RA_ENTRY(append, 15)
RA_ENTRY(decode, 11)
#undef RA_ENTRY

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f));
}

PyMethodDef g_methods[] = {
    {"on_status", on_status, METH_O, "Set the function that raises for a status of the library."},
    {"qk_norm_rope", fast(norm_rope_entry), METH_FASTCALL, nullptr},
    {"qk_norm_rope_backward", fast(norm_rope_backward_entry), METH_FASTCALL, nullptr},
    {"paged_extend", fast(extend_entry), METH_FASTCALL, nullptr},
    {"paged_release", fast(release_entry), METH_FASTCALL, nullptr},
    {"paged_append", fast(append_entry), METH_FASTCALL, nullptr},
    {"paged_decode", fast(decode_entry), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_serve", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve(void) { return PyModule_Create(&g_module); }
