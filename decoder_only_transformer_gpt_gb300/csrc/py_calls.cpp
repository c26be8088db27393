// The module _calls: the calls of binding.py whose kernels take a few microseconds. Argument checks and marshalling in C++ on
// torch's own tensors, then the C entry (include/gpt_kernels.h). The same checks in Python and the call through ctypes take
// 5 us of the host's time (nine tensors and a dozen numbers: 7.7 us with the launch), more than most of these kernels run.
//
// Every function takes its arguments by position, in the order of the function of the same name in binding.py, raises
// ValueError for tensors and numbers that the kernels cannot take, and returns the C entry's status.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "../../include/gpt.h"
#include "../../include/gpt_kernels.h"

#include <initializer_list>
#include <string>

namespace {

using at::ScalarType;

struct Refused {};                                   // a Python exception is set

std::string text_of(PyObject* o) {
  PyObject* s = o ? PyObject_Str(o) : nullptr;
  const char* c = s ? PyUnicode_AsUTF8(s) : nullptr;
  std::string r = c ? c : "?";
  Py_XDECREF(s);
  Py_XDECREF(o);
  if (!c) PyErr_Clear();
  return r;
}

std::string shape_text(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + (shape.size() == 1 ? ",)" : ")");
}

const char* type_text(ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    default: return "torch.uint8";
  }
}

[[noreturn]] void refuse(const std::string& why) {
  PyErr_SetString(PyExc_ValueError, why.c_str());
  throw Refused();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_SetString(PyExc_TypeError, (std::string(name) + ": needs a tensor").c_str());
    throw Refused();
  }
  return THPVariable_Unpack(o);
}

int64_t number(PyObject* o, const char* name) {      // an int32
  const long long n = PyLong_AsLongLong(o);
  if (n == -1 && PyErr_Occurred()) {
    if (!PyErr_ExceptionMatches(PyExc_OverflowError)) throw Refused();
    PyErr_Clear();
    Py_INCREF(o);
    refuse(std::string(name) + ": " + text_of(o) + ", needs an int32");
  }
  if (n < -2147483648LL || n > 2147483647LL) refuse(std::string(name) + ": " + std::to_string(n) + ", needs an int32");
  return n;
}

int32_t flag(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw Refused();
  return r;
}

// The current device, and the checks of the tensors of one call.
struct Device {
  int dev = -1;                                      // asked when the first tensor on a GPU comes

  bool holds(const at::Tensor& t) {
    if (!t.is_cuda()) return false;
    if (dev < 0) dev = c10::cuda::current_device();
    return t.get_device() == dev;
  }

  [[noreturn]] static void refuse_tensor(PyObject* o, const char* name, const at::Tensor& t, ScalarType type, at::IntArrayRef shape,
                                         bool layout) {
    const std::string n = std::string(name) + ": ";
    if (t.scalar_type() != type) refuse(n + text_of(PyObject_GetAttrString(o, "dtype")) + ", needs " + type_text(type));
    if (t.sizes() != shape) refuse(n + "shape " + shape_text(t.sizes()) + ", needs " + shape_text(shape));
    if (layout && !t.is_contiguous()) refuse(n + "not contiguous");
    refuse(n + "on " + text_of(PyObject_GetAttrString(o, "device")) + ", needs the current CUDA device");
  }

  // The address of a tensor whose type, shape, layout and device the kernels can take.
  void* take(PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape) {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous() || !holds(t)) refuse_tensor(o, name, t, type, shape, true);
    return t.data_ptr();
  }
  template <typename T>
  T* take_as(PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape) {
    return static_cast<T*>(take(o, name, type, shape));
  }
  // The same of one that may be None.
  template <typename T>
  T* maybe(PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape) {
    return o == Py_None ? nullptr : static_cast<T*>(take(o, name, type, shape));
  }

  void* stream(PyObject* o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    PyObject* on = PyObject_GetAttrString(o, "device_index");
    if (on) {
      const long of = PyLong_AsLong(on);
      Py_DECREF(on);
      if (of != dev)
        refuse("stream: of device " + std::to_string(of) + ", needs one of the current device " + std::to_string(dev));
    } else {
      PyErr_Clear();
    }
    PyObject* s = PyObject_GetAttrString(o, "cuda_stream");
    if (!s) throw Refused();
    void* p = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    if (!p && PyErr_Occurred()) throw Refused();
    return p;
  }
};

void dims(const at::Tensor& t, const char* name, int64_t n, const char* needs) {
  if (t.dim() != n) refuse(std::string(name) + ": shape " + shape_text(t.sizes()) + ", needs " + needs);
}

struct Turns {
  const uint64_t* p = nullptr;
  int32_t rot = 0;
  Turns(Device& d, PyObject* o) {
    if (o == Py_None) return;
    const at::Tensor& t = tensor(o, "turns");
    dims(t, "turns", 1, "[rot / 2]");
    p = d.take_as<uint64_t>(o, "turns", at::kLong, t.sizes());
    rot = static_cast<int32_t>(2 * t.size(0));
  }
};

// A paged cache: pool [pages, 2, Hkv, page, D / per] and the table [B, max_pages].
struct Cache {
  int32_t pages, Hkv, page, D, B, max_pages;
  void* pool;
  int32_t* table;
  Cache(Device& d, PyObject* o, const char* name, const char* needs, ScalarType type, int per, PyObject* tab) {
    const at::Tensor &t = tensor(o, name), &u = tensor(tab, "table");
    if (t.dim() != 5 || t.size(1) != 2) refuse(std::string(name) + ": shape " + shape_text(t.sizes()) + ", needs " + needs);
    dims(u, "table", 2, "[B, max_pages]");
    for (int64_t n : {t.size(0), t.size(2), t.size(3), per * t.size(4), u.size(0), u.size(1)})
      if (n > 2147483647LL) refuse(std::string(name) + ": shape " + shape_text(t.sizes()) + ", table: shape " + shape_text(u.sizes()));
    pages = static_cast<int32_t>(t.size(0));
    Hkv = static_cast<int32_t>(t.size(2));
    page = static_cast<int32_t>(t.size(3));
    D = static_cast<int32_t>(per * t.size(4));
    B = static_cast<int32_t>(u.size(0));
    max_pages = static_cast<int32_t>(u.size(1));
    pool = d.take(o, name, type, t.sizes());
    table = d.take_as<int32_t>(tab, "table", at::kInt, u.sizes());
  }
};

struct Cache4 : Cache {
  void* ranges;
  Cache4(Device& d, PyObject* codes, PyObject* rng, PyObject* tab)
      : Cache(d, codes, "codes", "[pages, 2, Hkv, page, D / 2]", at::kByte, 2, tab) {
    ranges = d.take(rng, "ranges", at::kBFloat16, {pages, 2, Hkv, page, 2});
  }
};

// Tokens that go into a paged cache: qkv [B, T, (H + 2 Hkv) D], out and the numbers of each sequence.
struct Rows {
  int32_t T;
  void *qkv, *out;
  int32_t *start, *count, *pos;
  Rows(Device& d, const Cache& c, int64_t H, PyObject* q, PyObject* o, PyObject* st, PyObject* ct, PyObject* ps) {
    const at::Tensor& t = tensor(q, "qkv");
    const int64_t n = t.dim() == 3 ? t.size(1) : 0;
    if (n > 2147483647LL) refuse("qkv: shape " + shape_text(t.sizes()));
    const int64_t shape[3] = {c.B, n, (H + 2LL * c.Hkv) * c.D};
    T = static_cast<int32_t>(n);
    qkv = d.take(q, "qkv", at::kBFloat16, shape);
    out = d.maybe<void>(o, "out", at::kBFloat16, shape);
    start = d.maybe<int32_t>(st, "start", at::kInt, {c.B});
    count = d.maybe<int32_t>(ct, "count", at::kInt, {c.B});
    pos = d.maybe<int32_t>(ps, "pos", at::kInt, {c.B});
  }
};

template <typename F>
PyObject* status_of(F&& f) {
  int rc = 0;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

PyObject* rotary(PyObject* const* a) {               // qkv, out, H, Hkv, turns, pos, interleaved, inverse, stream
  Device d;
  const int64_t H = number(a[2], "H"), Hkv = number(a[3], "Hkv");
  const at::Tensor& q = tensor(a[0], "qkv");
  const int64_t heads = H + 2 * Hkv;
  if (q.dim() != 3 || H < 1 || Hkv < 1 || q.size(2) % heads)
    refuse("qkv: shape " + shape_text(q.sizes()) + ", needs [B, T, (H + 2 Hkv) D] for H = " + std::to_string(H) + ", Hkv = " +
           std::to_string(Hkv));
  const int64_t B = q.size(0), T = q.size(1), D = q.size(2) / heads;
  if (B > 2147483647LL || T > 2147483647LL || q.size(2) > 2147483647LL) refuse("qkv: shape " + shape_text(q.sizes()));
  const Turns t(d, a[4]);
  const void* x = d.take(a[0], "qkv", at::kBFloat16, q.sizes());
  void* out = d.take(a[1], "out", at::kBFloat16, q.sizes());
  const int32_t* pos = d.maybe<int32_t>(a[5], "pos", at::kInt, {B});
  const int32_t inter = flag(a[6]), inverse = flag(a[7]);
  void* s = d.stream(a[8]);
  return status_of([&] {
    return gptk_rotary(x, out, pos, t.p, static_cast<int32_t>(B), static_cast<int32_t>(T), static_cast<int32_t>(H),
                       static_cast<int32_t>(Hkv), static_cast<int32_t>(D), t.rot, inter, inverse, s);
  });
}

PyObject* paged_append(PyObject* const* a) {         // qkv, pool, table, H, turns, start, count, pos, weight, out, interleaved, stream
  Device d;
  const int32_t H = static_cast<int32_t>(number(a[3], "H"));
  const Cache c(d, a[1], "pool", "[pages, 2, Hkv, page, D]", at::kBFloat16, 1, a[2]);
  float* weight = d.maybe<float>(a[8], "weight", at::kFloat, {c.pages, c.Hkv, c.page});
  const Rows r(d, c, H, a[0], a[9], a[5], a[6], a[7]);
  const Turns t(d, a[4]);
  const int32_t inter = flag(a[10]);
  void* s = d.stream(a[11]);
  return status_of([&] {
    return gptk_paged_append(r.qkv, r.out, c.pool, weight, c.table, r.start, r.count, r.pos, t.p, c.B, r.T, H, c.Hkv, c.D, t.rot,
                             inter, c.pages, c.page, c.max_pages, s);
  });
}

PyObject* paged_append4(PyObject* const* a) {        // qkv, codes, ranges, table, H, turns, start, count, pos, out, interleaved, stream
  Device d;
  const int32_t H = static_cast<int32_t>(number(a[4], "H"));
  const Cache4 c(d, a[1], a[2], a[3]);
  const Rows r(d, c, H, a[0], a[9], a[6], a[7], a[8]);
  const Turns t(d, a[5]);
  const int32_t inter = flag(a[10]);
  void* s = d.stream(a[11]);
  return status_of([&] {
    return gptk_paged_append4(r.qkv, r.out, c.pool, c.ranges, c.table, r.start, r.count, r.pos, t.p, c.B, r.T, H, c.Hkv, c.D, t.rot,
                              inter, c.pages, c.page, c.max_pages, s);
  });
}

PyObject* paged_load4(PyObject* const* a) {          // codes, ranges, table, rows, start, count, stream
  Device d;
  const Cache4 c(d, a[0], a[1], a[2]);
  const at::Tensor& t = tensor(a[3], "rows");
  const int64_t T = t.dim() == 3 ? t.size(1) : 0;
  if (T > 2147483647LL) refuse("rows: shape " + shape_text(t.sizes()));
  const int32_t* start = d.maybe<int32_t>(a[4], "start", at::kInt, {c.B});
  const int32_t* count = d.maybe<int32_t>(a[5], "count", at::kInt, {c.B});
  void* rows = d.take(a[3], "rows", at::kBFloat16, {c.B, T, 2LL * c.Hkv * c.D});
  void* s = d.stream(a[6]);
  return status_of([&] {
    return gptk_paged_load4(c.pool, c.ranges, c.table, start, count, rows, c.B, static_cast<int32_t>(T), c.Hkv, c.D, c.pages, c.page,
                            c.max_pages, s);
  });
}

PyObject* paged_attention4(PyObject* const* a) {     // qkv, codes, ranges, table, lens, y, H, lse2, window, sinks, added, stream
  Device d;
  const int32_t H = static_cast<int32_t>(number(a[6], "H")), window = static_cast<int32_t>(number(a[8], "window"));
  const int32_t sinks = static_cast<int32_t>(number(a[9], "sinks")), added = static_cast<int32_t>(number(a[10], "added"));
  const Cache4 c(d, a[1], a[2], a[3]);
  const void* qkv = d.take(a[0], "qkv", at::kBFloat16, {c.B, (H + 2LL * c.Hkv) * c.D});
  const int32_t* lens = d.take_as<int32_t>(a[4], "lens", at::kInt, {c.B});
  void* y = d.take(a[5], "y", at::kBFloat16, {c.B, static_cast<int64_t>(H) * c.D});
  float* lse2 = d.maybe<float>(a[7], "lse2", at::kFloat, {c.B, H});
  void* s = d.stream(a[11]);
  return status_of([&] {
    return gptk_paged_attention4(qkv, c.pool, c.ranges, c.table, lens, y, lse2, c.B, H, c.Hkv, c.D, c.pages, c.page, c.max_pages,
                                 window, sinks, added, s);
  });
}

// Logits [M, V], or their gradient: rows of contiguous values, one row from the next ld apart.
struct Logits {
  int64_t M, V, ld;
  ScalarType type;
  void* p;
  Logits(PyObject* o) {
    const at::Tensor& t = tensor(o, "logits");
    type = t.scalar_type();
    if (t.dim() != 2 || (type != at::kFloat && type != at::kBFloat16))
      refuse("logits: " + text_of(PyObject_GetAttrString(o, "dtype")) + " of shape " + shape_text(t.sizes()) +
             ", needs float32 or bfloat16 [M, V]");
    M = t.size(0);
    V = t.size(1);
    if (M > 2147483647LL || V > 2147483647LL) refuse("logits: shape " + shape_text(t.sizes()));
  }
  int64_t rows(Device& d, PyObject* o, const char* name) {
    const at::Tensor& t = tensor(o, name);
    const int64_t shape[2] = {M, V};
    if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape) || !d.holds(t))
      Device::refuse_tensor(o, name, t, type, shape, false);
    if ((t.stride(1) != 1 && V > 1) || (t.stride(0) < V && M > 1))
      refuse(std::string(name) + ": strides " + shape_text(t.strides()) + ", needs rows of contiguous values");
    p = t.data_ptr();
    return t.stride(0) > V ? t.stride(0) : V;
  }
};

bool given(PyObject* o) { return o != Py_None; }

PyObject* logprobs(PyObject* const* a) {             // logits, targets, logp, entropy, stats, top_ids, top_logp, stream
  Device d;
  Logits z(a[0]);
  const int64_t ld = z.rows(d, a[0], "logits");
  int64_t K = 0;
  if (a[5] != Py_None) {
    const at::Tensor& t = tensor(a[5], "top_ids");
    K = t.dim() == 2 ? t.size(1) : 0;
  }
  int32_t* ids = d.maybe<int32_t>(a[5], "top_ids", at::kInt, {z.M, K});
  const int32_t* targets = d.maybe<int32_t>(a[1], "targets", at::kInt, {z.M});
  float* logp = d.maybe<float>(a[2], "logp", at::kFloat, {z.M});
  float* entropy = d.maybe<float>(a[3], "entropy", at::kFloat, {z.M});
  float* stats = d.maybe<float>(a[4], "stats", at::kFloat, {z.M, 2});
  float* top = d.maybe<float>(a[6], "top_logp", at::kFloat, {z.M, K});
  void* s = d.stream(a[7]);
  if (z.M == 0) {                                    // no rows: nothing to do, where some would be taken (no tensor has an address)
    const bool pairs = given(a[1]) == given(a[2]) && given(a[5]) == given(a[6]);
    const bool some = given(a[2]) || given(a[3]) || given(a[4]) || given(a[5]);
    return PyLong_FromLong(z.V >= 1 && K <= 32 && K <= z.V && pairs && some ? GPT_OK : GPT_EINVAL);
  }
  return status_of([&] {
    return gptk_logprobs(z.p, targets, logp, entropy, stats, ids, top, static_cast<int32_t>(z.M), static_cast<int32_t>(z.V), ld,
                         K > 2147483647LL ? 2147483647 : static_cast<int32_t>(K), z.type == at::kBFloat16, s);
  });
}

PyObject* logprobs_bwd(PyObject* const* a) {         // logits, targets, stats, dlogp, dlogits, entropy, dentropy, stream
  Device d;
  Logits z(a[0]), g(a[0]);
  const int64_t ld = z.rows(d, a[0], "logits"), dld = g.rows(d, a[4], "dlogits");
  const int32_t* targets = d.maybe<int32_t>(a[1], "targets", at::kInt, {z.M});
  const float* stats = d.take_as<float>(a[2], "stats", at::kFloat, {z.M, 2});
  const float* entropy = d.maybe<float>(a[5], "entropy", at::kFloat, {z.M});
  const float* dlogp = d.maybe<float>(a[3], "dlogp", at::kFloat, {z.M});
  const float* dentropy = d.maybe<float>(a[6], "dentropy", at::kFloat, {z.M});
  void* s = d.stream(a[7]);
  if (z.M == 0) {
    const bool pairs = given(a[1]) == given(a[3]) && given(a[5]) == given(a[6]);
    return PyLong_FromLong(z.V >= 1 && pairs && (given(a[3]) || given(a[6])) ? GPT_OK : GPT_EINVAL);
  }
  return status_of([&] {
    return gptk_logprobs_bwd(z.p, targets, stats, entropy, dlogp, dentropy, g.p, static_cast<int32_t>(z.M), static_cast<int32_t>(z.V),
                             ld, dld, z.type == at::kBFloat16, s);
  });
}

// N arguments by position; no C++ exception leaves.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, needs %zd", n, N);
    return nullptr;
  }
  try {
    return F(a);
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "a call failed");
  }
  return nullptr;
}

#define CALL(name, n) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<name, n>)), METH_FASTCALL, nullptr }

PyMethodDef g_calls[] = {CALL(rotary, 9),           CALL(paged_append, 12), CALL(paged_append4, 12), CALL(paged_load4, 7),
                         CALL(paged_attention4, 12), CALL(logprobs, 8),      CALL(logprobs_bwd, 8),   {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_calls, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&g_module); }
