// The serving-step calls of include/pa.h for torch tensors: a Python extension that checks its
// arguments and calls the library. The other calls go through ctypes; these take a few
// microseconds on the GPU at decode sizes, and the checks and marshalling of 10 to 31 arguments
// took 7 to 11 us of host time a call in Python (2.0 to 2.5 here). Same rules: contiguous tensors of
// one CUDA device, the current stream of that device unless `stream` is given, TypeError /
// ValueError for tensors that do not fit, PAError for what the library refuses.
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "pa.h"

namespace {

PyObject* g_error = nullptr;  // PAError, from init()

struct Refused {};  // a Python error is set

[[noreturn]] void refuse(PyObject* type, const char* fmt, const char* name, const char* more = "") {
  PyErr_Format(type, fmt, name, more);
  throw Refused{};
}

// ---------------------------------------------------------------- arguments by name
// names[0 .. positional) may be given by position, all by name; defaults (null: required) as given.
template <int N>
struct Args {
  PyObject* v[N] = {};
  Args(const char* fn, const char* const (&names)[N], int positional, int required, PyObject* const* args, Py_ssize_t n,
       PyObject* kwnames) {
    if (n > positional) {
      PyErr_Format(PyExc_TypeError, "%s() takes %d positional arguments but %zd were given", fn, positional, n);
      throw Refused{};
    }
    for (Py_ssize_t i = 0; i < n; ++i) v[i] = args[i];
    const Py_ssize_t k = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
    for (Py_ssize_t i = 0; i < k; ++i) {
      const char* key = PyUnicode_AsUTF8(PyTuple_GET_ITEM(kwnames, i));
      if (!key) throw Refused{};
      int at = 0;
      while (at < N && std::strcmp(key, names[at]) != 0) ++at;
      if (at == N || v[at]) {
        PyErr_Format(PyExc_TypeError, at == N ? "%s() got an unexpected keyword argument '%s'" :
                     "%s() got multiple values for argument '%s'", fn, key);
        throw Refused{};
      }
      v[at] = args[n + i];
    }
    for (int i = 0; i < required; ++i)
      if (!v[i]) {
        PyErr_Format(PyExc_TypeError, "%s() missing required argument: '%s'", fn, names[i]);
        throw Refused{};
      }
  }
};

int64_t integer(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Refused{};
  return x;
}
int int32(PyObject* o, const char* name) {
  const int64_t x = integer(o);
  if (x != int64_t(int(x))) refuse(PyExc_ValueError, "%s is out of range", name);
  return int(x);
}
double real(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Refused{};
  return x;
}

// ---------------------------------------------------------------- tensors
const at::Tensor& tensor(PyObject* o, const char* name, int dims) {
  if (!THPVariable_Check(o)) refuse(PyExc_ValueError, "%s must be a tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.dim() != dims) refuse(PyExc_ValueError, "%s has the wrong number of dims", name);
  return t;
}

int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", name);
  return t.get_device();
}

void check(const at::Tensor& t, const char* name, int dev, at::ScalarType type, std::initializer_list<int64_t> shape) {
  if (!t.is_cuda() || t.get_device() != dev) refuse(PyExc_ValueError, "%s must be on the CUDA device of the others", name);
  if (t.scalar_type() != type) refuse(PyExc_TypeError, "%s must be %s", name, c10::toString(type));
  bool same = t.dim() == int64_t(shape.size());
  if (same) {
    int i = 0;
    for (int64_t n : shape) same = same && t.size(i++) == n;
  }
  if (!same) refuse(PyExc_ValueError, "%s has the wrong shape", name);
}

// Address of a contiguous tensor of the given device, type and shape.
void* address(PyObject* o, const char* name, int dev, at::ScalarType type, std::initializer_list<int64_t> shape) {
  if (!THPVariable_Check(o)) refuse(PyExc_ValueError, "%s must be a tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  check(t, name, dev, type, shape);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
  return t.data_ptr();
}
template <typename T>
T* at_(PyObject* o, const char* name, int dev, at::ScalarType type, std::initializer_list<int64_t> shape) {
  return static_cast<T*>(address(o, name, dev, type, shape));
}

// A [num_tokens, heads, head_dim] tensor whose tokens may lie apart (a slice of a wider
// projection): its address, and the elements between tokens.
void* token_rows(PyObject* o, const char* name, int dev, at::ScalarType type, int64_t T, int64_t H, int64_t D,
                 int64_t* stride) {
  if (!THPVariable_Check(o)) refuse(PyExc_ValueError, "%s must be a tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  check(t, name, dev, type, {T, H, D});
  if (T > 0 && (t.stride(2) != 1 || (t.stride(1) != D && H > 1)))
    refuse(PyExc_ValueError, "%s: a token's heads must be contiguous", name);
  *stride = T > 1 ? t.stride(0) : H * D;
  return t.data_ptr();
}

pa_dtype code(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kFloat: return PA_F32;
    case at::kBFloat16: return PA_BF16;
    case at::kFloat8_e4m3fn: return PA_FP8_E4M3;
    default: refuse(PyExc_TypeError, "%s: unsupported dtype (float32, bfloat16 or float8_e4m3fn)", name);
  }
}

// The device made current while it lasts (the library works on the current device), and the
// stream to launch on: `stream`, or the device's current one.
struct On {
  int before;
  bool moved;
  pa_stream_t stream;
  On(int dev, PyObject* s) : before(c10::cuda::current_device()), moved(before != dev) {
    if (s && s != Py_None) {
      PyObject* h = PyObject_GetAttrString(s, "cuda_stream");
      if (!h) throw Refused{};
      stream = static_cast<pa_stream_t>(PyLong_AsVoidPtr(h));
      Py_DECREF(h);
      if (PyErr_Occurred()) throw Refused{};
    } else {
      stream = reinterpret_cast<pa_stream_t>(c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(dev)).stream());
    }
    if (moved) c10::cuda::set_device(c10::DeviceIndex(dev));
  }
  ~On() {
    if (moved) c10::cuda::set_device(c10::DeviceIndex(before));
  }
};

// Calls the library with the interpreter's lock released, as ctypes does: a launch waits where the
// stream's queue is full, perhaps for a Python function queued there. (The arguments' tensors are
// held by the caller.) Returns `value`, or raises.
template <typename F>
PyObject* result(const char* fn, PyObject* value, F call) {
  PyThreadState* const state = PyEval_SaveThread();
  const int status = call();
  PyEval_RestoreThread(state);
  if (status != PA_OK) {
    PyObject* e = PyObject_CallFunction(g_error, "is", status, fn);
    if (e) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
    return nullptr;
  }
  Py_INCREF(value);
  return value;
}

// Runs a call's body; C++ exceptions end here.
template <typename F>
PyObject* guarded(F body) {
  try {
    return body();
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

constexpr auto kI32 = at::kInt;
constexpr auto kI64 = at::kLong;

// ---------------------------------------------------------------- the calls
PyObject* advance_batch(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"block_table", "seq_lens", "query_lens", "free_blocks", "free_head", "seq_lens_out",
                                        "free_head_out", "query_start_loc", "slot_mapping", "positions", "block_size",
                                        "num_blocks", "stream"};
    const Args<13> a("advance_batch", names, 10, 12, args, n, kw);
    const at::Tensor& table = tensor(a.v[0], names[0], 2);
    const int dev = device_of(table, names[0]);
    const int64_t S = table.size(0), W = table.size(1), F = tensor(a.v[3], names[3], 1).size(0),
                  T = tensor(a.v[8], names[8], 1).size(0);
    if (S > INT32_MAX - 1 || W > INT32_MAX || F > INT32_MAX || T > INT32_MAX)
      refuse(PyExc_ValueError, "%s: too many elements", names[0]);
    auto i32 = [&](int i, std::initializer_list<int64_t> shape) { return at_<int32_t>(a.v[i], names[i], dev, kI32, shape); };
    int32_t* p[10] = {i32(0, {S, W}), i32(1, {S}), i32(2, {S}),     i32(3, {F}), i32(4, {1}),
                      i32(5, {S}),    i32(6, {1}), i32(7, {S + 1}), nullptr,     i32(9, {T})};
    auto slots = at_<int64_t>(a.v[8], names[8], dev, kI64, {T});
    const int B = int32(a.v[10], names[10]);
    const int64_t NB = integer(a.v[11]);
    const On on(dev, a.v[12]);
    return result("pa_advance_batch", Py_None, [&] {
      return pa_advance_batch(p[0], int(W), p[1], p[2], p[3], int(F), p[4], p[5], p[6], p[7], slots, p[9], int(S), int(T),
                              B, NB, on.stream);
    });
  });
}

PyObject* norm_rope_write(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"q_out", "q", "k", "v", "q_weight", "k_weight", "cos_sin", "positions",
                                        "slot_mapping", "k_cache", "v_cache", "eps", "interleaved", "sections", "k_scale",
                                        "v_scale", "stream"};
    const Args<17> a("norm_rope_write", names, 11, 11, args, n, kw);
    const at::Tensor &kc = tensor(a.v[9], names[9], 4), &q = tensor(a.v[1], names[1], 3), &cs = tensor(a.v[6], names[6], 2);
    const int dev = device_of(kc, names[9]);
    const int64_t NB = kc.size(0), B = kc.size(1), Hkv = kc.size(2), D = kc.size(3), T = q.size(0), Hq = q.size(1),
                  limit = cs.size(0), rot = cs.size(1);
    if (B > INT32_MAX || Hkv > INT32_MAX || D > INT32_MAX || Hq > INT32_MAX || limit > INT32_MAX || rot > INT32_MAX)
      refuse(PyExc_ValueError, "%s: too many elements", names[9]);
    const auto type = q.scalar_type(), cache_type = kc.scalar_type();
    int axes = 1, sections[4] = {int(rot / 2), 0, 0, 0};
    if (a.v[13] && a.v[13] != Py_None) {
      PyObject* seq = PySequence_Fast(a.v[13], "sections must be a sequence");
      if (!seq) throw Refused{};
      const Py_ssize_t len = PySequence_Fast_GET_SIZE(seq);
      bool fits = len >= 1 && len <= 4;
      for (Py_ssize_t i = 0; fits && i < len; ++i) {
        const long long x = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(seq, i));
        if (x == -1 && PyErr_Occurred()) {
          Py_DECREF(seq);
          throw Refused{};
        }
        fits = x >= 0 && x <= INT32_MAX;
        sections[i] = int(x);
      }
      Py_DECREF(seq);
      if (!fits) refuse(PyExc_ValueError, "%s: one to four pair counts", names[13]);
      axes = int(len);
    }
    const bool many = a.v[13] && a.v[13] != Py_None;
    int64_t qs, ks, vs;
    void* out = address(a.v[0], names[0], dev, type, {T, Hq, D});
    void* qp = token_rows(a.v[1], names[1], dev, type, T, Hq, D, &qs);
    void* kp = token_rows(a.v[2], names[2], dev, type, T, Hkv, D, &ks);
    void* vp = token_rows(a.v[3], names[3], dev, type, T, Hkv, D, &vs);
    void* w[2];
    for (int i = 0; i < 2; ++i)
      w[i] = a.v[4 + i] == Py_None ? nullptr : address(a.v[4 + i], names[4 + i], dev, type, {D});
    auto table = at_<float>(a.v[6], names[6], dev, at::kFloat, {limit, rot});
    auto pos = many ? at_<int32_t>(a.v[7], names[7], dev, kI32, {axes, T}) : at_<int32_t>(a.v[7], names[7], dev, kI32, {T});
    auto slots = at_<int64_t>(a.v[8], names[8], dev, kI64, {T});
    void* kcp = address(a.v[9], names[9], dev, cache_type, {NB, B, Hkv, D});
    void* vcp = address(a.v[10], names[10], dev, cache_type, {NB, B, Hkv, D});
    const float eps = a.v[11] ? float(real(a.v[11])) : 1e-6f;
    const int interleaved = a.v[12] ? PyObject_IsTrue(a.v[12]) : 0;
    if (interleaved < 0) throw Refused{};
    const float k_scale = a.v[14] ? float(real(a.v[14])) : 1.f, v_scale = a.v[15] ? float(real(a.v[15])) : 1.f;
    const pa_dtype dt = code(q, names[1]), cdt = code(kc, names[9]);
    const On on(dev, a.v[16]);
    return result("pa_norm_rope_write", a.v[0], [&] {
      return pa_norm_rope_write(out, qp, kp, vp, qs, ks, vs, w[0], w[1], eps, table, int(limit), int(rot), interleaved,
                                pos, axes, sections, slots, kcp, vcp, T, NB, int(B), int(Hq), int(Hkv), int(D), dt, cdt,
                                k_scale, v_scale, on.stream);
    });
  });
}

// block_table, seq_lens, query_start_loc of a batch, at arguments `at`, at + 1, at + 2
struct Batch {
  int32_t *table, *lens, *qsl;
  int S, W;
  Batch(PyObject* const* v, const char* const* names, int at, int dev) {
    const at::Tensor& t = tensor(v[at], names[at], 2);
    const int64_t s = t.size(0), w = t.size(1);
    if (s > INT32_MAX - 1 || w > INT32_MAX) refuse(PyExc_ValueError, "%s: too many elements", names[at]);
    table = at_<int32_t>(v[at], names[at], dev, kI32, {s, w});
    lens = at_<int32_t>(v[at + 1], names[at + 1], dev, kI32, {s});
    qsl = at_<int32_t>(v[at + 2], names[at + 2], dev, kI32, {s + 1});
    S = int(s);
    W = int(w);
  }
};

int size32(const at::Tensor& t, int i, const char* name) {
  if (t.size(i) > INT32_MAX) refuse(PyExc_ValueError, "%s: too many elements", name);
  return int(t.size(i));
}

PyObject* block_bounds(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"bounds", "k_cache", "block_table", "seq_lens", "query_start_loc", "max_query_len",
                                        "max_seq_len", "num_tokens", "stream"};
    const Args<9> a("block_bounds", names, 5, 7, args, n, kw);
    const at::Tensor& kc = tensor(a.v[1], names[1], 4);
    const int dev = device_of(kc, names[1]);
    const int64_t NB = kc.size(0);
    const int B = size32(kc, 1, names[1]), Hkv = size32(kc, 2, names[1]), D = size32(kc, 3, names[1]);
    void* bounds = address(a.v[0], names[0], dev, at::kBFloat16, {NB, Hkv, 2, D});
    void* kcp = address(a.v[1], names[1], dev, kc.scalar_type(), {NB, B, Hkv, D});
    const Batch b(a.v, names, 2, dev);
    const int max_q = int32(a.v[5], names[5]), max_s = int32(a.v[6], names[6]);
    const int64_t most = int64_t(b.S) * max_q;
    const int T = a.v[7] && a.v[7] != Py_None ? int32(a.v[7], names[7]) : most > INT32_MAX ? INT32_MAX : int(most);
    const pa_dtype dt = code(kc, names[1]);
    const On on(dev, a.v[8]);
    return result("pa_block_bounds", a.v[0], [&] {
      return pa_block_bounds(bounds, kcp, b.table, b.W, b.lens, b.qsl, b.S, T, max_q, max_s, Hkv, D, B, NB, dt,
                             on.stream);
    });
  });
}

PyObject* block_scores(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"scores", "q", "bounds", "block_table", "seq_lens", "query_start_loc", "block_size",
                                        "max_query_len", "max_seq_len", "stream"};
    const Args<10> a("block_scores", names, 6, 9, args, n, kw);
    const at::Tensor &q = tensor(a.v[1], names[1], 3), &bd = tensor(a.v[2], names[2], 4), &sc = tensor(a.v[0], names[0], 3);
    const int dev = device_of(q, names[1]);
    const int T = size32(q, 0, names[1]), Hq = size32(q, 1, names[1]), D = size32(q, 2, names[1]),
              Hkv = size32(bd, 1, names[2]), width = size32(sc, 2, names[0]);
    const int64_t NB = bd.size(0);
    auto scores = at_<float>(a.v[0], names[0], dev, at::kFloat, {T, Hkv, width});
    void* qp = address(a.v[1], names[1], dev, at::kBFloat16, {T, Hq, D});
    void* bp = address(a.v[2], names[2], dev, at::kBFloat16, {NB, Hkv, 2, D});
    const Batch b(a.v, names, 3, dev);
    const int B = int32(a.v[6], names[6]), max_q = int32(a.v[7], names[7]), max_s = int32(a.v[8], names[8]);
    const On on(dev, a.v[9]);
    return result("pa_block_scores", a.v[0], [&] {
      return pa_block_scores(scores, width, qp, bp, b.table, b.W, b.lens, b.qsl, b.S, T, max_q, max_s, Hq, Hkv, D, B, NB,
                             on.stream);
    });
  });
}

PyObject* select_blocks(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"block_idx", "scores", "seq_lens", "query_start_loc", "block_size", "init_blocks",
                                        "local_blocks", "stream"};
    const Args<8> a("select_blocks", names, 4, 5, args, n, kw);
    const at::Tensor &sc = tensor(a.v[1], names[1], 3), &ix = tensor(a.v[0], names[0], 3), &ln = tensor(a.v[2], names[2], 1);
    const int dev = device_of(sc, names[1]);
    const int T = size32(sc, 0, names[1]), Hkv = size32(sc, 1, names[1]), width = size32(sc, 2, names[1]),
              k = size32(ix, 2, names[0]), S = size32(ln, 0, names[2]);
    auto idx = at_<int32_t>(a.v[0], names[0], dev, kI32, {T, Hkv, k});
    auto scores = at_<float>(a.v[1], names[1], dev, at::kFloat, {T, Hkv, width});
    auto lens = at_<int32_t>(a.v[2], names[2], dev, kI32, {S});
    auto qsl = at_<int32_t>(a.v[3], names[3], dev, kI32, {int64_t(S) + 1});
    const int B = int32(a.v[4], names[4]), init = a.v[5] ? int32(a.v[5], names[5]) : 0,
              local = a.v[6] ? int32(a.v[6], names[6]) : 0;
    const On on(dev, a.v[7]);
    return result("pa_select_blocks", a.v[0], [&] {
      return pa_select_blocks(idx, k, scores, width, lens, qsl, S, T, Hkv, B, init, local, on.stream);
    });
  });
}

PyObject* attention_sparse(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"out", "q", "k_cache", "v_cache", "block_table", "seq_lens", "query_start_loc",
                                        "block_idx", "max_seq_len", "scale", "k_scale", "v_scale", "stream"};
    const Args<13> a("attention_sparse", names, 8, 10, args, n, kw);
    const at::Tensor &kc = tensor(a.v[2], names[2], 4), &q = tensor(a.v[1], names[1], 3), &ix = tensor(a.v[7], names[7], 3);
    const int dev = device_of(kc, names[2]);
    const int64_t NB = kc.size(0);
    const int B = size32(kc, 1, names[2]), Hkv = size32(kc, 2, names[2]), D = size32(kc, 3, names[2]),
              T = size32(q, 0, names[1]), Hq = size32(q, 1, names[1]), k = size32(ix, 2, names[7]);
    void* out = address(a.v[0], names[0], dev, at::kBFloat16, {T, Hq, D});
    void* qp = address(a.v[1], names[1], dev, at::kBFloat16, {T, Hq, D});
    void* kcp = address(a.v[2], names[2], dev, kc.scalar_type(), {NB, B, Hkv, D});
    void* vcp = address(a.v[3], names[3], dev, kc.scalar_type(), {NB, B, Hkv, D});
    const Batch b(a.v, names, 4, dev);
    auto idx = at_<int32_t>(a.v[7], names[7], dev, kI32, {T, Hkv, k});
    const int max_s = int32(a.v[8], names[8]);
    const float scale = float(real(a.v[9])), k_scale = a.v[10] ? float(real(a.v[10])) : 1.f,
                v_scale = a.v[11] ? float(real(a.v[11])) : 1.f;
    const pa_dtype dt = code(kc, names[2]);
    const On on(dev, a.v[12]);
    return result("pa_attention_sparse", a.v[0], [&] {
      return pa_attention_sparse(out, qp, kcp, vcp, b.table, b.W, b.lens, b.qsl, idx, k, b.S, T, max_s, Hq, Hkv, D, B, NB,
                                 scale, dt, k_scale, v_scale, on.stream);
    });
  });
}

PyObject* init(PyObject*, PyObject* error) {
  Py_INCREF(error);
  Py_XDECREF(g_error);
  g_error = error;
  Py_RETURN_NONE;
}

#define PA_CALL(name, doc) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL | METH_KEYWORDS, doc}

PyMethodDef methods[] = {
    PA_CALL(advance_batch,
            "advance_batch($module, block_table, seq_lens, query_lens, free_blocks, free_head, seq_lens_out,\n"
            "              free_head_out, query_start_loc, slot_mapping, positions, *, block_size,\n"
            "              num_blocks, stream=None)\n--\n\n"
            "pa_advance_batch: a step's block tables, slots and positions from request lengths, on the GPU.\n\n"
            "block_table int32 [S, W] (new entries written), seq_lens and query_lens int32 [S], free_blocks\n"
            "int32 [F] with free_head int32 [1] entries already taken; writes seq_lens_out [S] and\n"
            "free_head_out [1] (each may be its input), query_start_loc int32 [S + 1], slot_mapping int64\n"
            "[T] and positions int32 [T]; tokens behind the last request's get slot -1 and position 0. A\n"
            "step that does not fit changes nothing (read_device_errors tells)."),
    PA_CALL(norm_rope_write,
            "norm_rope_write($module, q_out, q, k, v, q_weight, k_weight, cos_sin, positions, slot_mapping,\n"
            "                k_cache, v_cache, *, eps=1e-6, interleaved=False, sections=None, k_scale=1.0,\n"
            "                v_scale=1.0, stream=None)\n--\n\n"
            "pa_norm_rope_write: RMS norm of each query and key head (weights [head_dim], or None: no norm),\n"
            "rotary positions, and the cache write, in one pass; returns q_out.\n\n"
            "q [T, Hq, D], k and v [T, Hkv, D]: bfloat16 or float32, tokens may lie apart (slices of one\n"
            "projection); q_out [T, Hq, D] contiguous (may be q). cos_sin float32 [max_position, rot_dim]\n"
            "(cosines, then sines); positions int32 [T], or [axes, T] with sections = the pair counts of\n"
            "the axes. Caches in q's dtype or float8_e4m3fn (codes of x / scale)."),
    PA_CALL(block_bounds,
            "block_bounds($module, bounds, k_cache, block_table, seq_lens, query_start_loc, *, max_query_len,\n"
            "             max_seq_len, num_tokens=None, stream=None)\n--\n\n"
            "pa_block_bounds: bounds[block, head, 0 / 1] = the smallest / largest cached key per dimension,\n"
            "for every block that holds one of the batch's query tokens; returns bounds, bfloat16\n"
            "[num_blocks, Hkv, 2, D]. Caches bfloat16 or float8_e4m3fn (bounds of the codes' values).\n"
            "num_tokens: the batch's query tokens or more (it sizes the grid; None: S * max_query_len)."),
    PA_CALL(block_scores,
            "block_scores($module, scores, q, bounds, block_table, seq_lens, query_start_loc, *, block_size,\n"
            "             max_query_len, max_seq_len, stream=None)\n--\n\n"
            "pa_block_scores: scores[t, head, block] = an upper bound of the block's logits (before the\n"
            "softmax scale) over the head's query group; -inf behind the token's context; returns scores,\n"
            "float32 [T, Hkv, score_width], score_width * block_size >= max_seq_len. q bfloat16 [T, Hq, D]."),
    PA_CALL(select_blocks,
            "select_blocks($module, block_idx, scores, seq_lens, query_start_loc, *, block_size,\n"
            "              init_blocks=0, local_blocks=0, stream=None)\n--\n\n"
            "pa_select_blocks: block_idx[t, head] = the first init_blocks and last local_blocks of the\n"
            "token's context and the blocks of the largest scores (equal ones: the lowest), ascending, -1\n"
            "behind them; returns block_idx, int32 [T, Hkv, num_select]. scores float32 [T, Hkv, width]."),
    PA_CALL(attention_sparse,
            "attention_sparse($module, out, q, k_cache, v_cache, block_table, seq_lens, query_start_loc,\n"
            "                 block_idx, *, max_seq_len, scale, k_scale=1.0, v_scale=1.0, stream=None)\n--\n\n"
            "pa_attention_sparse: attention of each query token over the blocks listed in block_idx\n"
            "[T, Hkv, num_select] (logical blocks of its request, entries < 0 skipped), causal; zeros for\n"
            "an empty list; returns out. out, q bfloat16 [T, Hq, D]; caches bfloat16, or float8_e4m3fn\n"
            "with scales."),
    {"init", init, METH_O, "init(PAError): the class raised for what the library refuses."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pa_torch", "The serving-step calls of the library for torch tensors.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pa_torch() { return PyModule_Create(&module); }
