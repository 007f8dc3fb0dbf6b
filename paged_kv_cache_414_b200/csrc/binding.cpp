// Argument marshalling of the calls whose GPU work is a few microseconds: the
// rotary cache write, the 8-bit pool's calls and prompt attention.  Checks the
// torch tensors it is given (place, type, shape, layout), and passes their
// pointers, sizes and the current stream to the C entry points; no step of the
// computation.  The same checks in Python took 4 to 8 us of a call of 7 to 13.
//
// Each function takes the Python wrapper's arguments in order and returns the
// call's status; it raises ValueError or TypeError for what no C entry point
// can see.  bind() hands over the entry points' addresses.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>
#include <string>

#include "pa.h"

namespace {

struct EntryPoints {
  decltype(&pa_rope_and_cache) rope;
  decltype(&pa_rope_and_cache_fp8) rope_fp8;
  decltype(&pa_paged_decode_workspace_bytes) decode_bytes;
  decltype(&pa_paged_decode_attention_fp8) decode_fp8;
  decltype(&pa_copy_blocks_fp8) copy_fp8;
  decltype(&pa_gather_cache_fp8) gather_fp8;
  decltype(&pa_prompt_attention_workspace_bytes) prompt_bytes;
  decltype(&pa_prompt_attention) prompt;
};
EntryPoints entry = {};

// A refusal: the Python exception to raise.
struct Refused {
  PyObject *type;
  std::string what;
};

std::string text(std::initializer_list<int64_t> shape) {
  std::string s = "[";
  for (int64_t n : shape) s += (s.size() > 1 ? ", " : "") + std::to_string(n);
  return s + "]";
}

// One call's device and the tensors seen on it.
class Call {
 public:
  Call(PyObject *const *args, Py_ssize_t have, Py_ssize_t want) : args_(args) {
    if (have != want) throw Refused{PyExc_TypeError, "wrong number of arguments"};
  }

  bool none(int i) const { return args_[i] == Py_None; }

  const at::Tensor &tensor(int i, const char *name) const {
    if (!THPVariable_Check(args_[i]))
      throw Refused{PyExc_TypeError, std::string(name) + " must be a torch tensor"};
    return THPVariable_Unpack(args_[i]);
  }

  // The device the call launches on is the current one; `t` must lie there.
  void place(const at::Tensor &t, const char *name) {
    if (!t.is_cuda()) throw Refused{PyExc_ValueError, std::string(name) + " must be a CUDA tensor"};
    const int current = c10::cuda::current_device();
    if (t.get_device() != current)
      throw Refused{PyExc_ValueError, std::string(name) + " is on cuda:" +
                                          std::to_string(t.get_device()) +
                                          ", the current device is " + std::to_string(current)};
    device_ = current;
  }

  // Checks place, type and shape.
  void check(const at::Tensor &t, const char *name, at::ScalarType type,
             std::initializer_list<int64_t> shape) const {
    if (!t.is_cuda() || t.get_device() != device_)
      throw Refused{PyExc_ValueError, std::string(name) + " must be a tensor on the current CUDA "
                                                          "device"};
    if (t.scalar_type() != type)
      throw Refused{PyExc_TypeError, std::string(name) + " must be " + c10::toString(type) +
                                         ", got " + c10::toString(t.scalar_type())};
    bool same = t.dim() == (int64_t)shape.size();
    int64_t k = 0;
    for (int64_t n : shape) same = same && t.size(k++) == n;
    if (!same) throw Refused{PyExc_ValueError, std::string(name) + " must be " + text(shape)};
  }

  // Pointer of a dense tensor of that type and shape.
  template <typename P>
  P *flat(int i, const char *name, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    const at::Tensor &t = tensor(i, name);
    check(t, name, type, shape);
    if (!t.is_contiguous())
      throw Refused{PyExc_ValueError, std::string(name) + " must be contiguous"};
    return static_cast<P *>(t.data_ptr());
  }

  // Pointer and token stride (elements) of [tokens, heads, head_dim] whose
  // tokens may lie apart (columns of a fused projection), heads dense.
  void *rows(int i, const char *name, at::ScalarType type, int64_t n, int64_t h, int64_t d,
             int64_t *stride) const {
    const at::Tensor &t = tensor(i, name);
    check(t, name, type, {n, h, d});
    if (n > 0 && ((d > 1 && t.stride(2) != 1) || (h > 1 && t.stride(1) != d)))
      throw Refused{PyExc_ValueError, std::string(name) + ": the heads of a token must be dense"};
    *stride = n > 1 ? t.stride(0) : h * d;
    if (*stride < h * d || *stride % 8 != 0)
      throw Refused{PyExc_ValueError, std::string(name) + ": token stride " +
                                          std::to_string(*stride) +
                                          " must be a multiple of 8, at least " +
                                          std::to_string(h * d)};
    return t.data_ptr();
  }

  int64_t whole(int i, const char *name) const {
    PyObject *n = PyNumber_Index(args_[i]);
    if (!n) {
      PyErr_Clear();
      throw Refused{PyExc_TypeError, std::string(name) + " must be an integer"};
    }
    const long long v = PyLong_AsLongLong(n);
    Py_DECREF(n);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused{PyExc_ValueError, std::string(name) + " is out of range"};
    }
    return v;
  }
  // As the C entry points take it.
  int integer(int i, const char *name) const { return narrow(whole(i, name), name); }
  static int narrow(int64_t v, const char *name) {
    if (v < INT32_MIN || v > INT32_MAX)
      throw Refused{PyExc_ValueError, std::string(name) + " is out of range"};
    return (int)v;
  }

  float real(int i, const char *name) const {
    const double v = PyFloat_AsDouble(args_[i]);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused{PyExc_TypeError, std::string(name) + " must be a number"};
    }
    return (float)v;
  }

  PyObject *object(int i) const { return args_[i]; }

  // The stream of the call: the current one, or the raw handle that argument i gives.
  cudaStream_t stream(int i) const {
    if (none(i)) return c10::cuda::getCurrentCUDAStream(device_).stream();
    return reinterpret_cast<cudaStream_t>(whole(i, "stream"));
  }

  // The caller's workspace, or scratch of `bytes` that lives until the call is
  // launched.  It is allocated on the stream that the call runs on: the memory is
  // then neither what another stream's earlier work still uses nor handed on
  // before the call is done.
  void *workspace(int i, int stream_arg, size_t bytes, size_t *have) {
    if (!none(i)) {
      const at::Tensor &t = tensor(i, "workspace");
      if (!t.is_cuda() || t.get_device() != device_ || !t.is_contiguous())
        throw Refused{PyExc_ValueError, "workspace must be a contiguous tensor on the current CUDA "
                                        "device"};
      *have = t.nbytes();
      return t.data_ptr();
    }
    *have = bytes;
    if (bytes == 0) return nullptr;
    const c10::cuda::CUDAStreamGuard on(
        none(stream_arg) ? c10::cuda::getCurrentCUDAStream(device_)
                         : c10::cuda::getStreamFromExternal(stream(stream_arg), device_));
    scratch_ = at::empty({(int64_t)bytes},
                         at::TensorOptions().dtype(at::kByte).device(at::kCUDA, device_));
    return scratch_.data_ptr();
  }

 private:
  PyObject *const *args_;
  int device_ = -1;
  at::Tensor scratch_;
};

pa_dtype code_of(const at::Tensor &t) {
  if (t.scalar_type() == at::kHalf) return PA_F16;
  if (t.scalar_type() == at::kBFloat16) return PA_BF16;
  throw Refused{PyExc_TypeError, std::string("K/V/q must be float16 or bfloat16, got ") +
                                     c10::toString(t.scalar_type())};
}

// The 8-bit pool in arguments i, i + 1, i + 2.
struct Pool8 {
  int64_t blocks, heads, block, dim;
  void *k, *v;
  float *scale;
};
void pool_shape(const at::Tensor &k) {
  if (k.dim() != 4)
    throw Refused{PyExc_ValueError,
                  "k_cache must be [num_blocks, num_kv_heads, block_size, head_dim]"};
}
Pool8 pool8(const Call &c, int i) {
  const at::Tensor &k = c.tensor(i, "k_cache");
  pool_shape(k);
  Pool8 p{k.size(0), k.size(1), k.size(2), k.size(3), nullptr, nullptr, nullptr};
  p.k = c.flat<void>(i, "k_cache", at::kFloat8_e4m3fn, {p.blocks, p.heads, p.block, p.dim});
  p.v = c.flat<void>(i + 1, "v_cache", at::kFloat8_e4m3fn, {p.blocks, p.heads, p.block, p.dim});
  p.scale = c.flat<float>(i + 2, "kv_scale", at::kFloat, {p.blocks, p.heads, 2, p.block});
  return p;
}

int n32(int64_t v) { return Call::narrow(v, "a size"); }

// q_out, q, key, value, k_cache, v_cache, kv_scale (None: 16-bit pool),
// slot_mapping, positions, cos_sin, sections, interleaved, stream
int rope(PyObject *const *args, Py_ssize_t n) {
  Call c(args, n, 13);
  const at::Tensor &key = c.tensor(2, "key");
  c.place(key, "key");
  const pa_dtype code = code_of(key);
  const at::ScalarType type = key.scalar_type();
  const bool fp8 = !c.none(6);
  Pool8 p;
  if (fp8) {
    p = pool8(c, 4);
  } else {
    const at::Tensor &k = c.tensor(4, "k_cache");
    pool_shape(k);
    p = {k.size(0), k.size(1), k.size(2), k.size(3), nullptr, nullptr, nullptr};
    p.k = c.flat<void>(4, "k_cache", type, {p.blocks, p.heads, p.block, p.dim});
    p.v = c.flat<void>(5, "v_cache", type, {p.blocks, p.heads, p.block, p.dim});
  }
  const int64_t T = key.dim() == 3 ? key.size(0) : 0;
  int64_t ks, vs, qs = 0, qos = 0, Hq = 0;
  const void *k = c.rows(2, "key", type, T, p.heads, p.dim, &ks);
  const void *v = c.rows(3, "value", type, T, p.heads, p.dim, &vs);
  const int64_t *slots = c.flat<int64_t>(7, "slot_mapping", at::kLong, {T});
  const void *q = nullptr;
  void *q_out = nullptr;
  if (!c.none(1)) {
    const at::Tensor &t = c.tensor(1, "q");
    Hq = t.dim() == 3 ? t.size(1) : 0;
    q = c.rows(1, "q", type, T, Hq, p.dim, &qs);
    q_out = c.rows(0, "q_out", type, T, Hq, p.dim, &qos);
  }
  int64_t most = 0, rot = 0, axes = 0;
  const float *table = nullptr;
  const int64_t *pos = nullptr;
  int sect[8] = {};
  if (!c.none(9)) {
    const at::Tensor &t = c.tensor(9, "cos_sin");
    if (t.dim() != 2) throw Refused{PyExc_ValueError, "cos_sin must be [max_position, rotary_dim]"};
    most = t.size(0);
    rot = t.size(1);
    table = c.flat<float>(9, "cos_sin", at::kFloat, {most, rot});
    const at::Tensor &ps = c.tensor(8, "positions");
    axes = ps.dim() == 2 ? ps.size(0) : 1;
    pos = ps.dim() == 2 ? c.flat<int64_t>(8, "positions", at::kLong, {axes, T})
                        : c.flat<int64_t>(8, "positions", at::kLong, {T});
    if (c.none(10)) {
      if (axes != 1) throw Refused{PyExc_ValueError, "sections must name every axis"};
      sect[0] = (int)(rot / 2);
    } else {
      PyObject *s = PySequence_Fast(c.object(10), "sections must be a sequence");
      if (!s) {
        PyErr_Clear();
        throw Refused{PyExc_TypeError, "sections must be a sequence"};
      }
      const Py_ssize_t many = PySequence_Fast_GET_SIZE(s);
      bool good = many == axes;
      for (Py_ssize_t i = 0; good && i < many && i < 8; ++i) {
        const long v = PyLong_AsLong(PySequence_Fast_GET_ITEM(s, i));
        if (v == -1 && PyErr_Occurred()) {
          PyErr_Clear();
          good = false;
        }
        sect[i] = v > INT32_MAX || v < INT32_MIN ? -1 : (int)v;
      }
      Py_DECREF(s);
      if (!good)
        throw Refused{PyExc_ValueError,
                      "sections must name every axis: " + std::to_string(axes) + " of them"};
    }
  }
  const int turn = PyObject_IsTrue(c.object(11));
  if (turn < 0) {
    PyErr_Clear();
    throw Refused{PyExc_TypeError, "interleaved must be true or false"};
  }
  const cudaStream_t st = c.stream(12);
  if (fp8)
    return entry.rope_fp8(q_out, q, k, v, p.k, p.v, p.scale, slots, pos, table, sect, n32(axes),
                          n32(rot), n32(most), turn, qos, qs, ks, vs, n32(T), n32(Hq),
                          n32(p.heads), n32(p.dim), n32(p.block), n32(p.blocks), code, st);
  return entry.rope(q_out, q, k, v, p.k, p.v, slots, pos, table, sect, n32(axes), n32(rot),
                    n32(most), turn, qos, qs, ks, vs, n32(T), n32(Hq), n32(p.heads), n32(p.dim),
                    n32(p.block), n32(p.blocks), code, st);
}

// out, q, k_cache, v_cache, kv_scale, block_tables, context_lens, scale,
// num_kv_heads, max_context_len, workspace, stream
int decode_fp8(PyObject *const *args, Py_ssize_t n) {
  Call c(args, n, 12);
  const at::Tensor &q = c.tensor(1, "q");
  c.place(q, "q");
  const pa_dtype code = code_of(q);
  const Pool8 p = pool8(c, 2);
  const at::Tensor &tables = c.tensor(5, "block_tables");
  if (q.dim() != 3 || p.heads != c.whole(8, "num_kv_heads") || tables.dim() != 2)
    throw Refused{PyExc_ValueError, "q [S, Hq, D], block_tables [S, max_blocks] and a cache of "
                                    "num_kv_heads heads expected"};
  const int64_t S = q.size(0), Hq = q.size(1), maxb = tables.size(1);
  const int most = c.none(9) ? n32(maxb * p.block) : c.integer(9, "max_context_len");
  float *out = c.flat<float>(0, "out", at::kFloat, {S, Hq, p.dim});
  const void *qp = c.flat<void>(1, "q", q.scalar_type(), {S, Hq, p.dim});
  const int32_t *tp = c.flat<int32_t>(5, "block_tables", at::kInt, {S, maxb});
  const int32_t *lens = c.flat<int32_t>(6, "context_lens", at::kInt, {S});
  size_t have, need = 0;
  if (c.none(10))
    need = entry.decode_bytes(n32(S), n32(Hq), n32(p.heads), n32(p.dim), n32(p.block), most);
  void *ws = c.workspace(10, 11, need, &have);
  return entry.decode_fp8(out, qp, p.k, p.v, p.scale, tp, lens, c.real(7, "scale"), n32(p.heads),
                          n32(S), n32(Hq), n32(p.dim), n32(p.block), n32(maxb), most,
                          n32(p.blocks), code, ws, have, c.stream(11));
}

// k_cache, v_cache, kv_scale, block_mapping, stream
int copy_fp8(PyObject *const *args, Py_ssize_t n) {
  Call c(args, n, 5);
  c.place(c.tensor(0, "k_cache"), "k_cache");
  const Pool8 p = pool8(c, 0);
  const at::Tensor &m = c.tensor(3, "block_mapping");
  const int64_t many = m.dim() == 2 ? m.size(0) : 0;
  const int64_t *pairs = c.flat<int64_t>(3, "block_mapping", at::kLong, {many, 2});
  return entry.copy_fp8(p.k, p.v, p.scale, pairs, n32(many), n32(p.heads), n32(p.dim),
                        n32(p.block), n32(p.blocks), c.stream(4));
}

// key, value, k_cache, v_cache, kv_scale, block_tables, key_start, stream
int gather_fp8(PyObject *const *args, Py_ssize_t n) {
  Call c(args, n, 8);
  const at::Tensor &key = c.tensor(0, "key");
  c.place(key, "key");
  const pa_dtype code = code_of(key);
  const Pool8 p = pool8(c, 2);
  const at::Tensor &tables = c.tensor(5, "block_tables"), &start = c.tensor(6, "key_start");
  if (key.dim() != 3 || tables.dim() != 2 || start.dim() != 1)
    throw Refused{PyExc_ValueError, "key [T, Hkv, D], block_tables [S, max_blocks] and key_start "
                                    "[S + 1] expected"};
  const int64_t T = key.size(0), maxb = tables.size(1);
  const int64_t S = start.size(0) > 0 ? start.size(0) - 1 : 0;
  void *kp = c.flat<void>(0, "key", key.scalar_type(), {T, p.heads, p.dim});
  void *vp = c.flat<void>(1, "value", key.scalar_type(), {T, p.heads, p.dim});
  const int32_t *tp = c.flat<int32_t>(5, "block_tables", at::kInt, {S, maxb});
  const int32_t *sp = c.flat<int32_t>(6, "key_start", at::kInt, {S + 1});
  return entry.gather_fp8(kp, vp, p.k, p.v, p.scale, tp, sp, n32(S), n32(T), n32(p.heads),
                          n32(p.dim), n32(p.block), n32(maxb), n32(p.blocks), code, c.stream(7));
}

// out, q, key, value, query_start, key_start, scale, num_kv_heads,
// max_query_len, max_key_len, workspace, stream
int prompt(PyObject *const *args, Py_ssize_t n) {
  Call c(args, n, 12);
  const at::Tensor &q = c.tensor(1, "q"), &key = c.tensor(2, "key");
  c.place(q, "q");
  const at::Tensor &start = c.tensor(4, "query_start");
  if (q.dim() != 3 || key.dim() != 3 || key.size(1) != c.whole(7, "num_kv_heads") ||
      start.dim() != 1)
    throw Refused{PyExc_ValueError,
                  "q [T, Hq, D], key [Tk, num_kv_heads, D] and query_start [S + 1] expected"};
  const pa_dtype code = code_of(q);
  const at::ScalarType type = q.scalar_type();
  const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), Tk = key.size(0), Hkv = key.size(1);
  const int64_t S = start.size(0) > 0 ? start.size(0) - 1 : 0;
  int64_t qs, ks, vs;
  const void *qp = c.rows(1, "q", type, T, Hq, D, &qs);
  const void *k = c.rows(2, "key", type, Tk, Hkv, D, &ks);
  const void *v = c.rows(3, "value", type, Tk, Hkv, D, &vs);
  void *out = c.flat<void>(0, "out", type, {T, Hq, D});
  const int32_t *qst = c.flat<int32_t>(4, "query_start", at::kInt, {S + 1});
  const int32_t *kst = c.flat<int32_t>(5, "key_start", at::kInt, {S + 1});
  const int mq = c.integer(8, "max_query_len"), mk = c.integer(9, "max_key_len");
  size_t have, need = 0;
  if (c.none(10)) need = entry.prompt_bytes(n32(S), n32(T), n32(Hq), n32(Hkv), n32(D), mq, mk);
  void *ws = c.workspace(10, 11, need, &have);
  return entry.prompt(out, qp, k, v, qst, kst, c.real(6, "scale"), n32(Hkv), n32(S), n32(T),
                      n32(Tk), n32(Hq), n32(D), mq, mk, qs, ks, vs, code, ws, have, c.stream(11));
}

template <int (*F)(PyObject *const *, Py_ssize_t)>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
  try {
    if (!entry.prompt) throw Refused{PyExc_RuntimeError, "bind() was not called"};
    return PyLong_FromLong(F(args, n));
  } catch (const Refused &r) {
    PyErr_SetString(r.type, r.what.c_str());
  } catch (const std::exception &e) {   // torch's own: out of memory, no device
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// The addresses of the entry points, in the order of EntryPoints.
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "bind: eight addresses expected");
    return nullptr;
  }
  void *at[8];
  for (int i = 0; i < 8; ++i) {
    at[i] = PyLong_AsVoidPtr(args[i]);
    if (!at[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null address");
      return nullptr;
    }
  }
  entry.rope = reinterpret_cast<decltype(entry.rope)>(at[0]);
  entry.rope_fp8 = reinterpret_cast<decltype(entry.rope_fp8)>(at[1]);
  entry.decode_bytes = reinterpret_cast<decltype(entry.decode_bytes)>(at[2]);
  entry.decode_fp8 = reinterpret_cast<decltype(entry.decode_fp8)>(at[3]);
  entry.copy_fp8 = reinterpret_cast<decltype(entry.copy_fp8)>(at[4]);
  entry.gather_fp8 = reinterpret_cast<decltype(entry.gather_fp8)>(at[5]);
  entry.prompt_bytes = reinterpret_cast<decltype(entry.prompt_bytes)>(at[6]);
  entry.prompt = reinterpret_cast<decltype(entry.prompt)>(at[7]);
  Py_RETURN_NONE;
}

#define PA_METHOD(name, fn) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(fn)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PA_METHOD("bind", bind),
                         PA_METHOD("rope", call<rope>),
                         PA_METHOD("decode_fp8", call<decode_fp8>),
                         PA_METHOD("copy_fp8", call<copy_fp8>),
                         PA_METHOD("gather_fp8", call<gather_fp8>),
                         PA_METHOD("prompt", call<prompt>),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr,               nullptr,  nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
