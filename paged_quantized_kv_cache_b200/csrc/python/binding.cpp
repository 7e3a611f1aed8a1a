// binding.cpp -- argument marshalling of the calls around a serving step, for
// Python: checks the tensors of a call and hands their pointers to the C ABI
// (include/pqkv.h). A step of a few tokens takes the GPU some microseconds, and
// the same checks and conversions written in Python took as long again: 6 of
// the 11 us of a qk_norm_rope call of one token.
//
// The module holds no library code: bind() gives it the addresses of libpqkv's
// functions. Each function takes the device's index, a stream handle and the
// call's arguments, raises ValueError for tensors that the call does not take,
// and returns the library's status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>

#include "pqkv.h"

namespace {

decltype(&pqkv_build_batch) f_build_batch = nullptr;
decltype(&pqkv_qk_norm_rope) f_qk_norm_rope = nullptr;
decltype(&pqkv_qkv_norm_rope_write) f_qkv_norm_rope_write = nullptr;
decltype(&pqkv_paged_cross_attention) f_paged_cross_attention = nullptr;
decltype(&pqkv_cache_layout) f_cache_layout = nullptr;

struct Refused {
  std::string why;
};

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kInt: return "int32";
    case at::kFloat: return "float32";
    case at::kHalf: return "float16";
    case at::kBFloat16: return "bfloat16";
    case at::kByte: return "uint8";
    default: return "another type";
  }
}

// The arguments of a call, taken one after the other.
class Args {
 public:
  Args(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : a_(a) {
    if (n != want) throw Refused{"expected " + std::to_string(want) + " arguments"};
    device_ = (int)integer("device");
    stream_ = reinterpret_cast<pqkv_stream_t>((uintptr_t)integer("stream"));
  }
  pqkv_stream_t stream() const { return stream_; }
  long long integer(const char* name) {
    const long long v = PyLong_AsLongLong(a_[i_++]);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused{std::string(name) + " must be an integer"};
    }
    return v;
  }
  int small(const char* name) {
    const long long v = integer(name);
    if (v < INT32_MIN || v > INT32_MAX) throw Refused{std::string(name) + " does not fit 32 bits"};
    return (int)v;
  }
  double number(const char* name) {
    const double v = PyFloat_AsDouble(a_[i_++]);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused{std::string(name) + " must be a number"};
    }
    return v;
  }
  bool none() const { return a_[i_] == Py_None; }
  void skip() { ++i_; }
  // bytes, or None and empty bytes as null
  const uint8_t* bytes(const char* name, Py_ssize_t& n) {
    PyObject* o = a_[i_++];
    n = 0;
    if (o == Py_None) return nullptr;
    if (!PyBytes_Check(o)) throw Refused{std::string(name) + " must be bytes"};
    n = PyBytes_GET_SIZE(o);
    return n ? reinterpret_cast<const uint8_t*>(PyBytes_AS_STRING(o)) : nullptr;
  }
  const at::Tensor& tensor(const char* name, at::ScalarType type, bool contiguous = true) {
    const at::Tensor& t = any(name);
    if (t.scalar_type() != type) throw Refused{std::string(name) + " must be " + type_name(type)};
    if (contiguous && !t.is_contiguous()) throw Refused{std::string(name) + " must be contiguous"};
    return t;
  }
  // the queries, whose type the other operands share
  const at::Tensor& tensor16(const char* name) {
    const at::Tensor& t = any(name);
    if (t.scalar_type() != at::kHalf && t.scalar_type() != at::kBFloat16)
      throw Refused{std::string(name) + " must be float16 or bfloat16"};
    return t;
  }

 private:
  const at::Tensor& any(const char* name) {
    PyObject* o = a_[i_++];
    if (!THPVariable_Check(o)) throw Refused{std::string(name) + " must be a tensor"};
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != device_)
      throw Refused{std::string(name) + " must be a tensor on cuda:" + std::to_string(device_)};
    return t;
  }
  PyObject* const* a_;
  Py_ssize_t i_ = 0;
  int device_ = 0;
  pqkv_stream_t stream_ = nullptr;
};

void need(bool ok, const char* why) {
  if (!ok) throw Refused{why};
}

int32_t* i32(const at::Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }

// A count that the C ABI takes as an int.
int count(int64_t n, const char* why) {
  need(n <= INT32_MAX, why);
  return (int)n;
}

// Runs `body(args)` (which returns a status) with C++ errors turned into Python's.
template <typename Body>
PyObject* guarded(Body body) {
  try {
    return PyLong_FromLong(body());
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.why.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// The library call itself, without the interpreter's lock.
template <typename F, typename... A>
int launch(F f, A... a) {
  need(f != nullptr, "the library is not bound");
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = f(a...);
  Py_END_ALLOW_THREADS
  return st;
}

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> int {
    need(n == 5, "expected five addresses");
    void* f[5];
    for (int i = 0; i < 5; ++i) f[i] = PyLong_AsVoidPtr(a[i]);
    need(!PyErr_Occurred(), "addresses must be integers");
    f_build_batch = reinterpret_cast<decltype(f_build_batch)>(f[0]);
    f_qk_norm_rope = reinterpret_cast<decltype(f_qk_norm_rope)>(f[1]);
    f_qkv_norm_rope_write = reinterpret_cast<decltype(f_qkv_norm_rope_write)>(f[2]);
    f_paged_cross_attention = reinterpret_cast<decltype(f_paged_cross_attention)>(f[3]);
    f_cache_layout = reinterpret_cast<decltype(f_cache_layout)>(f[4]);
    return PQKV_OK;
  });
}

// device, stream, start_pos, num_new, new_block_ids, block_tables, num_blocks,
// slot_mapping, positions, cu_q_lens, seq_lens, err_flag
PyObject* build_batch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> int {
    Args x(a, n, 12);
    const at::Tensor& start = x.tensor("start_pos", at::kInt);
    const at::Tensor& num_new = x.tensor("num_new", at::kInt);
    const at::Tensor& ids = x.tensor("new_block_ids", at::kInt);
    const at::Tensor& tables = x.tensor("block_tables", at::kInt);
    const int num_blocks = x.small("num_blocks");
    const at::Tensor& slots = x.tensor("slot_mapping", at::kInt);
    const at::Tensor& positions = x.tensor("positions", at::kInt);
    const at::Tensor& cu = x.tensor("cu_q_lens", at::kInt);
    const at::Tensor& lens = x.tensor("seq_lens", at::kInt);
    const at::Tensor& err = x.tensor("err_flag", at::kInt);
    const int B = count(start.numel(), "too many requests");
    need(num_new.numel() == B && lens.numel() == B && cu.numel() == (int64_t)B + 1,
         "num_new and seq_lens must be [B], cu_q_lens [B + 1]");
    need(tables.dim() == 2 && tables.size(0) == B, "block_tables must be int32 [B][max_blocks_per_seq]");
    need(positions.numel() == slots.numel(), "positions and slot_mapping must be of one size");
    need(err.numel() >= 1, "err_flag must be int32 [1]");
    return launch(f_build_batch, i32(start), i32(num_new), B, i32(ids), count(ids.numel(), "too many block ids"),
                  i32(tables), count(tables.size(1), "too many blocks per sequence"), num_blocks,
                  count(slots.numel(), "too many tokens"), i32(slots), i32(positions), i32(cu), i32(lens), i32(err),
                  x.stream());
  });
}

// [T][heads][D] rows whose heads are contiguous within a token.
struct Heads {
  const void* p = nullptr;
  int heads = 0;
  int64_t stride = 0;
};

Heads heads_of(const at::Tensor& t, const char* name, int64_t T, int64_t D) {
  Heads h;
  if (t.dim() != 3 || t.size(0) != T || t.size(2) != D || t.stride(2) != 1 || (t.stride(1) != D && t.size(1) > 1))
    throw Refused{std::string(name) + " must be [T][heads][head_dim] with contiguous heads"};
  h.p = t.data_ptr();
  h.heads = count(t.size(1), "too many heads");
  h.stride = T > 1 ? t.stride(0) : t.size(1) * D;  // the stride of a dimension of one token means nothing
  return h;
}

// q_weight, k_weight, eps, positions, cos_sin, axis_of_pair, interleaved
struct Turn {
  const float *qw = nullptr, *kw = nullptr, *table = nullptr;
  const int32_t* positions = nullptr;
  const uint8_t* axis = nullptr;
  float eps = 0;
  int axes = 0, num_positions = 0, rot = 0, interleaved = 0;

  Turn(Args& x, int64_t T, int64_t D) {
    for (const float** w : {&qw, &kw}) {
      if (x.none()) {
        x.skip();
        continue;
      }
      const at::Tensor& t = x.tensor(w == &qw ? "q_weight" : "k_weight", at::kFloat);
      need(t.numel() == D, "q_weight and k_weight must be float32 [head_dim]");
      *w = static_cast<const float*>(t.data_ptr());
    }
    eps = (float)x.number("eps");
    const at::Tensor* pos = nullptr;
    if (x.none()) x.skip();
    else pos = &x.tensor("positions", at::kInt);
    const at::Tensor* tab = nullptr;
    if (x.none()) x.skip();
    else tab = &x.tensor("cos_sin", at::kFloat);
    Py_ssize_t n = 0;
    axis = x.bytes("axis_of_pair", n);
    interleaved = x.integer("interleaved") != 0;
    need(!tab || tab->dim() == 2, "cos_sin must be float32 [num_positions][rot_dim]");
    if (!tab || tab->size(1) == 0) {  // no rotation
      axis = nullptr;
      return;
    }
    rot = count(tab->size(1), "rot_dim does not fit 32 bits");
    num_positions = count(tab->size(0), "too many positions");
    table = static_cast<const float*>(tab->data_ptr());
    need(!axis || n == rot / 2, "axis_of_pair must hold rot_dim / 2 bytes");
    need(pos && (pos->dim() == 1 || pos->dim() == 2) && pos->size(-1) == T, "positions must be int32 [T] or [axes][T]");
    axes = pos->dim() == 2 ? count(pos->size(0), "too many axes") : 1;
    positions = i32(*pos);
  }
};

// device, stream, q, k, q_weight, k_weight, eps, positions, cos_sin,
// axis_of_pair, interleaved, q_out, k_out, err_flag
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> int {
    Args x(a, n, 14);
    const at::Tensor& q = x.tensor16("q");
    need(q.dim() == 3, "q must be [T][num_q_heads][head_dim]");
    const at::ScalarType type = q.scalar_type();
    const int64_t T = q.size(0), D = q.size(2);
    const at::Tensor* k = nullptr;
    if (x.none()) x.skip();
    else k = &x.tensor("k", type, false);
    const Turn turn(x, T, D);
    const at::Tensor& q_out = x.tensor("q_out", type);
    const at::Tensor* k_out = nullptr;
    if (x.none()) x.skip();
    else k_out = &x.tensor("k_out", type);
    const at::Tensor& err = x.tensor("err_flag", at::kInt);
    need(q_out.sizes() == q.sizes() && !k == !k_out && (!k || k_out->sizes() == k->sizes()),
         "q_out and k_out must match q and k");
    need(err.numel() >= 1, "err_flag must be int32 [1]");
    const Heads hq = heads_of(q, "q", T, D);
    const Heads hk = k ? heads_of(*k, "k", T, D) : Heads{};
    return launch(f_qk_norm_rope, hq.p, hk.p, type == at::kHalf ? PQKV_DTYPE_FP16 : PQKV_DTYPE_BF16,
                  count(T, "too many tokens"), hq.heads, hk.heads, count(D, "head_dim does not fit 32 bits"), hq.stride,
                  hk.stride, turn.qw, turn.kw, turn.eps, turn.positions, turn.axes, turn.axis, turn.table,
                  turn.num_positions, turn.rot, turn.interleaved, q_out.data_ptr(), k_out ? k_out->data_ptr() : nullptr,
                  i32(err), x.stream());
  });
}

// cache, scales, outliers_idx, outliers_val (None where a format has none),
// kv_dtype, num_blocks, num_kv_heads, head_dim: the kernels go by these numbers,
// so each array must hold what they make of it
struct CacheArgs {
  void* arrays[4] = {nullptr, nullptr, nullptr, nullptr};
  int kv_dtype, num_blocks, heads, D;
  explicit CacheArgs(Args& x) {
    const char* names[4] = {"cache", "scales", "outliers_idx", "outliers_val"};
    const at::Tensor* given[4] = {nullptr, nullptr, nullptr, nullptr};
    for (int i = 0; i < 4; ++i) {
      if (x.none()) x.skip();
      else given[i] = &x.tensor(names[i], at::kByte);
    }
    kv_dtype = x.small("kv_dtype");
    num_blocks = x.small("num_blocks");
    heads = x.small("num_kv_heads");
    D = x.small("head_dim");
    need(f_cache_layout != nullptr, "the library is not bound");
    size_t bytes[4] = {0, 0, 0, 0};
    f_cache_layout(kv_dtype, num_blocks, heads, D, bytes);  // numbers that it refuses, the call itself refuses
    for (int i = 0; i < 4; ++i) {
      if (!given[i]) continue;
      if ((size_t)given[i]->numel() < bytes[i])
        throw Refused{std::string(names[i]) + " must have at least " + std::to_string(bytes[i]) +
                      " bytes for this num_blocks, num_kv_heads and head_dim"};
      arrays[i] = given[i]->data_ptr();
    }
  }
};

// device, stream, q, k, v, q_weight, k_weight, eps, positions, cos_sin,
// axis_of_pair, interleaved, q_out, slot_mapping, cache ... head_dim, err_flag
PyObject* qkv_norm_rope_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> int {
    Args x(a, n, 23);
    const at::Tensor& q = x.tensor16("q");
    need(q.dim() == 3, "q must be [T][num_q_heads][head_dim]");
    const at::ScalarType type = q.scalar_type();
    const int64_t T = q.size(0), D = q.size(2);
    const at::Tensor& k = x.tensor("k", type, false);
    const at::Tensor& v = x.tensor("v", type, false);
    const Turn turn(x, T, D);
    const at::Tensor& q_out = x.tensor("q_out", type);
    const at::Tensor& slots = x.tensor("slot_mapping", at::kInt);
    const CacheArgs c(x);
    const at::Tensor& err = x.tensor("err_flag", at::kInt);
    need(q_out.sizes() == q.sizes(), "q_out must match q");
    need(slots.numel() == T, "slot_mapping must be int32 [T]");
    need(err.numel() >= 1, "err_flag must be int32 [1]");
    const Heads hq = heads_of(q, "q", T, D), hk = heads_of(k, "k", T, D), hv = heads_of(v, "v", T, D);
    need(hk.heads == c.heads && hv.heads == c.heads && D == c.D, "k and v must be [T][num_kv_heads][head_dim]");
    return launch(f_qkv_norm_rope_write, hq.p, hk.p, hv.p, type == at::kHalf ? PQKV_DTYPE_FP16 : PQKV_DTYPE_BF16,
                  count(T, "too many tokens"), hq.heads, hk.heads, c.D, hq.stride, hk.stride, hv.stride, turn.qw,
                  turn.kw, turn.eps, turn.positions, turn.axes, turn.axis, turn.table, turn.num_positions, turn.rot,
                  turn.interleaved, q_out.data_ptr(), i32(slots), c.arrays[0], c.arrays[1], c.arrays[2], c.arrays[3],
                  c.kv_dtype, c.num_blocks, i32(err), x.stream());
  });
}

// device, stream, q, cu_q_lens, max_q_len, cache ... head_dim, block_tables,
// kv_lens, kv_ranges, scale, out, err_flag
PyObject* paged_cross_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> int {
    Args x(a, n, 19);
    const at::Tensor& q = x.tensor16("q");
    const at::ScalarType type = q.scalar_type();
    const at::Tensor& cu = x.tensor("cu_q_lens", at::kInt);
    const int max_q_len = x.small("max_q_len");
    const CacheArgs c(x);
    const at::Tensor& tables = x.tensor("block_tables", at::kInt);
    const at::Tensor& lens = x.tensor("kv_lens", at::kInt);
    const at::Tensor* ranges = nullptr;
    if (x.none()) x.skip();
    else ranges = &x.tensor("kv_ranges", at::kInt);
    const float scale = (float)x.number("scale");
    const at::Tensor& out = x.tensor("out", type);
    const at::Tensor& err = x.tensor("err_flag", at::kInt);
    need(q.dim() == 3 && q.is_contiguous() && q.size(2) == c.D && out.sizes() == q.sizes(),
         "q must be [T][num_q_heads][head_dim], contiguous and of the cache's head_dim, and out match it");
    const int B = count(lens.numel(), "too many sequences");
    need(cu.numel() == (int64_t)B + 1, "cu_q_lens must be int32 [B + 1]");
    need(tables.dim() == 2 && tables.size(0) == B, "block_tables must be int32 [B][max_blocks_per_seq]");
    need(!ranges || (ranges->dim() == 2 && ranges->size(0) == q.size(0) && ranges->size(1) == 2),
         "kv_ranges must be int32 [T][2]");
    need(err.numel() >= 1, "err_flag must be int32 [1]");
    if (q.size(0) == 0) return PQKV_OK;
    return launch(f_paged_cross_attention, q.data_ptr(), type == at::kHalf ? PQKV_DTYPE_FP16 : PQKV_DTYPE_BF16, B,
                  max_q_len, count(q.size(1), "too many heads"), i32(cu), c.arrays[0], c.arrays[1], c.arrays[2],
                  c.arrays[3], c.kv_dtype, c.num_blocks, c.heads, c.D, i32(tables),
                  count(tables.size(1), "too many blocks per sequence"), i32(lens), ranges ? i32(*ranges) : nullptr,
                  scale, out.data_ptr(), i32(err), x.stream());
  });
}

#define PQKV_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PQKV_METHOD(bind),
                         PQKV_METHOD(build_batch),
                         PQKV_METHOD(qk_norm_rope),
                         PQKV_METHOD(qkv_norm_rope_write),
                         PQKV_METHOD(paged_cross_attention),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// BUILT_FOR: the Python and torch whose headers this was compiled against; the
// package refuses a module that is not for the running ones.
PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "BUILT_FOR", PQKV_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
