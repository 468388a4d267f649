// binding.cpp -- marshals the windowed-attention, page and serving-step calls between PyTorch
// tensors and the C ABI of libattn.so (include/attn.h): checks, outputs and
// workspaces, the current stream, and errors.  Nothing is computed here.
//
// These calls are often a few microseconds of GPU work, and the same marshalling
// in Python costs more than that (one windowed prefill call of a 128-row prompt:
// 16 us on the host in Python and 4.3 us on the GPU).  The package's Python
// functions document the calls and pass their arguments on.
#include <Python.h>

#include <ATen/core/DimVector.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <string>

#include "../../include/attn.h"

namespace {

using at::Tensor;

PyObject* g_attn_error = nullptr;  // the package's AttnError

struct Refused {  // becomes a ValueError
  std::string what;
};
struct Failed {  // becomes an AttnError
  int status;
  const char* what;
};
struct PythonError {};  // a Python exception is set already

[[noreturn]] void refuse(std::string what) { throw Refused{std::move(what)}; }

void raise_if(int status, const char* what) {
  if (status != ATTN_OK) throw Failed{status, what};
}

// ------------------------------------------------------------------ arguments
const Tensor& tensor(PyObject* obj, const char* name) {
  if (!THPVariable_Check(obj)) refuse(std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(obj);
}

void check(const Tensor& t, const char* name, at::ScalarType type, const char* type_name, int ndim,
           at::Device device) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  if (t.scalar_type() != type)
    refuse(std::string(name) + " must be " + type_name + ", got " + c10::toString(t.scalar_type()));
  if (t.dim() != ndim)
    refuse(std::string(name) + " must have " + std::to_string(ndim) + " dims, got " +
           std::to_string(t.dim()));
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  if (t.device() != device) refuse(std::string(name) + " must be on " + device.str());
}

const Tensor& bf16(PyObject* obj, const char* name, int ndim, const Tensor* like = nullptr) {
  const Tensor& t = tensor(obj, name);
  check(t, name, at::kBFloat16, "bfloat16", ndim, like != nullptr ? like->device() : t.device());
  return t;
}

std::string shape_string(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i)
    s += (i ? ", " : "") + (shape[i] < 0 ? std::string("any") : std::to_string(shape[i]));
  return s + ")";
}

// shape: -1 is any size.
void check_shape(const Tensor& t, const char* name, at::IntArrayRef shape) {
  bool same = t.dim() == static_cast<int64_t>(shape.size());
  for (size_t i = 0; same && i < shape.size(); ++i) same = shape[i] < 0 || shape[i] == t.size(i);
  if (!same)
    refuse(std::string(name) + " must have shape " + shape_string(shape) + ", got " +
           shape_string(t.sizes()));
}

const Tensor& int32(PyObject* obj, const char* name, at::IntArrayRef shape, at::Device device) {
  const Tensor& t = tensor(obj, name);
  check(t, name, at::kInt, "int32", static_cast<int>(shape.size()), device);
  check_shape(t, name, shape);
  return t;
}

// An uninitialised tensor, straight from the CUDA allocator (at::empty's dispatch
// costs as much again as the allocation).
Tensor fresh(at::IntArrayRef shape, at::ScalarType type, at::Device device) {
  return at::detail::empty_cuda(shape, type, device, std::nullopt);
}

// The output that the caller gave, or a new one from get().
class Output {
 public:
  Output(PyObject* given, at::IntArrayRef shape, at::ScalarType type, const char* type_name,
         at::Device device, const char* name)
      : shape_(shape.begin(), shape.end()), type_(type), device_(device) {
    if (given == Py_None) return;
    given_ = &tensor(given, name);
    check(*given_, name, type, type_name, static_cast<int>(shape.size()), device);
    check_shape(*given_, name, shape);
  }
  bool given() const { return given_ != nullptr; }
  Tensor get() const { return given_ != nullptr ? *given_ : fresh(shape_, type_, device_); }

 private:
  const Tensor* given_ = nullptr;
  at::DimVector shape_;
  at::ScalarType type_;
  at::Device device_;
};
Output output_bf16(PyObject* given, at::IntArrayRef shape, at::Device device, const char* name) {
  return Output(given, shape, at::kBFloat16, "bfloat16", device, name);
}
Output output_f32(PyObject* given, at::IntArrayRef shape, at::Device device, const char* name) {
  return Output(given, shape, at::kFloat, "float32", device, name);
}
Output output_int32(PyObject* given, at::IntArrayRef shape, at::Device device, const char* name) {
  return Output(given, shape, at::kInt, "int32", device, name);
}
Tensor new_int32(int64_t n, at::Device device) {
  return fresh({n}, at::kInt, device);
}

int64_t padded(int64_t n) { return (n + 3) / 4 * 4; }  // to 16 bytes of int32

// Tensors that share one allocation of int32: an allocation and its tensor cost
// over a microsecond each, a further tensor on its storage a tenth of that.  Each begins
// at a multiple of 16 bytes, for the vector accesses of the calls that take it next.
class Carver {
 public:
  Carver(int64_t n, at::Device device) : all_(new_int32(n, device)) {}
  Tensor take(at::IntArrayRef shape) {
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(
        c10::Storage(all_.storage()), c10::DispatchKeySet(c10::DispatchKey::CUDA), all_.dtype());
    t.unsafeGetTensorImpl()->set_storage_offset(at_);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    at_ += padded(t.numel());
    return t;
  }

 private:
  Tensor all_;
  int64_t at_ = 0;
};

// An integer in [least, most]; larger ones (all keys, all room) become `most`.  Without
// a least one the C ABI refuses what is too low: any number below int's is as low.
constexpr long long kAny = LLONG_MIN;
int integer(PyObject* obj, const char* name, long long least, long long most) {
  PyObject* index = PyNumber_Index(obj);
  if (index == nullptr) throw PythonError{};
  int overflow = 0;
  long long x = PyLong_AsLongLongAndOverflow(index, &overflow);
  Py_DECREF(index);
  if (overflow != 0) x = overflow > 0 ? LLONG_MAX : LLONG_MIN;
  if (x < least) refuse(std::string(name) + " must be at least " + std::to_string(least));
  return static_cast<int>(std::max<long long>(std::min(x, most), INT_MIN));
}

constexpr long long kAll = 1ll << 30;  // beyond every sequence

float scale_of(PyObject* obj, int64_t D) {
  if (obj == Py_None) return static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
  const double x = PyFloat_AsDouble(obj);
  if (x == -1.0 && PyErr_Occurred()) throw PythonError{};
  return static_cast<float>(x);
}

// A size as the C ABI's int.
int size_int(int64_t n, const char* name) {
  if (n > INT_MAX) refuse(std::string(name) + " is too large");
  return static_cast<int>(n);
}

struct Sizes {
  int B, Hq, Hkv, Sq, Sk, D;
};
Sizes sizes_of(const Tensor& q, const Tensor& k, const Tensor& v) {
  if (k.size(0) != q.size(0) || k.size(3) != q.size(3) || v.sizes() != k.sizes())
    refuse("q/k/v shape mismatch");
  return {size_int(q.size(0), "q"), size_int(q.size(1), "q"), size_int(k.size(1), "k"),
          size_int(q.size(2), "q"), size_int(k.size(2), "k"), size_int(q.size(3), "q")};
}

void* current_stream(at::Device device) {
  return static_cast<void*>(c10::cuda::getCurrentCUDAStream(device.index()).stream());
}

int* ints(const Tensor& t) { return t.numel() > 0 ? static_cast<int*>(t.data_ptr()) : nullptr; }
float* floats(const Tensor& t) { return static_cast<float*>(t.data_ptr()); }

// The GPU part of a call, without Python's lock: allocations and launches can wait for
// the GPU (a full launch queue, a pool that has to grow), other threads go on meanwhile,
// and a host function in a stream that takes the lock cannot be waited for by its holder.
// No Python object is touched in it.
class GpuPart {
 public:
  explicit GpuPart(at::Device device) : lock_(PyEval_SaveThread()), guard_(device) {}
  GpuPart(const GpuPart&) = delete;

 private:
  struct Lock {
    explicit Lock(PyThreadState* state) : state(state) {}
    ~Lock() { PyEval_RestoreThread(state); }
    PyThreadState* state;
  } lock_;
  c10::cuda::CUDAGuard guard_;
};

// ------------------------------------------------------------------ results
PyObject* pack(std::initializer_list<Tensor> tensors) {
  PyObject* tuple = PyTuple_New(static_cast<Py_ssize_t>(tensors.size()));
  if (tuple == nullptr) throw PythonError{};
  Py_ssize_t i = 0;
  for (const Tensor& t : tensors) {
    PyObject* obj = THPVariable_Wrap(t);
    if (obj == nullptr) {
      Py_DECREF(tuple);
      throw PythonError{};
    }
    PyTuple_SET_ITEM(tuple, i++, obj);
  }
  return tuple;
}

PyObject* pack_one(const Tensor& t) {
  PyObject* obj = THPVariable_Wrap(t);
  if (obj == nullptr) throw PythonError{};
  return obj;
}

// One call: `n` positional arguments, exceptions turned into Python's.
template <typename F>
PyObject* call(Py_ssize_t given, Py_ssize_t n, F body) {
  HANDLE_TH_ERRORS
  if (given != n) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", n, given);
    return nullptr;
  }
  try {
    return body();
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const Failed& e) {
    PyObject* exc = PyObject_CallFunction(g_attn_error, "is", e.status, e.what);
    if (exc != nullptr) {
      PyErr_SetObject(g_attn_error, exc);
      Py_DECREF(exc);
    }
  } catch (const PythonError&) {
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ attention
// q, k, v, window, sinks, scale, o, lse, num_splits
PyObject* window_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 9, [&] {
    const Tensor& q = bf16(a[0], "q", 4);
    const Tensor &k = bf16(a[1], "k", 4, &q), &v = bf16(a[2], "v", 4, &q);
    const Sizes s = sizes_of(q, k, v);
    const int window = integer(a[3], "window", 1, kAll), sinks = integer(a[4], "sinks", 0, kAll);
    const float scale = scale_of(a[5], s.D);
    const Output o_out = output_bf16(a[6], q.sizes(), q.device(), "o");
    const Output lse_out = output_f32(a[7], {s.B, s.Hq, s.Sq}, q.device(), "lse");
    const bool pick = a[8] == Py_None;
    int splits = pick ? 0 : integer(a[8], "num_splits", kAny, INT_MAX);
    Tensor o, lse;
    {
      const GpuPart gpu(q.device());
      if (pick)
        raise_if(attn_window_fwd_num_splits(s.B, s.Hq, s.Hkv, s.Sq, s.Sk, s.D, window, sinks, &splits),
                 "attn_window_fwd_num_splits");
      o = o_out.get();
      lse = lse_out.get();
      Tensor ws;
      if (splits > 1 && splits <= (static_cast<int64_t>(s.Sk) + 127) / 128) {  // (more are refused below)
        long long need = 0;
        raise_if(attn_window_fwd_workspace(s.B, s.Hq, s.Hkv, s.Sq, s.D, splits, &need),
                 "attn_window_fwd");
        ws = fresh({std::max(need, 1ll)}, at::kFloat, q.device());  // full rounds need none
      }
      raise_if(attn_window_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), floats(lse),
                               ws.defined() ? floats(ws) : nullptr, s.B, s.Hq, s.Hkv, s.Sq, s.Sk,
                               s.D, window, sinks, splits, scale, current_stream(q.device())),
               "attn_window_fwd");
    }
    return pack({o, lse});
  });
}

// q, k, v, o, lse, dout, window, sinks, scale, dq, dk, dv, workspace
PyObject* window_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 13, [&] {
    const Tensor& q = bf16(a[0], "q", 4);
    const Tensor &k = bf16(a[1], "k", 4, &q), &v = bf16(a[2], "v", 4, &q);
    const Tensor &o = bf16(a[3], "o", 4, &q), &dout = bf16(a[5], "dout", 4, &q);
    const Sizes s = sizes_of(q, k, v);
    check_shape(o, "o", q.sizes());
    check_shape(dout, "dout", q.sizes());
    const Tensor& lse = tensor(a[4], "lse");
    check(lse, "lse", at::kFloat, "float32", 3, q.device());
    check_shape(lse, "lse", {s.B, s.Hq, s.Sq});
    const int window = integer(a[6], "window", 1, kAll), sinks = integer(a[7], "sinks", 0, kAll);
    const float scale = scale_of(a[8], s.D);
    const Output dq_out = output_bf16(a[9], q.sizes(), q.device(), "dq");
    const Output dk_out = output_bf16(a[10], k.sizes(), q.device(), "dk");
    const Output dv_out = output_bf16(a[11], k.sizes(), q.device(), "dv");
    Tensor ws;
    if (a[12] != Py_None) {
      ws = tensor(a[12], "workspace");
      check(ws, "workspace", at::kFloat, "float32", static_cast<int>(ws.dim()), q.device());
    }
    Tensor dq, dk, dv;
    {
      const GpuPart gpu(q.device());
      long long need = 0;
      raise_if(attn_window_bwd_workspace(s.B, s.Hq, s.Hkv, s.Sq, s.Sk, s.D, window, sinks, &need),
               "attn_window_bwd_workspace");
      if (ws.defined() && ws.numel() < need)
        refuse("workspace must have at least " + std::to_string(need) + " entries");
      dq = dq_out.get();
      dk = dk_out.get();
      dv = dv_out.get();
      if (!ws.defined()) ws = fresh({need}, at::kFloat, q.device());
      raise_if(attn_window_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), floats(lse),
                               dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                               floats(ws), s.B, s.Hq, s.Hkv, s.Sq, s.Sk, s.D, window, sinks, scale,
                               current_stream(q.device())),
               "attn_window_bwd");
    }
    return pack({dq, dk, dv});
  });
}

// The cache of a decode: Sk its capacity in keys; table and page size when paged.
struct Cache {
  const Tensor &k, &v;
  const Tensor* table;
  int Hkv, Sk;
};

// a: seqlens, window, sinks, num_splits, scale, o, lse
PyObject* decode(const Tensor& q, const Cache& c, PyObject* const* a, const char* what) {
  if (q.size(2) != 1) refuse("decode takes one query row per head (q.shape[2] == 1)");
  const int B = size_int(q.size(0), "q"), Hq = size_int(q.size(1), "q"),
            D = size_int(q.size(3), "q");
  const at::Device device = q.device();
  const int* seqlens = a[0] == Py_None ? nullptr : ints(int32(a[0], "seqlens", {B}, device));
  const int window = integer(a[1], "window", 1, kAll), sinks = integer(a[2], "sinks", 0, kAll);
  const float scale = scale_of(a[4], D);
  const bool pick = a[3] == Py_None;
  int splits = pick ? 0 : integer(a[3], "num_splits", kAny, INT_MAX);
  const Output o_out = output_bf16(a[5], {B, Hq, D}, device, "o");
  const Output lse_out = output_f32(a[6], {B, Hq}, device, "lse");
  Tensor o, lse;
  {
    const GpuPart gpu(device);
    if (pick)
      raise_if(attn_decode_window_num_splits(B, Hq, c.Hkv, c.Sk, D, window, sinks, &splits),
               "attn_decode_window_num_splits");
    o = o_out.get();
    lse = lse_out.get();
    if (c.table == nullptr)
      raise_if(attn_decode_window(q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), seqlens,
                                  o.data_ptr(), floats(lse), B, Hq, c.Hkv, c.Sk, D, window, sinks,
                                  splits, scale, current_stream(device)),
               what);
    else
      raise_if(attn_decode_window_paged(
                   q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), ints(*c.table), seqlens,
                   o.data_ptr(), floats(lse), B, Hq, c.Hkv, size_int(c.k.size(0), "k_cache"),
                   size_int(c.k.size(2), "k_cache"), size_int(c.table->size(1), "block_table"), D,
                   window, sinks, splits, scale, current_stream(device)),
               what);
  }
  return pack({o, lse});
}

// q, k, v, then decode's
PyObject* decode_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 10, [&] {
    const Tensor& q = bf16(a[0], "q", 4);
    const Tensor &k = bf16(a[1], "k", 4, &q), &v = bf16(a[2], "v", 4, &q);
    const Sizes s = sizes_of(q, k, v);
    return decode(q, {k, v, nullptr, s.Hkv, s.Sk}, a + 3, "attn_decode_window");
  });
}

// q, k_cache, v_cache, block_table, then decode's
PyObject* decode_window_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 11, [&] {
    const Tensor& q = bf16(a[0], "q", 4);
    const Tensor &k = bf16(a[1], "k_cache", 4, &q), &v = bf16(a[2], "v_cache", 4, &q);
    if (k.size(3) != q.size(3) || v.sizes() != k.sizes()) refuse("q/cache shape mismatch");
    const Tensor& table = int32(a[3], "block_table", {q.size(0), -1}, q.device());
    if (a[4] == Py_None) refuse("a paged cache needs seqlens");
    const int64_t capacity = table.size(1) * k.size(2);
    return decode(q, {k, v, &table, size_int(k.size(1), "k_cache"),
                      static_cast<int>(std::min<int64_t>(capacity, INT_MAX))},
                  a + 4, "attn_decode_window_paged");
  });
}

// ------------------------------------------------------------------ pages
struct Pages {
  const Tensor &table, &refs;
  int B, M, P;
  at::Device device;
};
Pages pages_of(PyObject* table_obj, PyObject* refs_obj) {
  const Tensor& table = tensor(table_obj, "block_table");
  check(table, "block_table", at::kInt, "int32", 2, table.device());
  const Tensor& refs = int32(refs_obj, "refs", {-1}, table.device());
  return {table,
          refs,
          size_int(table.size(0), "block_table"),
          size_int(table.size(1), "block_table"),
          size_int(refs.size(0), "refs"),
          table.device()};
}

// block_table, refs, seqlens, page_size, window, sinks, room, block_table_out, refs_out
PyObject* pages_free(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 9, [&] {
    const Pages p = pages_of(a[0], a[1]);
    const Tensor& lens = int32(a[2], "seqlens", {p.B}, p.device);
    const int page = integer(a[3], "page_size", kAny, INT_MAX);
    const int window = a[4] == Py_None ? static_cast<int>(kAll) : integer(a[4], "window", 1, kAll);
    const int sinks = integer(a[5], "sinks", 0, kAll), room = integer(a[6], "room", 0, kAll);
    const Output table_out = output_int32(a[7], {p.B, p.M}, p.device, "block_table_out");
    const Output refs_out = output_int32(a[8], {p.P}, p.device, "refs_out");
    Tensor table, refs;
    {
      const GpuPart gpu(p.device);
      if (!table_out.given() && !refs_out.given()) {
        Carver results(padded(static_cast<int64_t>(p.B) * p.M) + p.P, p.device);
        table = results.take({p.B, p.M});
        refs = results.take({p.P});
      } else {
        table = table_out.get();
        refs = refs_out.get();
      }
      raise_if(attn_pages_free(ints(p.table), ints(p.refs), ints(lens), ints(table), ints(refs), p.B,
                               p.M, p.P, page, window, sinks, room, current_stream(p.device)),
               "attn_pages_free");
    }
    return pack({table, refs});
  });
}

Tensor pages_workspace(const Pages& p, int rows) {
  long long n = 0;
  raise_if(attn_pages_workspace(p.P, rows, &n), "attn_pages_workspace");
  return new_int32(n, p.device);
}

// block_table, refs, seqlens, parents, page_size, room
PyObject* pages_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 6, [&] {
    const Pages p = pages_of(a[0], a[1]);
    const Tensor& lens = int32(a[2], "seqlens", {p.B}, p.device);
    const Tensor& parents = int32(a[3], "parents", {-1}, p.device);
    const int R = size_int(parents.size(0), "parents");
    const int page = integer(a[4], "page_size", kAny, INT_MAX);
    const int room = integer(a[5], "room", 0, kAll);
    Tensor table, refs, lens_out, src, dst, counts;
    {
      const GpuPart gpu(p.device);
      Tensor ws = pages_workspace(p, R);
      Carver results(padded(static_cast<int64_t>(R) * p.M) + padded(p.P) + 3 * padded(R) + 2, p.device);
      table = results.take({R, p.M});
      refs = results.take({p.P});
      lens_out = results.take({R});
      src = results.take({R});
      dst = results.take({R});
      counts = results.take({2});
      raise_if(attn_pages_fork(ints(p.table), ints(p.refs), ints(lens), ints(parents), ints(table),
                               ints(refs), ints(lens_out), ints(src), ints(dst), ints(counts),
                               ints(ws), p.B, R, p.M, p.P, page, room, current_stream(p.device)),
               "attn_pages_fork");
    }
    return pack({table, refs, lens_out, src, dst, counts});
  });
}

// block_table, refs
PyObject* pages_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 2, [&] {
    const Pages p = pages_of(a[0], a[1]);
    Tensor table, refs, src, dst, live;
    {
      const GpuPart gpu(p.device);
      Tensor ws = pages_workspace(p, 0);
      Carver results(padded(static_cast<int64_t>(p.B) * p.M) + padded(p.P) + 2 * padded(p.P / 2) + 1,
                     p.device);
      table = results.take({p.B, p.M});
      refs = results.take({p.P});
      src = results.take({p.P / 2});
      dst = results.take({p.P / 2});
      live = results.take({1});
      raise_if(attn_pages_compact(ints(p.table), ints(p.refs), ints(table), ints(refs), ints(src),
                                  ints(dst), ints(live), ints(ws), p.B, p.M, p.P,
                                  current_stream(p.device)),
               "attn_pages_compact");
    }
    return pack({table, refs, src, dst, live});
  });
}

// k_cache, v_cache, src, dst
PyObject* pages_copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 4, [&]() -> PyObject* {
    const Tensor &k = tensor(a[0], "k_cache"), &v = tensor(a[1], "v_cache");
    for (const Tensor* t : {&k, &v})
      if (!t->is_cuda() || !t->is_contiguous() || t->dim() < 2 || t->numel() == 0)
        refuse("the caches must be contiguous CUDA tensors [num_pages, ...]");
    if (k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type() || k.device() != v.device())
      refuse("the caches must have one shape, type and device");
    const Tensor& src = int32(a[2], "src", {-1}, k.device());
    const Tensor& dst = int32(a[3], "dst", {src.size(0)}, k.device());
    const long long page_bytes = k.numel() / k.size(0) * k.element_size();
    {
      const GpuPart gpu(k.device());
      raise_if(attn_pages_copy(k.data_ptr(), v.data_ptr(), ints(src), ints(dst),
                               size_int(src.size(0), "src"), size_int(k.size(0), "k_cache"),
                               page_bytes, current_stream(k.device())),
               "attn_pages_copy");
    }
    Py_RETURN_NONE;
  });
}

// ------------------------------------------------------------------ a serving step
// block_table, refs, seqlens, new_lens, tokens, page_size, block_table_out, refs_out,
// seqlens_out
PyObject* pages_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 9, [&] {
    const Pages p = pages_of(a[0], a[1]);
    const Tensor& lens = int32(a[2], "seqlens", {p.B}, p.device);
    const Tensor& news = int32(a[3], "new_lens", {p.B}, p.device);
    const int T = integer(a[4], "tokens", 1, INT_MAX);
    const int page = integer(a[5], "page_size", kAny, INT_MAX);
    const Output table_out = output_int32(a[6], {p.B, p.M}, p.device, "block_table_out");
    const Output refs_out = output_int32(a[7], {p.P}, p.device, "refs_out");
    const Output lens_out = output_int32(a[8], {p.B}, p.device, "seqlens_out");
    if (T > kAll) throw Failed{ATTN_ERR_UNSUPPORTED, "attn_pages_append"};
    Tensor table, refs, lens_new, cu, positions, slots, counts;
    {
      const GpuPart gpu(p.device);
      long long need = 0;
      raise_if(attn_pages_append_workspace(p.P, p.B, &need), "attn_pages_append");
      // (The workspace too is of the results' allocation: one allocation is what the call costs
      // the host.)
      Carver results((table_out.given() ? 0 : padded(static_cast<int64_t>(p.B) * p.M)) +
                         (refs_out.given() ? 0 : padded(p.P)) + (lens_out.given() ? 0 : padded(p.B)) +
                         padded(static_cast<int64_t>(p.B) + 1) + 2 * padded(T) + 4 + need,
                     p.device);
      table = table_out.given() ? table_out.get() : results.take({p.B, p.M});
      refs = refs_out.given() ? refs_out.get() : results.take({p.P});
      lens_new = lens_out.given() ? lens_out.get() : results.take({p.B});
      cu = results.take({static_cast<int64_t>(p.B) + 1});
      positions = results.take({T});
      slots = results.take({T});
      counts = results.take({2});
      const Tensor ws = results.take({need});
      raise_if(attn_pages_append(ints(p.table), ints(p.refs), ints(lens), ints(news), ints(table),
                                 ints(refs), ints(lens_new), ints(cu), ints(positions), ints(slots),
                                 ints(counts), ints(ws), p.B, T, p.M, p.P, page,
                                 current_stream(p.device)),
               "attn_pages_append");
    }
    return pack({table, refs, lens_new, cu, positions, slots, counts});
  });
}

// Rows of bf16 heads: [..., N] whose last dim is contiguous and whose others are one run of
// rows, `ld` elements apart.
struct Rows {
  const Tensor& t;
  int64_t count, width;
  long long ld;
};
Rows rows_of(PyObject* obj, const char* name, int ndim, const Tensor* like = nullptr) {
  const Tensor& t = tensor(obj, name);
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  if (t.scalar_type() != at::kBFloat16)
    refuse(std::string(name) + " must be bfloat16, got " + c10::toString(t.scalar_type()));
  if (t.dim() != ndim)
    refuse(std::string(name) + " must have " + std::to_string(ndim) + " dims, got " +
           std::to_string(t.dim()));
  if (like != nullptr && t.device() != like->device())
    refuse(std::string(name) + " must be on " + like->device().str());
  const int64_t width = t.size(ndim - 1);
  int64_t count = 1;
  for (int i = 0; i + 1 < ndim; ++i) count *= t.size(i);
  // (The stride of a dim of size 1 means nothing.)
  long long ld = width;
  bool regular = t.numel() > 0 && (width == 1 || t.stride(ndim - 1) == 1);
  int64_t step = -1, above = 1;
  for (int i = ndim - 2; i >= 0 && regular; --i) {
    if (t.size(i) == 1) continue;
    if (step < 0) {
      step = t.stride(i) / above;
      regular = t.stride(i) % above == 0;
    }
    regular = regular && t.stride(i) == step * above;
    above *= t.size(i);
  }
  if (step >= 0) ld = step;
  if (!regular) refuse(std::string(name) + " must be rows of contiguous elements, equally far apart");
  return {t, count, width, ld};
}

// The table of attn_rope_table: [max_pos, R/2, 2].
struct RopeTable {
  const float* data;
  int max_pos, R;
};
RopeTable rope_table_of(PyObject* obj, at::Device device) {
  const Tensor& t = tensor(obj, "rope_table");
  check(t, "rope_table", at::kFloat, "float32", 3, device);
  if (t.size(2) != 2) refuse("rope_table must come from attn_rope_table");
  return {static_cast<const float*>(t.data_ptr()), size_int(t.size(0), "rope_table"),
          size_int(2 * t.size(1), "rope_table")};
}
const int* positions_of(PyObject* obj, int64_t count, at::Device device) {
  if (obj == Py_None) return nullptr;
  const Tensor& t = tensor(obj, "positions");
  check(t, "positions", at::kInt, "int32", static_cast<int>(t.dim()), device);
  if (t.numel() != count) refuse("positions must have " + std::to_string(count) + " entries");
  return static_cast<const int*>(t.data_ptr());
}

// qkv, rope_table, Hq, Hkv, positions, style, q, k, v
PyObject* rope_split(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 9, [&] {
    const Rows x = rows_of(a[0], "qkv", 3);
    const at::Device device = x.t.device();
    const RopeTable table = rope_table_of(a[1], device);
    const int Hq = integer(a[2], "Hq", 1, INT_MAX), Hkv = integer(a[3], "Hkv", 1, INT_MAX);
    const int* positions = positions_of(a[4], x.count, device);
    const int style = integer(a[5], "style", kAny, INT_MAX);
    const int64_t heads = static_cast<int64_t>(Hq) + 2ll * Hkv;
    if (x.width % heads != 0) refuse("qkv must have (Hq + 2 * Hkv) * D columns");
    const int64_t B = x.t.size(0), S = x.t.size(1), D = x.width / heads;
    const Output q_out = output_bf16(a[6], {B, Hq, S, D}, device, "q");
    const Output k_out = output_bf16(a[7], {B, Hkv, S, D}, device, "k");
    const Output v_out = output_bf16(a[8], {B, Hkv, S, D}, device, "v");
    Tensor q, k, v;
    {
      const GpuPart gpu(device);
      q = q_out.get();
      k = k_out.get();
      v = v_out.get();
      raise_if(attn_rope_split(x.t.data_ptr(), x.ld, table.data, positions, q.data_ptr(),
                               k.data_ptr(), v.data_ptr(), size_int(B, "qkv"), size_int(S, "qkv"),
                               Hq, Hkv, size_int(D, "qkv"), table.R, table.max_pos, style,
                               current_stream(device)),
               "attn_rope_split");
    }
    return pack({q, k, v});
  });
}

// dq, dk, dv, rope_table, positions, style, dqkv
PyObject* rope_split_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 7, [&] {
    const Tensor& dq = tensor(a[0], "dq");
    const at::Device device = dq.device();
    const bool fp32 = dq.scalar_type() == at::kFloat;
    const auto type = fp32 ? at::kFloat : at::kBFloat16;
    const char* type_name = fp32 ? "float32" : "bfloat16";
    check(dq, "dq", type, type_name, 4, device);
    const Tensor &dk = tensor(a[1], "dk"), &dv = tensor(a[2], "dv");
    check(dk, "dk", type, type_name, 4, device);
    check(dv, "dv", type, type_name, 4, device);
    if (dk.sizes() != dv.sizes() || dk.size(0) != dq.size(0) || dk.size(2) != dq.size(2) ||
        dk.size(3) != dq.size(3))
      refuse("dq/dk/dv shape mismatch");
    const RopeTable table = rope_table_of(a[3], device);
    const int64_t B = dq.size(0), Hq = dq.size(1), S = dq.size(2), D = dq.size(3), Hkv = dk.size(1);
    const int* positions = positions_of(a[4], B * S, device);
    const int style = integer(a[5], "style", kAny, INT_MAX);
    const int64_t N = (Hq + 2 * Hkv) * D;
    Tensor dqkv;
    long long ld = N;
    if (a[6] != Py_None) {
      const Rows y = rows_of(a[6], "dqkv", 3, &dq);
      check_shape(y.t, "dqkv", {B, S, N});
      dqkv = y.t;
      ld = y.ld;
    }
    {
      const GpuPart gpu(device);
      if (!dqkv.defined()) dqkv = fresh({B, S, N}, at::kBFloat16, device);
      raise_if(attn_rope_split_bwd(dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), fp32, table.data,
                                   positions, dqkv.data_ptr(), ld, size_int(B, "dq"),
                                   size_int(S, "dq"), size_int(Hq, "dq"), size_int(Hkv, "dk"),
                                   size_int(D, "dq"), table.R, table.max_pos, style,
                                   current_stream(device)),
               "attn_rope_split_bwd");
    }
    return pack_one(dqkv);
  });
}

// qkv, rope_table, positions, slots, k_cache, v_cache, Hq, style, q
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 9, [&] {
    const Rows x = rows_of(a[0], "qkv", 2);
    const at::Device device = x.t.device();
    const RopeTable table = rope_table_of(a[1], device);
    const Tensor& positions = int32(a[2], "positions", {x.count}, device);
    const Tensor& slots = int32(a[3], "slots", {x.count}, device);
    const Tensor &k = bf16(a[4], "k_cache", 4, &x.t), &v = bf16(a[5], "v_cache", 4, &x.t);
    if (k.sizes() != v.sizes()) refuse("the caches must have one shape");
    const int Hq = integer(a[6], "Hq", 1, INT_MAX), style = integer(a[7], "style", kAny, INT_MAX);
    const int64_t Hkv = k.size(1), D = k.size(3);
    if (x.width != (Hq + 2 * Hkv) * D) refuse("qkv must have (Hq + 2 * Hkv) * D columns");
    const Output q_out = output_bf16(a[8], {x.count, Hq, D}, device, "q");
    Tensor q;
    {
      const GpuPart gpu(device);
      q = q_out.get();
      raise_if(attn_rope_append(x.t.data_ptr(), x.ld, table.data, ints(positions), ints(slots),
                                q.data_ptr(), k.data_ptr(), v.data_ptr(), size_int(x.count, "qkv"),
                                Hq, size_int(Hkv, "k_cache"), size_int(D, "k_cache"), table.R,
                                table.max_pos, size_int(k.size(0), "k_cache"),
                                size_int(k.size(2), "k_cache"), style, current_stream(device)),
               "attn_rope_append");
    }
    return pack_one(q);
  });
}

// cu_tokens, seqlens, tokens, Hq, Hkv, D, max_keys, window, sinks, plan, slots
PyObject* chunk_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 11, [&] {
    const Tensor& lens = tensor(a[1], "seqlens");
    check(lens, "seqlens", at::kInt, "int32", 1, lens.device());
    const at::Device device = lens.device();
    const int B = size_int(lens.size(0), "seqlens");
    const Tensor& cu = int32(a[0], "cu_tokens", {static_cast<int64_t>(B) + 1}, device);
    const int T = integer(a[2], "tokens", kAny, INT_MAX), Hq = integer(a[3], "Hq", kAny, INT_MAX);
    const int Hkv = integer(a[4], "Hkv", kAny, INT_MAX), D = integer(a[5], "D", kAny, INT_MAX);
    const int max_keys = integer(a[6], "max_keys", kAny, INT_MAX);
    const int window = a[7] == Py_None ? static_cast<int>(kAll) : integer(a[7], "window", 1, kAll);
    const int sinks = integer(a[8], "sinks", 0, kAll);
    Tensor plan;
    if (a[9] != Py_None) plan = int32(a[9], "plan", {-1}, device);
    const bool has_slots = a[10] != Py_None;
    const int* slots = has_slots ? ints(int32(a[10], "slots", {T}, device)) : nullptr;
    {
      const GpuPart gpu(device);
      long long need = 0;
      raise_if(attn_chunk_plan_size(B, T, Hq, Hkv, D, &need), "attn_chunk_plan");
      if (plan.defined() && plan.numel() < need)
        refuse("plan must have at least " + std::to_string(need) + " entries");
      if (!plan.defined()) plan = new_int32(need, device);
      raise_if(has_slots ? attn_chunk_plan_slots(ints(cu), ints(lens), slots, ints(plan), B, T, Hq,
                                                 Hkv, D, max_keys, window, sinks,
                                                 current_stream(device))
                         : attn_chunk_plan(ints(cu), ints(lens), ints(plan), B, T, Hq, Hkv, D,
                                           max_keys, window, sinks, current_stream(device)),
               "attn_chunk_plan");
    }
    return pack_one(plan);
  });
}

// q, k_cache, v_cache, block_table, plan, scale, o, lse, workspace
PyObject* chunk_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 9, [&] {
    const Tensor& q = bf16(a[0], "q", 3);
    const Tensor &k = bf16(a[1], "k_cache", 4, &q), &v = bf16(a[2], "v_cache", 4, &q);
    if (k.size(3) != q.size(2) || v.sizes() != k.sizes()) refuse("q/cache shape mismatch");
    const at::Device device = q.device();
    const Tensor& table = int32(a[3], "block_table", {-1, -1}, device);
    const Tensor& plan = int32(a[4], "plan", {-1}, device);
    const int B = size_int(table.size(0), "block_table"), T = size_int(q.size(0), "q"),
              Hq = size_int(q.size(1), "q"), Hkv = size_int(k.size(1), "k_cache"),
              D = size_int(q.size(2), "q");
    const float scale = scale_of(a[5], D);
    const Output o_out = output_bf16(a[6], q.sizes(), device, "o");
    const Output lse_out = output_f32(a[7], {T, Hq}, device, "lse");
    Tensor ws;
    if (a[8] != Py_None) {
      ws = tensor(a[8], "workspace");
      check(ws, "workspace", at::kFloat, "float32", static_cast<int>(ws.dim()), device);
    }
    Tensor o, lse;
    {
      const GpuPart gpu(device);
      long long need = 0, entries = 0;
      raise_if(attn_chunk_plan_size(B, T, Hq, Hkv, D, &entries), "attn_chunk_paged");
      if (plan.numel() < entries) refuse("plan must come from attn_chunk_plan for these sizes");
      raise_if(attn_chunk_workspace(D, &need), "attn_chunk_paged");
      if (ws.defined() && ws.numel() < need)
        refuse("workspace must have at least " + std::to_string(need) + " entries");
      o = o_out.get();
      lse = lse_out.get();
      if (!ws.defined()) ws = fresh({need}, at::kFloat, device);
      raise_if(attn_chunk_paged(q.data_ptr(), k.data_ptr(), v.data_ptr(), ints(table), ints(plan),
                                o.data_ptr(), floats(lse), floats(ws), B, T, Hq, Hkv,
                                size_int(k.size(0), "k_cache"), size_int(k.size(2), "k_cache"),
                                size_int(table.size(1), "block_table"), D, scale,
                                current_stream(device)),
               "attn_chunk_paged");
    }
    return pack({o, lse});
  });
}

// attn_error: the exception class of failed calls, called with (status, what)
PyObject* setup(PyObject*, PyObject* attn_error) {
  Py_INCREF(attn_error);
  Py_XSETREF(g_attn_error, attn_error);
  Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {{"setup", setup, METH_O, nullptr},
                          FAST(window_fwd),
                          FAST(window_bwd),
                          FAST(decode_window),
                          FAST(decode_window_paged),
                          FAST(pages_free),
                          FAST(pages_fork),
                          FAST(pages_compact),
                          FAST(pages_copy),
                          FAST(pages_append),
                          FAST(rope_split),
                          FAST(rope_split_bwd),
                          FAST(rope_append),
                          FAST(chunk_plan),
                          FAST(chunk_paged),
                          {nullptr, nullptr, 0, nullptr}};
#undef FAST

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods,
                       nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&kModule); }
