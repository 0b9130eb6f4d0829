// Python calls of the operators whose kernels take a few microseconds
// (speculate.py; append and attention of attention.py), on torch tensors: checks,
// output tensors, the C ABI.  Written against the interpreter and torch's C++ side
// because through ctypes and torch's Python side a call's own cost was two to three
// times its kernel's (verification 16 us around 5, a step of the pool 23 around 10,
// the append of 64 tokens 15 around 4).
#include <ATen/core/Tensor.h>
#include <array>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/exl3.h"

namespace {

PyObject* g_error;  // _lib.Exl3Error

// Thrown where a Python exception has been set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* format, const char* name, const char* more = "") {
  PyErr_Format(type, format, name, more);
  throw Raised{};
}

// The device of a call: its cache's or pool's, else its first tensor's (-1: none yet).
thread_local int t_device;
// The tensors that a call was given.
thread_local std::array<const at::Tensor*, 16> t_given;
thread_local size_t t_count;

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) raise(PyExc_ValueError, "%s must be a CUDA tensor", name);
  if (t_device < 0) t_device = t.get_device();
  if (t.get_device() != t_device)
    raise(PyExc_ValueError, "%s is on another device than the rest of the call", name);
  t_given[t_count++] = &t;
  return t;
}
// A contiguous vector of n values (n < 0: any number).
const at::Tensor& vector(PyObject* o, const char* name, at::ScalarType type, int64_t n) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, "%s has another dtype than %s", name, c10::toString(type));
  if (t.dim() != 1 || (n >= 0 && t.size(0) != n))
    raise(PyExc_ValueError, "%s has the wrong shape", name);
  if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
  return t;
}
// The lengths of a step's n sequences, or none.
const int32_t* lens_of(PyObject* o, int64_t n) {
  return o == Py_None ? nullptr
                      : static_cast<const int32_t*>(vector(o, "step.seq_lens", at::kInt, n).data_ptr());
}
int64_t whole(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v;
}
template <class T>
T* address(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Raised{};
  return static_cast<T*>(p);
}

// The stream of a call: stream= (an object with a cuda_stream) or the device's
// current one.  Outputs are made on it, and are for use on the current one later;
// what the call was given stays its own until the stream is done with it.
// The tensors' device is the current one as long as it lives: a raw default stream
// is the current device's, whichever that is.
struct Stream {
  c10::cuda::OptionalCUDAGuard device;
  c10::cuda::CUDAStream current, launch;
  bool other;
  Stream(PyObject* given, const at::Tensor& t)
      : current(c10::cuda::getCurrentCUDAStream(t.get_device())), launch(current), other(false) {
    if (c10::cuda::current_device() != t.get_device()) device.set_index(t.get_device());
    if (given == Py_None) return;
    const auto tensors = t_given;  // (what Python runs below may make calls of its own)
    const size_t count = t_count;
    PyObject* raw = PyObject_GetAttrString(given, "cuda_stream");
    if (!raw) throw Raised{};
    const auto s = reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(raw));
    Py_DECREF(raw);
    if (PyErr_Occurred()) throw Raised{};
    launch = c10::cuda::getStreamFromExternal(s, t.get_device());
    other = s != current.stream();
    if (other)
      for (size_t i = 0; i < count; i++) tensors[i]->record_stream(launch);
  }
  // Small int32 tensors side by side in one allocation: each one's own costs as much
  // as the rest of a small call.  (Of one type: torch saves no two that share memory
  // as different ones.  Small: what is kept of them keeps all.)
  template <int N>
  std::array<at::Tensor, N> words(const at::IntArrayRef (&shapes)[N]) const {
    int64_t at[N], n = 0;
    for (int i = 0; i < N; i++) {
      at[i] = n;
      int64_t size = 1;
      for (const int64_t d : shapes[i]) size *= d;
      n += (size + 3) & ~(int64_t)3;  // 16 bytes aligned
    }
    const c10::Storage all = memory(4 * n);
    std::array<at::Tensor, N> r;
    for (int i = 0; i < N; i++) {
      r[i] = view(all, shapes[i], at::kInt);
      r[i].unsafeGetTensorImpl()->set_storage_offset(at[i]);
    }
    return r;
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    int64_t size = (int64_t)c10::elementSize(type);
    for (const int64_t d : shape) size *= d;
    return view(memory(size), shape, type);
  }

 private:
  // From torch's allocator as it is: at::empty takes as long again on the way to it.
  c10::Storage memory(int64_t bytes) const {
    c10::Allocator* const from = c10::cuda::CUDACachingAllocator::get();
    const auto make = [&] {
      return c10::Storage(c10::Storage::use_byte_size_t(), (size_t)bytes, from->allocate((size_t)bytes),
                          from, /*resizable=*/true);
    };
    if (!other) return make();
    c10::cuda::CUDAStreamGuard guard(launch);
    c10::Storage s = make();
    c10::cuda::CUDACachingAllocator::recordStream(s.data_ptr(), current);
    return s;
  }
  static at::Tensor view(const c10::Storage& of, at::IntArrayRef shape, at::ScalarType type) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
        c10::Storage(of), c10::DispatchKeySet(c10::DispatchKey::CUDA),
        caffe2::TypeMeta::fromScalarType(type));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    return t;
  }
};

void check(exl3_status s, const char* what) {
  if (s == EXL3_OK) return;
  if (PyObject* e = PyObject_CallFunction(g_error, "is", (int)s, what)) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

// Runs f, which touches nothing of Python's, while other Python threads may run:
// an allocation may wait for the GPU, a launch for room in a full queue.
template <class F>
auto unlocked(F f) {
  struct Lock {
    PyThreadState* state = PyEval_SaveThread();
    ~Lock() { PyEval_RestoreThread(state); }
  } lock;
  return f();
}

// The tensors, and after them `last` (whose reference it takes) if there is one.
PyObject* tuple(std::initializer_list<at::Tensor> of, PyObject* last = nullptr) {
  PyObject* r = PyTuple_New((Py_ssize_t)of.size() + (last != nullptr));
  if (!r) throw Raised{};
  Py_ssize_t i = 0;
  for (const at::Tensor& t : of) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
  if (last) PyTuple_SET_ITEM(r, i, last);
  return r;
}

// [rows, vocab] probabilities (vocab < 0: any): the row stride.
int64_t rows_of(const at::Tensor& x, const char* name, int64_t rows, int64_t vocab) {
  if (x.scalar_type() != at::kFloat && x.scalar_type() != at::kHalf &&
      x.scalar_type() != at::kBFloat16)
    raise(PyExc_TypeError, "%s must be fp32, fp16 or bf16", name);
  if (x.dim() != 2 || x.size(0) != rows || (vocab >= 0 && x.size(1) != vocab) ||
      (x.stride(1) != 1 && x.size(1) > 1))
    raise(PyExc_ValueError, "%s must be [rows, vocab] with contiguous rows: a row per draft (q), and "
                            "one more per sequence (p)", name);
  return rows > 1 ? x.stride(0) : x.size(1);
}

// (p, draft, cu_draft, accept_u, sample_u, q, stream, the step's seq_lens)
PyObject* verify_drafts(PyObject* const* a) {
  const at::Tensor& draft = vector(a[1], "draft", at::kInt, -1);
  const at::Tensor& su = vector(a[4], "sample_u", at::kFloat, -1);
  const int64_t D = draft.size(0), B = su.size(0);
  const at::Tensor& p = tensor(a[0], "p");
  const int64_t ps = rows_of(p, "p", D + B, -1), vocab = p.size(1);
  const void* q = nullptr;
  int64_t qs = 0;
  if (a[5] != Py_None) {
    const at::Tensor& t = tensor(a[5], "q");
    qs = rows_of(t, "q", D, vocab);
    if (t.scalar_type() != p.scalar_type())
      raise(PyExc_ValueError, "%s must have the same dtype", "p and q");
    if (D > 0) q = t.data_ptr();
  }
  const at::Tensor& cu = vector(a[2], "cu_draft", at::kInt, B + 1);
  const at::Tensor& au = vector(a[3], "accept_u", at::kFloat, D);
  const int32_t* lens = lens_of(a[7], B);
  if (D > INT32_MAX || B > INT32_MAX || vocab > INT32_MAX)
    raise(PyExc_ValueError, "%s has too many rows or columns", "p");
  const Stream st(a[6], p);
  const exl3_dtype dt = p.scalar_type() == at::kFloat  ? EXL3_F32
                        : p.scalar_type() == at::kHalf ? EXL3_F16
                                                       : EXL3_BF16;
  std::array<at::Tensor, 3> out;  // tokens, accepted, dropped
  const exl3_status s = unlocked([&] {
    out = st.words<3>({{D + B}, {B}, {B}});
    return exl3_verify_drafts_step(p.data_ptr(), ps, q, qs, dt, (int)vocab, (int)B, (int)D,
                                   static_cast<const int32_t*>(cu.data_ptr()),
                                   static_cast<const int32_t*>(draft.data_ptr()),
                                   static_cast<const float*>(au.data_ptr()),
                                   static_cast<const float*>(su.data_ptr()), lens,
                                   static_cast<int32_t*>(out[0].data_ptr()),
                                   static_cast<int32_t*>(out[1].data_ptr()),
                                   static_cast<int32_t*>(out[2].data_ptr()), st.launch.stream());
  });
  check(s, "exl3_verify_drafts");
  return tuple({out[0], out[1], out[2]});
}

const at::Tensor& rows_named(PyObject* o, const exl3_page_pool* pool) {
  const at::Tensor& seqs = vector(o, "seqs", at::kInt, -1);
  if (seqs.size(0) > pool->max_seqs) raise(PyExc_ValueError, "%s names more rows than the pool has", "seqs");
  return seqs;
}

// (pool, ws, ws_bytes, seqs, q_lens, max_tokens, max_q, stream, device), the first
// three as numbers; the step's tensors and its exl3_kv_batch as bytes
PyObject* pages_extend(PyObject* const* a) {
  t_device = (int)whole(a[8]);
  const auto* pool = address<exl3_page_pool>(a[0]);
  const at::Tensor& seqs = rows_named(a[3], pool);
  const int64_t n = seqs.size(0), tokens = whole(a[5]), max_q = whole(a[6]);
  const at::Tensor& q = vector(a[4], "q_lens", at::kInt, n);
  if (tokens < 0 || tokens > INT32_MAX)
    raise(PyExc_ValueError, "%s must not be negative", "max_tokens");
  if (max_q < 0 || max_q > INT32_MAX) raise(PyExc_ValueError, "%s must not be negative", "max_q");
  void* const ws = address<void>(a[1]);
  const size_t bytes = (size_t)whole(a[2]);
  const Stream st(a[7], seqs);
  at::Tensor slots, pos, cu, lens, table;
  const exl3_status s = unlocked([&] {
    std::tie(pos, cu, lens) = std::tuple_cat(st.words<3>({{tokens}, {n + 1}, {n}}));
    table = st.empty({n, pool->max_pages}, at::kInt);
    slots = st.empty({tokens}, at::kLong);
    return exl3_pages_extend(pool, (int)n, static_cast<const int32_t*>(seqs.data_ptr()),
                             static_cast<const int32_t*>(q.data_ptr()), (int)tokens,
                             static_cast<int32_t*>(cu.data_ptr()),
                             static_cast<int32_t*>(lens.data_ptr()),
                             static_cast<int32_t*>(table.data_ptr()),
                             static_cast<int32_t*>(pos.data_ptr()),
                             static_cast<int64_t*>(slots.data_ptr()), ws, bytes, st.launch.stream());
  });
  check(s, "exl3_pages_extend");
  exl3_kv_batch batch{};
  batch.num_seqs = (int)n;
  batch.max_q = (int)max_q;
  batch.max_pages = pool->max_pages;
  batch.table_stride = pool->max_pages;
  batch.cu_q = static_cast<const int32_t*>(cu.data_ptr());
  batch.seq_lens = static_cast<const int32_t*>(lens.data_ptr());
  batch.block_table = static_cast<const int32_t*>(table.data_ptr());
  return tuple({cu, lens, table, pos, slots},
               PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&batch), sizeof batch));
}

// (pool, ws, ws_bytes, seqs, drop, stream, device, the step's seq_lens)
PyObject* pages_trim(PyObject* const* a) {
  t_device = (int)whole(a[6]);
  const auto* pool = address<exl3_page_pool>(a[0]);
  const at::Tensor& seqs = rows_named(a[3], pool);
  const int32_t* drop = nullptr;
  if (a[4] != Py_None)
    drop = static_cast<const int32_t*>(vector(a[4], "drop", at::kInt, seqs.size(0)).data_ptr());
  const int32_t* lens = lens_of(a[7], seqs.size(0));
  void* const ws = address<void>(a[1]);
  const size_t bytes = (size_t)whole(a[2]);
  const Stream st(a[5], seqs);
  const exl3_status s = unlocked([&] {
    return exl3_pages_trim_step(pool, (int)seqs.size(0), static_cast<const int32_t*>(seqs.data_ptr()),
                                drop, lens, ws, bytes, st.launch.stream());
  });
  check(s, "exl3_pages_trim");
  Py_RETURN_NONE;
}

// ---- append and attention
bool activation(const at::Tensor& t) {
  return t.scalar_type() == at::kHalf || t.scalar_type() == at::kBFloat16;
}
exl3_dtype code_of(const at::Tensor& t) {
  return t.scalar_type() == at::kHalf ? EXL3_F16 : EXL3_BF16;
}
// [tokens, heads, dim] activations with contiguous channels; the strides of a token
// and a head (0 where a dimension of one leaves them open).
const at::Tensor& heads_of(PyObject* o, const char* name, int64_t dim, int64_t* ts, int64_t* hs) {
  const at::Tensor& t = tensor(o, name);
  if (!activation(t)) raise(PyExc_TypeError, "%s must be fp16 or bf16", name);
  if (t.dim() != 3 || t.size(2) != dim || (t.stride(2) != 1 && t.numel() > 0))
    raise(PyExc_ValueError, "%s must be [tokens, heads, head_dim] with contiguous channels", name);
  if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX)
    raise(PyExc_ValueError, "%s has too many rows", name);
  *ts = t.size(0) == 1 ? 0 : t.stride(0);
  *hs = t.size(1) == 1 ? 0 : t.stride(1);
  return t;
}
const void* weight_of(PyObject* o, const char* name, at::ScalarType type, int64_t dim) {
  return o == Py_None ? nullptr : vector(o, name, type, dim).data_ptr();
}
// exl3_kv_batch: packed bytes or the address of one
const exl3_kv_batch* batch_of(PyObject* o) {
  return PyBytes_Check(o) ? reinterpret_cast<const exl3_kv_batch*>(PyBytes_AS_STRING(o))
                          : address<const exl3_kv_batch>(o);
}

// (cache, scales, batch, k, v, inv_freq, k_weight, q, q_weight, q_out, positions, eps,
//  interleaved, status, stream, device); cache, scales, batch and status as numbers
PyObject* kv_append(PyObject* const* a) {
  t_device = (int)whole(a[15]);
  const auto* cache = address<const exl3_kv_cache>(a[0]);
  const auto* scales = address<const exl3_kv_scales>(a[1]);
  const int64_t dim = cache->head_dim;
  exl3_heads k{}, v{}, q{};
  const at::Tensor& kt = heads_of(a[3], "k", dim, &k.token_stride, &k.head_stride);
  const at::Tensor& vt = heads_of(a[4], "v", dim, &v.token_stride, &v.head_stride);
  const int64_t T = kt.size(0);
  if (vt.scalar_type() != kt.scalar_type() || vt.size(0) != T || kt.size(1) != cache->kv_heads ||
      vt.size(1) != kt.size(1))
    raise(PyExc_ValueError, "%s must be [tokens, kv_heads, head_dim] of one dtype", "k and v");
  k.x = kt.data_ptr();
  v.x = vt.data_ptr();
  k.heads = v.heads = (int)kt.size(1);
  k.weight = weight_of(a[6], "k_weight", kt.scalar_type(), dim);
  at::Tensor out;
  const at::Tensor* made = nullptr;  // q, where its place is to be made
  if (a[7] != Py_None) {
    const at::Tensor& qt = heads_of(a[7], "q", dim, &q.token_stride, &q.head_stride);
    if (qt.scalar_type() != kt.scalar_type() || qt.size(0) != T)
      raise(PyExc_ValueError, "%s must have the same dtype and tokens", "q and k");
    q.x = qt.data_ptr();
    q.heads = (int)qt.size(1);
    q.weight = weight_of(a[8], "q_weight", qt.scalar_type(), dim);
    if (a[9] == Py_None) {
      made = &qt;
      q.out_token_stride = qt.size(1) * dim;
      q.out_head_stride = dim;
    } else {
      out = heads_of(a[9], "q_out", dim, &q.out_token_stride, &q.out_head_stride);
      if (out.scalar_type() != qt.scalar_type() || out.sizes() != qt.sizes())
        raise(PyExc_ValueError, "%s must have q's shape and dtype", "q_out");
      q.out = out.data_ptr();
    }
  }
  exl3_rope rope{};
  if (a[5] != Py_None) {
    const at::Tensor& f = vector(a[5], "inv_freq", at::kDouble, -1);
    if (f.size(0) > INT32_MAX / 2) raise(PyExc_ValueError, "%s is too long", "inv_freq");
    rope.inv_freq = static_cast<const double*>(f.data_ptr());
    rope.rotary_dim = 2 * (int)f.size(0);
    rope.interleaved = truth(a[12]);
  }
  const int32_t* positions =
      a[10] == Py_None ? nullptr
                       : static_cast<const int32_t*>(vector(a[10], "positions", at::kInt, T).data_ptr());
  const double eps = PyFloat_AsDouble(a[11]);
  if (eps == -1.0 && PyErr_Occurred()) throw Raised{};
  const exl3_heads* qp = a[7] != Py_None ? &q : nullptr;
  const exl3_rope* rp = rope.inv_freq || a[5] != Py_None ? &rope : nullptr;
  const exl3_kv_batch* const batch = batch_of(a[2]);
  int32_t* const status = address<int32_t>(a[13]);
  const Stream st(a[14], kt);
  const exl3_status s = unlocked([&] {
    if (made) {
      out = st.empty(made->sizes(), made->scalar_type());
      q.out = out.data_ptr();
    }
    return scales ? exl3_kv_append_blocks(cache, scales, batch, qp, &k, &v, code_of(kt), (int)T, rp,
                                          positions, (float)eps, status, st.launch.stream())
                  : exl3_kv_append(cache, batch, qp, &k, &v, code_of(kt), (int)T, rp, positions,
                                   (float)eps, status, st.launch.stream());
  });
  check(s, scales ? "exl3_kv_append_blocks" : "exl3_kv_append");
  if (!out.defined()) {  // (no q: what was given as its place comes back)
    Py_INCREF(a[9]);
    return a[9];
  }
  return THPVariable_Wrap(out);
}

// (cache, scales, batch, q, scale, causal, window, out, return_lse, path, ws, ws_bytes,
//  stream, device); cache, scales, batch and ws as numbers
PyObject* paged_attention(PyObject* const* a) {
  t_device = (int)whole(a[13]);
  const auto* cache = address<const exl3_kv_cache>(a[0]);
  const auto* scales = address<const exl3_kv_scales>(a[1]);
  const int64_t dim = cache->head_dim;
  int64_t ts, hs;
  const at::Tensor& q = heads_of(a[3], "q", dim, &ts, &hs);
  const double scale = PyFloat_AsDouble(a[4]);
  if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
  const int64_t window = whole(a[6]), path = whole(a[9]);
  const bool with_lse = truth(a[8]);
  if (window < INT32_MIN || window > INT32_MAX || path < INT32_MIN || path > INT32_MAX)
    raise(PyExc_ValueError, "%s out of range", "window or path");
  at::Tensor out, lse;
  if (a[7] != Py_None) {
    out = tensor(a[7], "out");
    if (out.scalar_type() != q.scalar_type()) raise(PyExc_TypeError, "%s must have q's dtype", "out");
    if (out.sizes() != q.sizes()) raise(PyExc_ValueError, "%s must have q's shape", "out");
    if (!out.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", "out");
  }
  void* const ws = address<void>(a[10]);
  const size_t bytes = (size_t)whole(a[11]);
  const int causal = truth(a[5]);
  const exl3_kv_batch* const batch = batch_of(a[2]);
  const Stream st(a[12], q);
  const exl3_status s = unlocked([&] {
    if (!out.defined()) out = st.empty(q.sizes(), q.scalar_type());
    if (with_lse) lse = st.empty({q.size(0), q.size(1)}, at::kFloat);
    float* const l = with_lse ? static_cast<float*>(lse.data_ptr()) : nullptr;
    return scales ? exl3_paged_attention_blocks(cache, scales, batch, q.data_ptr(), ts, hs, code_of(q),
                                                (int)q.size(0), (int)q.size(1), (float)scale, causal,
                                                (int)window, out.data_ptr(), l, (int)path, ws, bytes,
                                                st.launch.stream())
                  : exl3_paged_attention(cache, batch, q.data_ptr(), ts, hs, code_of(q),
                                         (int)q.size(0), (int)q.size(1), (float)scale, causal,
                                         (int)window, out.data_ptr(), l, (int)path, ws, bytes,
                                         st.launch.stream());
  });
  check(s, scales ? "exl3_paged_attention_blocks" : "exl3_paged_attention");
  if (with_lse) return tuple({out, lse});
  return THPVariable_Wrap(out);
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments, not %zd", N, n);
    return nullptr;
  }
  t_device = -1;
  t_count = 0;
  try {
    return F(args);
  } catch (const Raised&) {
  } catch (const std::exception& e) {  // torch's own (no memory)
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<F, N>)),
                     METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<verify_drafts, 8>("verify_drafts"),
                           method<pages_extend, 9>("pages_extend"),
                           method<pages_trim, 8>("pages_trim"),
                           method<kv_append, 16>("kv_append"),
                           method<paged_attention, 14>("paged_attention"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, g_methods,
                        nullptr,               nullptr,   nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() {
  PyObject* lib = PyImport_ImportModule("trellis_quantized_moe_exl3_gb300._lib");
  if (!lib) return nullptr;
  g_error = PyObject_GetAttrString(lib, "Exl3Error");
  Py_DECREF(lib);
  return g_error ? PyModule_Create(&g_module) : nullptr;
}
