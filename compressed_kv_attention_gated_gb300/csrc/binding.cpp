// binding.cpp -- CPython module that checks and unpacks torch tensors for the
// serving-step entry points of libckv (ckv.py wraps it).
//
// A decode step's calls take a few microseconds on the GPU; checking a dozen
// tensors and building a foreign call from Python takes 10 to 12, here about 1.
// Checks raise ValueError; a refusal by the C ABI comes back as its status,
// which ckv.py turns into CkvError.  No arithmetic, nothing kept between calls.
#include <Python.h>

#include <algorithm>
#include <cstdint>
#include <stdexcept>

#include <ATen/ATen.h>
#include <ATen/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "ckv.h"

namespace {

struct PyError {};  // a Python exception is set

void need(bool ok, const char* what) {
  if (!ok) throw std::invalid_argument(what);
}

// Positional arguments of a call, in order.
struct Args {
  PyObject* const* v;
  Py_ssize_t n, i = 0;
  int device = -1;

  Args(PyObject* const* values, Py_ssize_t count, Py_ssize_t expected) : v(values), n(count) {
    if (n != expected) {
      PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", expected, n);
      throw PyError{};
    }
  }
  PyObject* object() { return v[i++]; }
  int64_t integer() {
    const int64_t x = PyLong_AsLongLong(v[i++]);
    if (x == -1 && PyErr_Occurred()) throw PyError{};
    return x;
  }
  int32_t integer32(const char* what) {
    const int64_t x = integer();
    need(x >= INT32_MIN && x <= INT32_MAX, what);
    return static_cast<int32_t>(x);
  }
  double number() {
    const double x = PyFloat_AsDouble(v[i++]);
    if (x == -1.0 && PyErr_Occurred()) throw PyError{};
    return x;
  }
  int flag() {
    const int x = PyObject_IsTrue(v[i++]);
    if (x < 0) throw PyError{};
    return x;
  }
  // Every tensor on one CUDA device, which on_device() compares with the current one.
  const at::Tensor* check(PyObject* o, bool optional) {
    if (o == Py_None && optional) return nullptr;
    need(THPVariable_Check(o), "a torch tensor is expected");
    const at::Tensor& t = THPVariable_Unpack(o);
    need(t.is_cuda(), "every tensor must be on a CUDA device");
    const int d = t.get_device();
    need(device < 0 || d == device, "tensors on several CUDA devices");
    device = d;
    return &t;
  }
  const at::Tensor* optional() { return check(v[i++], true); }
  const at::Tensor& tensor() { return *check(v[i++], false); }
  // The kernels run on the current device, and a pointer into another one's memory would fault.
  void on_device() const {
    need(device < 0 || device == c10::cuda::current_device(),
         "the tensors are not on the current CUDA device (torch.cuda.set_device or torch.cuda.device(...) first)");
  }
  // -1: torch's current stream of the tensors' device.
  void* stream() {
    PyObject* o = v[i++];
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
    const unsigned long long s = PyLong_AsUnsignedLongLong(o);
    if (s == static_cast<unsigned long long>(-1) && PyErr_Occurred()) throw PyError{};
    return reinterpret_cast<void*>(static_cast<uintptr_t>(s));
  }
};

template <typename T>
T* ptr(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}
template <typename T>
T* ptr(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

bool vec(const at::Tensor& t, at::ScalarType type, int64_t n) {
  return t.scalar_type() == type && t.is_contiguous() && t.numel() == n;
}

ckv_dtype dtype_of(const at::Tensor& t) {
  need(t.scalar_type() == at::kFloat || t.scalar_type() == at::kBFloat16, "input must be float32 or bfloat16");
  return t.scalar_type() == at::kFloat ? CKV_F32 : CKV_BF16;
}

// A table of int32 rows, last dimension contiguous, and the step between its rows: 0 when all B > 1
// requests share one row (only where `shared`), else at least the width.
int64_t table_rows(const at::Tensor& t, int64_t B, bool shared, const char* what) {
  need(t.scalar_type() == at::kInt && t.dim() == 2 && t.size(0) == B && (t.stride(1) == 1 || t.size(1) <= 1), what);
  if (B <= 1) return t.size(1);  // the step of a dimension of one entry is never used
  if (shared && t.stride(0) == 0) return 0;
  need(t.stride(0) >= t.size(1), "rows of block_table overlap");
  return t.stride(0);
}

const char kStepNames[][16] = {"row_start",  "positions",  "batch_ids",     "slot_mapping",
                               "cache_loc",  "tail_slots", "row_positions", "ctx_rows"};
constexpr int kSteps = 8;

template <typename F>
PyObject* guarded(F&& f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const PyError&) {
    return nullptr;
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* step_maps(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(v, n, 14);
    const at::Tensor &seq = a.tensor(), &query = a.tensor(), &table = a.tensor(), &free = a.tensor(), &cursor = a.tensor();
    const int32_t P = a.integer32("pool_size"), ps = a.integer32("page_size"), T = a.integer32("num_tokens");
    const at::Tensor *tails = a.optional(), *cursor_out = a.optional();
    PyObject* given = a.object();
    const int pdl = a.flag();
    const at::Tensor* err = a.optional();
    const int64_t B = seq.numel();
    need(T >= 0, "num_tokens must not be negative");
    need(vec(seq, at::kInt, B) && vec(query, at::kInt, B) && (!tails || vec(*tails, at::kInt, B)),
         "seq_lens, query_lens and tail_blocks must be contiguous int32 [B]");
    need(B <= INT32_MAX, "too many requests");
    const int64_t stride = table_rows(table, B, false, "block_table must be int32 [B, max_pages], last dim contiguous");
    need(table.size(1) <= INT32_MAX, "block_table is too wide");
    need(free.scalar_type() == at::kInt && free.is_contiguous(), "free_pages must be contiguous int32");
    const bool inplace = !cursor_out || cursor_out->data_ptr() == cursor.data_ptr();
    need(cursor.scalar_type() == at::kInt && cursor.is_contiguous() && cursor.numel() >= (inplace ? 2 : 1),
         "cursor must be int32 [1], or [2] when it is moved in place");
    need(!cursor_out || (cursor_out->scalar_type() == at::kInt && cursor_out->numel() >= 1), "cursor_out must be int32 [1]");
    need(!err || err->scalar_type() == at::kInt, "err_word must be int32");
    PyObject* out = nullptr;
    at::Tensor made[kSteps];
    const at::Tensor* map[kSteps] = {};
    if (given == Py_None) {
      a.on_device();
      const auto opt = seq.options().dtype(at::kInt);
      for (int k = 0; k < kSteps; ++k) {
        if (k == 5 && !tails) continue;
        made[k] = at::empty({k == 0 ? B + 1 : static_cast<int64_t>(T)}, k == 4 ? opt.dtype(at::kLong) : opt);
        map[k] = &made[k];
      }
    } else {
      need(PyDict_Check(given), "out must be a dict of maps");
      Py_ssize_t known = 0;
      for (int k = 0; k < kSteps; ++k) {
        PyObject* o = PyDict_GetItemString(given, kStepNames[k]);
        if (!o) continue;
        ++known;
        map[k] = a.check(o, false);
        need(vec(*map[k], k == 4 ? at::kLong : at::kInt, k == 0 ? B + 1 : static_cast<int64_t>(T)),
             "a map in out has the wrong type or size");
      }
      need(known == PyDict_Size(given), "out holds a map that does not exist");
      need(!map[5] || tails, "tail_slots need tail_blocks");
      a.on_device();
    }
    void* stream = a.stream();
    const ckv_status s = ckv_build_step_maps(
        ptr<int32_t>(seq), ptr<int32_t>(query), static_cast<int32_t>(B), P, ps, ptr<int32_t>(table), stride,
        static_cast<int32_t>(table.size(1)), ptr<int32_t>(free), free.numel(), ptr<int32_t>(cursor),
        inplace ? ptr<int32_t>(cursor) : ptr<int32_t>(cursor_out), ptr<int32_t>(tails), T, ptr<int32_t>(map[0]),
        ptr<int32_t>(map[1]), ptr<int32_t>(map[2]), ptr<int32_t>(map[3]), ptr<int64_t>(map[4]), ptr<int32_t>(map[5]),
        ptr<int32_t>(map[6]), ptr<int32_t>(map[7]), pdl, ptr<int32_t>(err), stream);
    if (given == Py_None) {
      out = PyDict_New();
      if (!out) return nullptr;
      for (int k = 0; k < kSteps; ++k) {
        if (!map[k]) continue;
        PyObject* t = THPVariable_Wrap(made[k]);
        if (!t || PyDict_SetItemString(out, kStepNames[k], t) < 0) {
          Py_XDECREF(t);
          Py_DECREF(out);
          return nullptr;
        }
        Py_DECREF(t);
      }
    } else {
      out = given;
      Py_INCREF(out);
    }
    return Py_BuildValue("iN", static_cast<int>(s), out);
  });
}

// One row set of qk_norm_rope; allocates its output when none is given.
ckv_norm_rows row_set(const at::Tensor& x, const at::Tensor& positions, const at::Tensor* weight, at::Tensor& out, int64_t D) {
  need(x.dim() == 3 && x.size(2) == D && x.stride(2) == 1, "q and k must be [tokens, heads, D], last dim contiguous");
  const int64_t T = x.size(0), H = x.size(1);
  if (!out.defined()) out = at::empty({T, H, D}, x.options().dtype(at::kBFloat16));
  need(out.sizes() == x.sizes() && out.stride(2) == 1, "an output must have the shape of its input, last dim contiguous");
  need(vec(positions, at::kInt, T), "positions must be contiguous int32 [tokens]");
  need(!weight || vec(*weight, at::kFloat, D), "weights must be contiguous float32 [D]");
  need(H <= INT32_MAX, "too many heads");
  const int64_t st = out.stride(0), sh = out.stride(1);
  // rows that share memory would be written over one another
  need((T <= 1 || st >= D) && (H <= 1 || sh >= D) && (T <= 1 || H <= 1 || st >= (H - 1) * sh + D || sh >= (T - 1) * st + D),
       "rows of an output overlap");
  ckv_norm_rows r{};
  r.x = x.data_ptr();
  r.out = out.data_ptr();
  r.weight = ptr<float>(weight);
  r.positions = ptr<int32_t>(positions);
  r.stride_t = T > 1 ? x.stride(0) : 0;  // the step of a dimension of one entry is never used
  r.stride_h = H > 1 ? x.stride(1) : 0;
  r.out_stride_t = T > 1 ? st : 0;
  r.out_stride_h = H > 1 ? sh : 0;
  r.tokens = T;
  r.heads = static_cast<int32_t>(H);
  r.dtype = dtype_of(x);
  r.out_dtype = dtype_of(out);
  return r;
}

PyObject* qk_norm_rope(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(v, n, 15);
    const at::Tensor &q = a.tensor(), &qp = a.tensor();
    const at::Tensor *cs = a.optional(), *qw = a.optional(), *qo = a.optional();
    const at::Tensor *k = a.optional(), *kp = a.optional(), *kw = a.optional(), *ko = a.optional();
    PyObject* at_arg = a.object();
    const int interleaved = a.flag();
    const float eps = static_cast<float>(a.number());
    const int pdl = a.flag();
    const at::Tensor* err = a.optional();
    a.on_device();
    need(q.dim() == 3, "q must be [tokens, heads, D], last dim contiguous");
    const int64_t D = q.size(2);
    need(D <= 1024, "unsupported D");
    need(!cs || (cs->scalar_type() == at::kFloat && cs->dim() == 2 && cs->is_contiguous()), "cos_sin must be contiguous float32 [positions, rope_dim]");
    const int64_t R = cs ? cs->size(1) : 0;
    need(R <= D, "rope_dim must be at most D");
    need(!k || kp, "k needs k_positions");
    need(!err || err->scalar_type() == at::kInt, "err_word must be int32");
    int64_t at = D - R;
    if (at_arg != Py_None) {
      at = PyLong_AsLongLong(at_arg);
      if (at == -1 && PyErr_Occurred()) return nullptr;
      need(at >= 0 && at <= D, "rope_offset must be in 0..D - rope_dim");
    }
    at::Tensor q_out = qo ? *qo : at::Tensor(), k_out = ko ? *ko : at::Tensor();
    const ckv_norm_rows rq = row_set(q, qp, qw, q_out, D);
    ckv_norm_rows rk{};
    if (k) rk = row_set(*k, *kp, kw, k_out, D);
    const ckv_status s = ckv_qk_norm_rope(&rq, k ? &rk : nullptr, ptr<float>(cs), cs ? cs->size(0) : 0, static_cast<int32_t>(D),
                                          static_cast<int32_t>(R), static_cast<int32_t>(at), interleaved, eps, pdl, ptr<int32_t>(err),
                                          a.stream());
    PyObject* kt = Py_None;
    if (k) kt = THPVariable_Wrap(k_out);
    else Py_INCREF(kt);
    return Py_BuildValue("iNN", static_cast<int>(s), THPVariable_Wrap(q_out), kt);
  });
}

struct Cache {
  uint8_t* p;
  int64_t pages;
  int32_t page_size;
};
Cache fp4_cache(const at::Tensor& t, int64_t D) {
  need(t.scalar_type() == at::kByte && t.is_contiguous() && t.dim() == 3 && t.size(2) == D / 2 + D / 16,
       "kv_cache must be contiguous uint8 [pages, page_size, D/2 + D/16]");
  need(t.size(1) <= INT32_MAX, "page_size is too large");
  return {static_cast<uint8_t*>(t.data_ptr()), t.size(0), static_cast<int32_t>(t.size(1))};
}

// rows/out, kv_cache, loc, cache_scale, use_pdl, err_word, stream
PyObject* fp4_rows(PyObject* const* v, Py_ssize_t n, bool store) {
  return guarded([&]() -> PyObject* {
    Args a(v, n, 7);
    const at::Tensor &x = a.tensor(), &cache = a.tensor(), &loc = a.tensor();
    const float g = static_cast<float>(a.number());
    const int pdl = a.flag();
    const at::Tensor* err = a.optional();
    a.on_device();
    need(x.dim() == 2 && (x.stride(1) == 1 || x.numel() == 0), "rows must be [n, D], last dim contiguous");
    const int64_t rows = x.size(0), D = x.size(1);
    need(D <= 1024, "unsupported D");
    const Cache c = fp4_cache(cache, D);
    need(vec(loc, at::kLong, rows), "loc must be contiguous int64 [n]");
    need(!err || err->scalar_type() == at::kInt, "err_word must be int32");
    const int64_t stride = rows > 1 ? x.stride(0) : 0;
    const ckv_dtype type = dtype_of(x);
    void* stream = a.stream();
    const ckv_status s =
        store ? ckv_fp4_store(x.data_ptr(), type, stride, rows, static_cast<int32_t>(D), c.p, c.pages, c.page_size,
                              ptr<int64_t>(loc), g, pdl, ptr<int32_t>(err), stream)
              : ckv_fp4_load(c.p, c.pages, c.page_size, ptr<int64_t>(loc), rows, static_cast<int32_t>(D), x.data_ptr(), type, stride,
                             g, pdl, ptr<int32_t>(err), stream);
    return PyLong_FromLong(s);
  });
}
PyObject* fp4_store(PyObject*, PyObject* const* v, Py_ssize_t n) { return fp4_rows(v, n, true); }
PyObject* fp4_load(PyObject*, PyObject* const* v, Py_ssize_t n) { return fp4_rows(v, n, false); }

PyObject* fp4_attention(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(v, n, 15);
    const at::Tensor &q = a.tensor(), &cache = a.tensor(), &table = a.tensor(), &start = a.tensor(), &ctx = a.tensor();
    const int64_t max_rows = a.integer();
    const float scale = static_cast<float>(a.number()), g = static_cast<float>(a.number());
    const at::Tensor *sink = a.optional(), *out = a.optional(), *lse = a.optional(), *ws = a.optional();
    const int pdl = a.flag();
    const at::Tensor* err = a.optional();
    a.on_device();
    need(q.scalar_type() == at::kBFloat16 && q.dim() == 3 && (q.stride(2) == 1 || q.numel() == 0),
         "q must be bf16 [T, H, D], last dim contiguous");
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
    need(H <= INT32_MAX && D <= 1024, "unsupported H or D");
    const Cache c = fp4_cache(cache, D);
    need(start.scalar_type() == at::kInt && start.is_contiguous() && start.numel() >= 1 && start.numel() <= INT32_MAX,
         "row_start must be contiguous int32 [B + 1]");
    const int64_t B = start.numel() - 1;
    const int64_t stride = table_rows(table, B, true, "block_table must be int32 [B, max_pages], last dim contiguous");
    need(table.size(1) <= INT32_MAX, "block_table is too wide");
    need(vec(ctx, at::kInt, T), "ctx_rows must be contiguous int32 [T]");
    need(!sink || vec(*sink, at::kFloat, H), "sink must be contiguous float32 [H]");
    need(!err || err->scalar_type() == at::kInt, "err_word must be int32");
    at::Tensor o = out ? *out : at::empty({T, H, D}, q.options());
    at::Tensor l = lse ? *lse : at::empty({T, H}, q.options().dtype(at::kFloat));
    need(o.scalar_type() == at::kBFloat16 && o.is_contiguous() && o.sizes() == q.sizes(), "out must be contiguous bf16 [T, H, D]");
    need(l.scalar_type() == at::kFloat && l.is_contiguous() && l.dim() == 2 && l.size(0) == T && l.size(1) == H,
         "lse must be contiguous float32 [T, H]");
    need(!ws || ws->is_contiguous(), "workspace must be contiguous");
    const int64_t bytes = ckv_fp4_attention_workspace(T, static_cast<int32_t>(std::min<int64_t>(B, INT32_MAX)),
                                                      static_cast<int32_t>(H), static_cast<int32_t>(D), max_rows);
    at::Tensor w = ws ? *ws : bytes > 0 ? at::empty({bytes}, q.options().dtype(at::kByte)) : at::Tensor();
    const ckv_status s = ckv_fp4_attention(
        ptr<uint16_t>(q), T > 1 ? q.stride(0) : 0, H > 1 ? q.stride(1) : 0, T, static_cast<int32_t>(H), static_cast<int32_t>(D),
        c.p, c.pages, c.page_size, g, ptr<int32_t>(table), stride, static_cast<int32_t>(table.size(1)), ptr<int32_t>(start),
        static_cast<int32_t>(B), ptr<int32_t>(ctx), max_rows, scale, ptr<float>(sink), ptr<uint16_t>(o), ptr<float>(l),
        w.defined() ? w.data_ptr() : nullptr, w.defined() ? static_cast<int64_t>(w.nbytes()) : 0, pdl, ptr<int32_t>(err), a.stream());
    return Py_BuildValue("iNN", static_cast<int>(s), THPVariable_Wrap(o), THPVariable_Wrap(l));
  });
}

// A paged cache of uncompressed rows [pages, page_size, KH, D] and its strides; `written`: its rows
// may not share memory.
void kv_side(const at::Tensor& t, bool written, uint16_t*& p, int64_t& page, int64_t& row, int64_t& head) {
  need(t.scalar_type() == at::kBFloat16 && t.dim() == 4 && (t.stride(3) == 1 || t.numel() == 0),
       "a cache must be bf16 [pages, page_size, KH, D], last dim contiguous");
  p = static_cast<uint16_t*>(t.data_ptr());
  int64_t* to[3] = {&page, &row, &head};
  for (int i = 0; i < 3; ++i) *to[i] = t.size(i) > 1 ? t.stride(i) : 0;  // the step of a dimension of one entry is never used
  if (!written || t.numel() == 0) return;
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int x, int y) { return t.stride(x) < t.stride(y); });
  int64_t span = t.size(3);
  for (int i : order) {
    if (t.size(i) == 1) continue;
    need(t.stride(i) >= span, "rows of a cache overlap");
    span += (t.size(i) - 1) * t.stride(i);
  }
}
// A new tensor of the current device from torch's caching allocator: past the dispatcher, which takes longer than the
// allocation (tree masks, two tensors: 4.9 to 7 us of host time per call, 3.9 so).
at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type) {
  return at::Tensor(at::detail::empty_generic(sizes, c10::cuda::CUDACachingAllocator::get(), c10::DispatchKeySet(c10::DispatchKey::CUDA), type, {}));
}

ckv_kv_cache kv_cache(const at::Tensor& k, const at::Tensor* v, bool written) {
  ckv_kv_cache c{};
  kv_side(k, written, c.k, c.k_stride_page, c.k_stride_row, c.k_stride_head);
  if (v) {
    need(v->sizes() == k.sizes(), "the caches of keys and values must have one shape");
    kv_side(*v, written, c.v, c.v_stride_page, c.v_stride_row, c.v_stride_head);
  }
  need(k.size(1) <= INT32_MAX && k.size(2) <= INT32_MAX && k.size(3) <= 1024, "unsupported page_size, heads or D");
  c.num_pages = k.size(0);
  c.page_size = static_cast<int32_t>(k.size(1));
  c.heads = static_cast<int32_t>(k.size(2));
  c.D = static_cast<int32_t>(k.size(3));
  return c;
}

ckv_kv_rows kv_rows(const at::Tensor& x, int64_t T, int64_t D) {
  need(x.dim() == 3 && x.size(0) == T && x.size(2) == D && (x.stride(2) == 1 || x.numel() == 0),
       "q, k and v must be [T, heads, D], last dim contiguous");
  need(x.size(1) <= INT32_MAX, "too many heads");
  ckv_kv_rows r{};
  r.x = x.data_ptr();
  r.stride_t = T > 1 ? x.stride(0) : 0;
  r.stride_h = x.size(1) > 1 ? x.stride(1) : 0;
  r.heads = static_cast<int32_t>(x.size(1));
  r.dtype = dtype_of(x);
  return r;
}

PyObject* kv_append(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(v, n, 14);
    const at::Tensor& k = a.tensor();
    const at::Tensor* val = a.optional();
    const at::Tensor& kc = a.tensor();
    const at::Tensor* vc = a.optional();
    const at::Tensor& loc = a.tensor();
    const at::Tensor *pos = a.optional(), *cs = a.optional();
    PyObject* at_arg = a.object();
    const int interleaved = a.flag();
    const at::Tensor *q = a.optional(), *qo = a.optional();
    const int pdl = a.flag();
    const at::Tensor* err = a.optional();
    a.on_device();
    need(k.dim() == 3, "q, k and v must be [T, heads, D], last dim contiguous");
    need(!val || vc, "v needs v_cache");
    need(!qo || q, "q_out needs q");
    const ckv_kv_cache c = kv_cache(kc, val ? vc : nullptr, true);
    const int64_t T = k.size(0), D = c.D;
    need(vec(loc, at::kLong, T), "loc must be contiguous int64 [T]");
    need(!pos || vec(*pos, at::kInt, T), "positions must be contiguous int32 [T]");
    need(!cs || (cs->scalar_type() == at::kFloat && cs->dim() == 2 && cs->is_contiguous()), "cos_sin must be contiguous float32 [positions, rope_dim]");
    const int64_t R = cs ? cs->size(1) : 0;
    need(R <= D, "rope_dim must be at most D");
    need(!err || err->scalar_type() == at::kInt, "err_word must be int32");
    int64_t at = D - R;
    if (at_arg != Py_None) {
      at = PyLong_AsLongLong(at_arg);
      if (at == -1 && PyErr_Occurred()) return nullptr;
      need(at >= 0 && at <= D, "rope_offset must be in 0..D - rope_dim");
    }
    const ckv_kv_rows rk = kv_rows(k, T, D);
    ckv_kv_rows rv{}, rq{};
    if (val) rv = kv_rows(*val, T, D);
    at::Tensor out;
    int64_t st = 0, sh = 0;
    if (q) {
      rq = kv_rows(*q, T, D);
      out = qo ? *qo : fresh({T, q->size(1), D}, at::kBFloat16);
      need(out.scalar_type() == at::kBFloat16 && out.sizes() == q->sizes() && (out.stride(2) == 1 || out.numel() == 0),
           "q_out must be bf16 with the shape of q, last dim contiguous");
      const int64_t H = q->size(1);
      st = T > 1 ? out.stride(0) : 0;
      sh = H > 1 ? out.stride(1) : 0;
      need((T <= 1 || st >= D) && (H <= 1 || sh >= D) && (T <= 1 || H <= 1 || st >= (H - 1) * sh + D || sh >= (T - 1) * st + D),
           "rows of an output overlap");
    }
    const ckv_status s = ckv_kv_append(&rk, val ? &rv : nullptr, q ? &rq : nullptr, q ? static_cast<uint16_t*>(out.data_ptr()) : nullptr, st, sh,
                                       T, &c, ptr<int64_t>(loc), ptr<int32_t>(pos), ptr<float>(cs), cs ? cs->size(0) : 0,
                                       static_cast<int32_t>(R), static_cast<int32_t>(at), interleaved, pdl, ptr<int32_t>(err), a.stream());
    PyObject* made = Py_None;
    if (q) made = THPVariable_Wrap(out);
    else Py_INCREF(made);
    return Py_BuildValue("iN", static_cast<int>(s), made);
  });
}

PyObject* tree_masks(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(v, n, 9);
    const at::Tensor &parents = a.tensor(), &start = a.tensor();
    const at::Tensor* ctx = a.optional();
    const int32_t words = a.integer32("words");
    const at::Tensor *mask = a.optional(), *pos = a.optional();
    const int pdl = a.flag();
    const at::Tensor* err = a.optional();
    a.on_device();
    const int64_t T = parents.numel();
    need(vec(parents, at::kInt, T) && (!ctx || vec(*ctx, at::kInt, T)), "parents and ctx_rows must be contiguous int32 [T]");
    need(start.scalar_type() == at::kInt && start.is_contiguous() && start.numel() >= 1 && start.numel() <= INT32_MAX,
         "row_start must be contiguous int32 [B + 1]");
    need(words >= 1 && words <= 16, "words must be in 1..16");
    need(!err || err->scalar_type() == at::kInt, "err_word must be int32");
    at::Tensor m = mask ? *mask : fresh({T, words}, at::kLong);
    at::Tensor p = pos ? *pos : fresh({T}, at::kInt);
    need(m.scalar_type() == at::kLong && m.is_contiguous() && m.dim() == 2 && m.size(0) == T && m.size(1) == words,
         "tree_mask must be contiguous int64 [T, words]");
    need(vec(p, at::kInt, T), "positions must be contiguous int32 [T]");
    const ckv_status s = ckv_build_tree_masks(ptr<int32_t>(parents), ptr<int32_t>(start), static_cast<int32_t>(start.numel() - 1),
                                              ptr<int32_t>(ctx), T, words, ptr<uint64_t>(m), ptr<int32_t>(p), pdl, ptr<int32_t>(err), a.stream());
    return Py_BuildValue("iNN", static_cast<int>(s), THPVariable_Wrap(m), THPVariable_Wrap(p));
  });
}

PyObject* kv_attention(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(v, n, 18);
    const at::Tensor &q = a.tensor(), &kc = a.tensor(), &vc = a.tensor(), &table = a.tensor(), &start = a.tensor(), &ctx = a.tensor();
    const int64_t max_rows = a.integer();
    const float scale = static_cast<float>(a.number());
    const int32_t window = a.integer32("window"), first = a.integer32("first_rows");
    const at::Tensor *mask = a.optional(), *sink = a.optional(), *out = a.optional(), *lse = a.optional(), *ws = a.optional();
    const int pdl = a.flag();
    const at::Tensor* err = a.optional();
    a.on_device();
    need(q.scalar_type() == at::kBFloat16 && q.dim() == 3 && (q.stride(2) == 1 || q.numel() == 0),
         "q must be bf16 [T, H, D], last dim contiguous");
    const ckv_kv_cache c = kv_cache(kc, &vc, false);
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
    need(D == c.D, "q and the caches must have one D");
    need(H <= INT32_MAX, "unsupported H");
    need(start.scalar_type() == at::kInt && start.is_contiguous() && start.numel() >= 1 && start.numel() <= INT32_MAX,
         "row_start must be contiguous int32 [B + 1]");
    const int64_t B = start.numel() - 1;
    const int64_t stride = table_rows(table, B, true, "block_table must be int32 [B, max_pages], last dim contiguous");
    need(table.size(1) <= INT32_MAX, "block_table is too wide");
    need(vec(ctx, at::kInt, T), "ctx_rows must be contiguous int32 [T]");
    need(!mask || (mask->scalar_type() == at::kLong && mask->is_contiguous() && mask->dim() == 2 && mask->size(0) == T && mask->size(1) >= 1 &&
                   mask->size(1) <= 16),
         "tree_mask must be contiguous int64 [T, 1..16]");
    need(!sink || vec(*sink, at::kFloat, H), "sink must be contiguous float32 [H]");
    need(!err || err->scalar_type() == at::kInt, "err_word must be int32");
    const int32_t words = mask ? static_cast<int32_t>(mask->size(1)) : 0;
    at::Tensor o = out ? *out : fresh({T, H, D}, at::kBFloat16);
    at::Tensor l = lse ? *lse : fresh({T, H}, at::kFloat);
    need(o.scalar_type() == at::kBFloat16 && o.is_contiguous() && o.sizes() == q.sizes(), "out must be contiguous bf16 [T, H, D]");
    need(l.scalar_type() == at::kFloat && l.is_contiguous() && l.dim() == 2 && l.size(0) == T && l.size(1) == H,
         "lse must be contiguous float32 [T, H]");
    need(!ws || ws->is_contiguous(), "workspace must be contiguous");
    const int64_t bytes = ckv_kv_attention_workspace(T, static_cast<int32_t>(std::min<int64_t>(B, INT32_MAX)), static_cast<int32_t>(H), c.heads,
                                                     c.D, max_rows, window, first, words);
    at::Tensor w = ws ? *ws : bytes > 0 ? fresh({bytes}, at::kByte) : at::Tensor();
    const ckv_status s = ckv_kv_attention(
        ptr<uint16_t>(q), T > 1 ? q.stride(0) : 0, H > 1 ? q.stride(1) : 0, T, static_cast<int32_t>(H), &c, ptr<int32_t>(table), stride,
        static_cast<int32_t>(table.size(1)), ptr<int32_t>(start), static_cast<int32_t>(B), ptr<int32_t>(ctx), max_rows, window, first,
        ptr<uint64_t>(mask), words, scale, ptr<float>(sink), ptr<uint16_t>(o), ptr<float>(l), w.defined() ? w.data_ptr() : nullptr,
        w.defined() ? static_cast<int64_t>(w.nbytes()) : 0, pdl, ptr<int32_t>(err), a.stream());
    return Py_BuildValue("iNN", static_cast<int>(s), THPVariable_Wrap(o), THPVariable_Wrap(l));
  });
}

PyObject* merge_attention(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(v, n, 7);
    PyObject *outs = a.object(), *lses = a.object();
    const at::Tensor *pos = a.optional(), *out = a.optional(), *lse = a.optional();
    const int pdl = a.flag();
    need((PyList_Check(outs) || PyTuple_Check(outs)) && (PyList_Check(lses) || PyTuple_Check(lses)), "outs and lses must be lists of tensors");
    const Py_ssize_t parts = PySequence_Fast_GET_SIZE(outs);
    need(parts >= 1 && parts <= 8 && PySequence_Fast_GET_SIZE(lses) == parts, "1..8 outs, and as many lses");
    ckv_attention_part p[8];
    const at::Tensor& o0 = *a.check(PySequence_Fast_GET_ITEM(outs, 0), false);
    need(o0.dim() == 3, "outs must be contiguous [T, H, D] of one type");
    const int64_t T = o0.size(0), H = o0.size(1), D = o0.size(2);
    for (Py_ssize_t i = 0; i < parts; ++i) {
      const at::Tensor& o = *a.check(PySequence_Fast_GET_ITEM(outs, i), false);
      const at::Tensor& l = *a.check(PySequence_Fast_GET_ITEM(lses, i), false);
      need(o.is_contiguous() && o.sizes() == o0.sizes() && o.scalar_type() == o0.scalar_type(), "outs must be contiguous [T, H, D] of one type");
      need(l.scalar_type() == at::kFloat && l.is_contiguous() && l.dim() == 2 && l.size(0) == T && l.size(1) == H,
           "lses must be contiguous float32 [T, H]");
      p[i] = {o.data_ptr(), static_cast<const float*>(l.data_ptr())};
    }
    a.on_device();
    need(H <= INT32_MAX && D <= 1024, "unsupported H or D");
    need(!pos || vec(*pos, at::kInt, T), "positions must be contiguous int32 [T]");
    at::Tensor o = out ? *out : fresh({T, H, D}, at::kBFloat16);
    at::Tensor l = lse ? *lse : fresh({T, H}, at::kFloat);
    need(o.is_contiguous() && o.sizes() == o0.sizes(), "out must be contiguous [T, H, D]");
    need(l.scalar_type() == at::kFloat && l.is_contiguous() && l.dim() == 2 && l.size(0) == T && l.size(1) == H,
         "lse must be contiguous float32 [T, H]");
    const ckv_status s = ckv_merge_attention(p, static_cast<int32_t>(parts), dtype_of(o0), T, static_cast<int32_t>(H), static_cast<int32_t>(D),
                                             ptr<int32_t>(pos), o.data_ptr(), dtype_of(o), ptr<float>(l), pdl, a.stream());
    return Py_BuildValue("iNN", static_cast<int>(s), THPVariable_Wrap(o), THPVariable_Wrap(l));
  });
}

#define METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {
    {"step_maps", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(step_maps)), METH_FASTCALL, nullptr},
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(qk_norm_rope)), METH_FASTCALL, nullptr},
    {"fp4_store", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fp4_store)), METH_FASTCALL, nullptr},
    {"fp4_load", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fp4_load)), METH_FASTCALL, nullptr},
    {"fp4_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fp4_attention)), METH_FASTCALL, nullptr},
    METHOD(kv_append),
    METHOD(tree_masks),
    METHOD(kv_attention),
    METHOD(merge_attention),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "ckv_binding", "Tensor checks and calls of libckv's serving-step entry points.", -1,
                       kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ckv_binding() { return PyModule_Create(&kModule); }
