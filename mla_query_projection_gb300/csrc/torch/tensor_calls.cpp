// tensor_calls.cpp - the cache-side and prompt operators of libmla_query for torch tensors:
// a CPython module that checks the tensors of a call and hands their addresses,
// sizes and strides to the C ABI.
//
// A small step's call costs more on the host than on the GPU: reading a dozen
// tensors' type, sizes and device from Python and passing two dozen arguments
// through ctypes took 6.7 us (blocks_select) to 12.6 us (attention, two
// launches) a call, with the launches; here 2.9 to 5.1 us.
//
// The module does not link the library: bind() takes the addresses of its
// functions, so that whichever build is loaded is the one that is called.  A
// call returns None, or what is wrong as text, or the library's return code.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstdint>
#include <exception>

#include "../../../include/mla_query.h"

namespace {

decltype(&mla_tables_step) tables_step_c = nullptr;
decltype(&mla_blocks_mean_cols) blocks_mean_c = nullptr;
decltype(&mla_blocks_score) blocks_score_c = nullptr;
decltype(&mla_blocks_select) blocks_select_c = nullptr;
decltype(&mla_attn_decode_cols) attn_decode_c = nullptr;
decltype(&mla_rope_apply) rope_apply_c = nullptr;
decltype(&mla_cache_write) cache_write_c = nullptr;
decltype(&mla_cache_read) cache_read_c = nullptr;
decltype(&mla_prompt_attn) prompt_attn_c = nullptr;

// What a call asks of its tensors; the first thing that is wrong stays.
class Call {
 public:
  explicit Call(PyObject* first) {
    if (const at::Tensor* t = tensor(first, "tensors")) dev_ = t->get_device();
  }

  const at::Tensor* tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) {
      wrong(what);
      return nullptr;
    }
    return &THPVariable_Unpack(o);
  }
  // Address of a contiguous tensor with at least n elements; null for None.
  template <class T = void>
  T* flat(PyObject* o, at::ScalarType type, int64_t n, const char* what) {
    if (o == Py_None) return nullptr;
    const at::Tensor* t = tensor(o, what);
    if (t == nullptr) return nullptr;
    if (t->scalar_type() != type || !t->is_contiguous() || t->numel() < n || t->get_device() != dev_) {
      wrong(what);
      return nullptr;
    }
    return static_cast<T*>(t->data_ptr());
  }
  // The same of a contiguous tensor of `dim` dimensions; its sizes.
  template <class T = void>
  T* whole(PyObject* o, at::ScalarType type, int64_t dim, int64_t* sizes, const char* what) {
    for (int64_t i = 0; i < dim; ++i) sizes[i] = 0;
    const at::Tensor* t = tensor(o, what);
    if (t == nullptr) return nullptr;
    if (t->dim() != dim) {
      wrong(what);
      return nullptr;
    }
    for (int64_t i = 0; i < dim; ++i) sizes[i] = t->size(i);
    return flat<T>(o, type, 0, what);
  }
  // Address of a [rows, columns] tensor with unit inner stride.
  template <class T = void>
  T* rows(PyObject* o, at::ScalarType type, int64_t* stride, int64_t* rows, int64_t* cols, const char* what) {
    *stride = *rows = *cols = 0;
    const at::Tensor* t = tensor(o, what);
    if (t == nullptr) return nullptr;
    if (t->dim() != 2) {
      wrong(what);
      return nullptr;
    }
    *rows = t->size(0);
    *cols = t->size(1);
    const int64_t st = t->stride(0);
    if (t->scalar_type() != type || (t->stride(1) != 1 && *cols > 1) || (*rows > 1 && st < *cols) ||
        t->get_device() != dev_) {
      wrong(what);
      return nullptr;
    }
    *stride = *rows > 1 ? st : *cols;
    return static_cast<T*>(t->data_ptr());
  }
  // Address and strides of a [tokens, heads, width] tensor with unit inner stride.
  // A stride of 0 is one row for all to torch (an expanded tensor) and contiguous
  // rows to the library: refused, and what the library gets where there is one
  // token or head, whose stride in torch may be anything.
  void* heads(PyObject* o, int64_t tokens, int64_t heads, int64_t width, int64_t* ts, int64_t* hs,
              at::ScalarType* type, const char* what) {
    const at::Tensor* t = tensor(o, what);
    if (t == nullptr) return nullptr;
    if (t->dim() != 3 || t->size(0) != tokens || t->size(1) != heads || t->size(2) != width ||
        t->stride(2) != 1 || (tokens > 1 && t->stride(0) == 0) || (heads > 1 && t->stride(1) == 0) ||
        t->get_device() != dev_) {
      wrong(what);
      return nullptr;
    }
    *ts = tokens > 1 ? t->stride(0) : 0;
    *hs = heads > 1 ? t->stride(1) : 0;
    *type = t->scalar_type();
    return t->data_ptr();
  }
  int64_t number(PyObject* o, int64_t most, const char* what) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      wrong(what);
    } else if (v < INT_MIN || v > most) {
      wrong(what);
    }
    return v;
  }
  // A handle of the library: an address, which None is not.
  template <class T>
  T handle(PyObject* o) {
    void* p = o != Py_None ? PyLong_AsVoidPtr(o) : nullptr;
    if (PyErr_Occurred()) PyErr_Clear();
    if (p == nullptr) wrong("handle is closed");
    return static_cast<T>(p);
  }
  float real(PyObject* o, const char* what) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      wrong(what);
    }
    return (float)v;
  }
  // Positions int32 of `axes` axes for n tokens: [n] or more for one, else [axes, n or
  // more]; the distance between axes.
  const int32_t* positions(PyObject* o, int64_t axes, int64_t n, int64_t* stride) {
    *stride = 0;
    const at::Tensor* t = tensor(o, "positions");
    if (t == nullptr) return nullptr;
    const int64_t dim = t->dim();
    const bool one = dim == 1 && axes == 1;
    if (t->scalar_type() != at::kInt || t->get_device() != dev_ || !(one || (dim == 2 && t->size(0) >= axes)) ||
        t->size(dim - 1) < n || (t->size(dim - 1) > 1 && t->stride(dim - 1) != 1) ||
        (axes > 1 && t->stride(0) < n)) {
      wrong("positions");
      return nullptr;
    }
    *stride = axes > 1 ? t->stride(0) : 0;
    return static_cast<const int32_t*>(t->data_ptr());
  }
  // Address and strides of BF16 heads; rows that do not lie over one another are
  // asked for where they are written.
  void* bf16_heads(PyObject* o, int64_t tokens, int64_t heads, int64_t width, int64_t* ts, int64_t* hs, bool written,
                   const char* what) {
    at::ScalarType type = at::kFloat;
    void* p = this->heads(o, tokens, heads, width, ts, hs, &type, what);
    need(type == at::kBFloat16, what);
    if (written && tokens > 1 && heads > 1) {  // the closer ones in between the others
      const int64_t near = *ts < *hs ? *ts : *hs, far = *ts < *hs ? *hs : *ts, count = *ts < *hs ? tokens : heads;
      need(near >= width && (far - width) / near >= count - 1, what);
    } else if (written) {
      need((tokens <= 1 || *ts >= width) && (heads <= 1 || *hs >= width), what);
    }
    return p;
  }
  int integer(PyObject* o, const char* what) { return (int)number(o, INT_MAX, what); }
  void need(bool ok, const char* what) {
    if (!ok) wrong(what);
  }
  // The stream to launch on: a handle, an object that has one, or the current one.
  void* stream(PyObject* o) {
    if (wrong_ != nullptr) return nullptr;
    if (dev_ < 0 || dev_ != c10::cuda::current_device()) {
      wrong("tensors that are not on the current device");
      return nullptr;
    }
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev_).stream();
    PyObject* h = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
    void* p = h != nullptr ? PyLong_AsVoidPtr(h) : nullptr;
    Py_XDECREF(h);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      wrong("stream");
    }
    return p;
  }
  void wrong(const char* what) {
    if (wrong_ == nullptr) wrong_ = what;
  }
  bool ok() const { return wrong_ == nullptr; }
  PyObject* refusal() const { return PyUnicode_FromString(wrong_); }

 private:
  int64_t dev_ = -1;
  const char* wrong_ = nullptr;
};

// The library call itself, without the interpreter's lock: a launch may wait
// for room in the stream's queue.
template <class F>
PyObject* run(F call) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = call();
  Py_END_ALLOW_THREADS
  if (rc == MLA_OK) Py_RETURN_NONE;
  return PyLong_FromLong(rc);
}

// One entry of the module: `count` arguments, C++ exceptions as Python's.
template <Py_ssize_t COUNT, PyObject* (*BODY)(PyObject* const*)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != COUNT) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", COUNT, n);
    return nullptr;
  }
  try {
    return BODY(a);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

struct Query {
  int64_t tokens = 0, heads = 0, lt = 0, lh = 0, pt = 0, ph = 0;
  void *latent = nullptr, *pe = nullptr;
  const float* inv = nullptr;

  Query(Call& c, PyObject* q_latent, PyObject* q_pe, PyObject* q_scale_inv) {
    const at::Tensor* t = c.tensor(q_latent, "query");
    if (t == nullptr || t->dim() != 3) {
      c.wrong("query shape");
      return;
    }
    tokens = t->size(0);
    heads = t->size(1);
    at::ScalarType lat = at::kFloat, rope = at::kFloat;
    latent = c.heads(q_latent, tokens, heads, 512, &lt, &lh, &lat, "query shape");
    pe = c.heads(q_pe, tokens, heads, 64, &pt, &ph, &rope, "query shape");
    inv = c.flat<const float>(q_scale_inv, at::kFloat, 1, "q_scale_inv");
    const bool codes = lat == at::kByte || lat == at::kFloat8_e4m3fn;
    c.need(lat == rope && (q_scale_inv == Py_None ? lat == at::kBFloat16 : codes), "query type");
    c.need(tokens <= INT_MAX && heads <= INT_MAX, "query shape");
  }
};

struct Cache {
  const void* rows = nullptr;
  int64_t pages = 0;
  int page = 0, layout = 0;
  const float* scale = nullptr;

  Cache(Call& c, PyObject* cache, PyObject* layout_, PyObject* k_scale) {
    int64_t sizes[3];
    rows = c.whole<const void>(cache, at::kByte, 3, sizes, "cache");
    layout = c.integer(layout_, "layout");
    const int64_t bytes = layout == MLA_KV_FP8_DS_MLA ? 656 : layout == MLA_KV_NVFP4_DS_MLA ? 352 : 576;
    c.need(sizes[2] == bytes && sizes[1] <= INT_MAX, "cache");
    pages = sizes[0];
    page = (int)sizes[1];
    scale = c.flat<const float>(k_scale, at::kFloat, layout == MLA_KV_FP8_E4M3_PAGE ? pages : 1, "k_scale");
  }
};

PyObject* tables_step(PyObject* const* a) {
  Call c(a[1]);
  int64_t lens_n[1], table_n[2], pages_n[1], tokens_n[1];
  const char* what = "arrays";
  auto* lens = c.whole<const int32_t>(a[1], at::kInt, 1, lens_n, what);
  auto* table = c.whole<int32_t>(a[2], at::kInt, 2, table_n, "block table");
  auto* pages = c.whole<int32_t>(a[3], at::kInt, 1, pages_n, what);
  const int page = c.integer(a[5], "page size");
  auto* slots = c.whole<int64_t>(a[8], at::kLong, 1, tokens_n, what);
  const int64_t rows = lens_n[0], tokens = tokens_n[0];
  c.need(table_n[0] == rows, "block table");
  c.need(rows <= INT_MAX && tokens <= INT_MAX, what);
  auto* fresh = c.flat<const int32_t>(a[0], at::kInt, rows, what);
  auto* count = c.flat<const int32_t>(a[4], at::kInt, 1, what);
  auto* lens_out = c.flat<int32_t>(a[6], at::kInt, rows, what);
  auto* count_out = c.flat<int32_t>(a[7], at::kInt, 1, what);
  auto* row = c.flat<int32_t>(a[9], at::kInt, tokens, what);
  auto* len = c.flat<int32_t>(a[10], at::kInt, tokens, what);
  auto* cu = c.flat<int32_t>(a[11], at::kInt, rows + 1, what);
  auto* flags = c.flat<unsigned>(a[12], at::kInt, 1, "flags");
  void* stream = c.stream(a[13]);
  if (!c.ok()) return c.refusal();
  return run([&] { return tables_step_c((int)rows, fresh, lens, lens_out, table, table_n[1], pages, count, count_out,
                              pages_n[0], page, (int)tokens, slots, row, len, cu, flags, stream); });
}

PyObject* blocks_mean(PyObject* const* a) {
  Call c(a[0]);
  const Cache k(c, a[0], a[1], a[2]);
  int64_t stride, table_rows, width, rows_n[1];
  auto* table = c.rows<const int32_t>(a[3], at::kInt, &stride, &table_rows, &width, "block table");
  auto* to = c.whole<const int32_t>(a[5], at::kInt, 1, rows_n, "lengths");
  const int64_t rows = rows_n[0];
  c.need(table_rows >= rows && rows <= INT_MAX, "block table");
  auto* from = c.flat<const int32_t>(a[4], at::kInt, rows, "lengths");
  void* mean = c.flat(a[6], at::kBFloat16, k.pages * 576, "mean");
  auto* flags = c.flat<unsigned>(a[7], at::kInt, 1, "flags");
  void* stream = c.stream(a[8]);
  if (!c.ok()) return c.refusal();
  return run([&] { return blocks_mean_c(k.rows, k.pages, k.page, k.layout, k.scale, table, stride, width, (int)rows, from, to,
                              mean, flags, stream); });
}

PyObject* blocks_score(PyObject* const* a) {
  Call c(a[0]);
  const Query q(c, a[0], a[1], a[7]);
  int64_t mean_n[2], table_n[2], stride, rows, cols;
  void* mean = c.whole(a[2], at::kBFloat16, 2, mean_n, "mean");
  c.need(mean_n[1] == 576, "mean");
  const int page = c.integer(a[3], "page size");
  auto* table = c.whole<const int32_t>(a[4], at::kInt, 2, table_n, "block table");
  auto* lens = c.flat<const int32_t>(a[5], at::kInt, q.tokens, "lengths");
  auto* scores = c.rows<float>(a[6], at::kFloat, &stride, &rows, &cols, "scores");
  c.need(rows >= q.tokens && cols >= table_n[1], "scores");
  auto* token_row = c.flat<const int32_t>(a[8], at::kInt, q.tokens, "token_row");
  c.need(table_n[0] <= INT_MAX, "block table");
  auto* flags = c.flat<unsigned>(a[9], at::kInt, 1, "flags");
  void* stream = c.stream(a[10]);
  if (!c.ok()) return c.refusal();
  return run([&] { return blocks_score_c((int)q.tokens, (int)q.heads, q.latent, q.lt, q.lh, q.pe, q.pt, q.ph, q.inv,
                               mean, mean_n[0], page, table, table_n[1], (int)table_n[0], token_row, lens,
                               scores, stride, flags, stream); });
}

PyObject* blocks_select(PyObject* const* a) {
  Call c(a[0]);
  int64_t stride, rows, blocks, out_stride, tokens, k;
  auto* scores = c.rows<const float>(a[0], at::kFloat, &stride, &rows, &blocks, "scores");
  auto* sel = c.rows<int32_t>(a[5], at::kInt, &out_stride, &tokens, &k, "sel");
  c.need(rows >= tokens && tokens <= INT_MAX && blocks <= INT_MAX, "scores");
  c.need(k <= INT_MAX, "sel");
  auto* lens = c.flat<const int32_t>(a[1], at::kInt, tokens, "lengths");
  const int page = c.integer(a[2], "page size");
  const int first = c.integer(a[3], "keep_first"), last = c.integer(a[4], "keep_last");
  auto* count = c.flat<int32_t>(a[6], at::kInt, tokens, "sel_count");
  void* stream = c.stream(a[7]);
  if (!c.ok()) return c.refusal();
  return run([&] { return blocks_select_c((int)tokens, scores, stride, (int)blocks, lens, page, first, last, (int)k, sel,
                                out_stride, count, stream); });
}

PyObject* attn_decode(PyObject* const* a) {
  Call c(a[2]);
  c.need(a[0] != Py_None, "handle is closed");
  auto handle = a[0] != Py_None ? static_cast<mla_attn_t>(PyLong_AsVoidPtr(a[0])) : nullptr;
  if (PyErr_Occurred()) return nullptr;
  const Query q(c, a[2], a[3], a[10]);
  c.need(q.heads == c.number(a[1], INT_MAX, "heads"), "heads");
  const Cache k(c, a[4], a[5], a[9]);
  int64_t stride, table_rows, width, sel_stride = 0, sel_rows = 0, sel_cols = 0, ot = 0, oh = 0;
  auto* table = c.rows<const int32_t>(a[6], at::kInt, &stride, &table_rows, &width, "block table");
  c.need(table_rows <= INT_MAX, "block table");
  auto* lens = c.flat<const int32_t>(a[7], at::kInt, q.tokens, "lengths");
  const double scale = PyFloat_AsDouble(a[8]);
  if (PyErr_Occurred()) return nullptr;
  auto* token_row = c.flat<const int32_t>(a[11], at::kInt, q.tokens, "token_row");
  const int32_t* sel = nullptr;
  if (a[12] != Py_None) {
    sel = c.rows<const int32_t>(a[12], at::kInt, &sel_stride, &sel_rows, &sel_cols, "sel");
    c.need(sel_rows >= q.tokens, "sel");
  }
  auto* sel_count = c.flat<const int32_t>(a[13], at::kInt, q.tokens, "sel_count");
  at::ScalarType type = at::kFloat;
  void* out = c.heads(a[14], q.tokens, q.heads, 512, &ot, &oh, &type, "out");
  c.need(type == at::kBFloat16, "out");
  // rows that do not lie over one another: the closer ones in between the others
  const int64_t near = ot < oh ? ot : oh, far = ot < oh ? oh : ot;
  const int64_t count = ot < oh ? q.tokens : q.heads;
  c.need(q.tokens <= 1 || q.heads <= 1 || (near >= 512 && (far - 512) / near >= count - 1), "out");
  auto* lse = c.flat<float>(a[15], at::kFloat, q.tokens * q.heads, "lse");
  void* stream = c.stream(a[16]);
  if (!c.ok()) return c.refusal();
  return run([&] { return attn_decode_c(handle, (int)q.tokens, q.latent, q.lt, q.lh, q.pe, q.pt, q.ph, q.inv, k.rows,
                              k.pages, k.page, k.layout, k.scale, table, stride, width, (int)table_rows, token_row,
                              lens, sel, sel_stride, sel_cols, sel_count, (float)scale, out, ot, oh, lse, stream); });
}

PyObject* rope_apply(PyObject* const* a) {
  Call c(a[2]);
  auto rope = c.handle<mla_rope_t>(a[0]);
  const at::Tensor* t = c.tensor(a[2], "x");
  c.need(t != nullptr && t->dim() == 3, "x");
  if (!c.ok()) return c.refusal();
  const int64_t tokens = t->size(0), heads = t->size(1);
  int64_t xt, xh, ot, oh, ps;
  void* x = c.bf16_heads(a[2], tokens, heads, 64, &xt, &xh, false, "x");
  void* out = c.bf16_heads(a[5], tokens, heads, 64, &ot, &oh, true, "out");
  c.need(heads <= INT_MAX, "x");
  auto* pos = c.positions(a[3], c.number(a[1], INT_MAX, "axes"), tokens, &ps);
  const int64_t offset = c.number(a[4], INT_MAX, "offset");
  void* stream = c.stream(a[6]);
  if (!c.ok()) return c.refusal();
  return run([&] { return rope_apply_c(rope, tokens, (int)heads, x, xt, xh, pos, ps, offset, out, ot, oh, stream); });
}

PyObject* cache_write(PyObject* const* a) {
  Call c(a[0]);
  int64_t ks, kr, kc, ps, pr, pc, slots_n[1], pos_stride = 0, rs = 0, rr, rc;
  void* kv = c.rows(a[0], at::kBFloat16, &ks, &kr, &kc, "kv_c");
  void* pe = c.rows(a[1], at::kBFloat16, &ps, &pr, &pc, "k_pe");
  auto* slots = c.whole<const int64_t>(a[2], at::kLong, 1, slots_n, "slots");
  const int64_t tokens = slots_n[0];
  c.need(kc == 512 && kr >= tokens, "kv_c");
  c.need(pc == 64 && pr >= tokens, "k_pe");
  const Cache k(c, a[3], a[4], a[5]);
  void* gamma = c.flat(a[6], at::kBFloat16, 512, "gamma");
  const float eps = c.real(a[7], "eps");
  mla_rope_t rope = nullptr;
  const int32_t* pos = nullptr;
  if (a[8] != Py_None || a[10] != Py_None) {
    rope = c.handle<mla_rope_t>(a[8]);
    pos = c.positions(a[10], c.number(a[9], INT_MAX, "axes"), tokens, &pos_stride);
  }
  const int64_t offset = c.number(a[11], INT_MAX, "offset");
  void* rows = nullptr;
  if (a[12] != Py_None) {
    rows = c.rows(a[12], at::kBFloat16, &rs, &rr, &rc, "rows");
    c.need(rc == 576 && rr >= tokens, "rows");
  }
  auto* flags = c.flat<unsigned>(a[13], at::kInt, 1, "flags");
  void* stream = c.stream(a[14]);
  if (!c.ok()) return c.refusal();
  return run([&] { return cache_write_c(tokens, kv, ks, pe, ps, gamma, eps, rope, pos, pos_stride, offset, slots,
                              const_cast<void*>(k.rows), k.pages, k.page, k.layout, k.scale, rows, rs, flags, stream); });
}

PyObject* cache_read(PyObject* const* a) {
  Call c(a[0]);
  const Cache k(c, a[0], a[1], a[2]);
  int64_t stride, table_rows, width, cu_n[1], rs, rr, rc;
  auto* table = c.rows<const int32_t>(a[3], at::kInt, &stride, &table_rows, &width, "block table");
  auto* cu = c.whole<const int32_t>(a[4], at::kInt, 1, cu_n, "cu_rows");
  const int64_t requests = cu_n[0] - 1;
  c.need(requests >= 1 && requests <= INT_MAX, "cu_rows");
  c.need(table_rows >= requests, "block table");
  void* rows = c.rows(a[5], at::kBFloat16, &rs, &rr, &rc, "rows");
  c.need(rc == 576, "rows");
  auto* first = c.flat<const int32_t>(a[6], at::kInt, requests, "first");
  auto* flags = c.flat<unsigned>(a[7], at::kInt, 1, "flags");
  void* stream = c.stream(a[8]);
  if (!c.ok()) return c.refusal();
  return run([&] { return cache_read_c(k.rows, k.pages, k.page, k.layout, k.scale, table, stride, width, (int)requests, cu,
                             first, rr, rows, rs, flags, stream); });
}

PyObject* prompt_attn(PyObject* const* a) {
  Call c(a[2]);
  auto handle = c.handle<mla_prompt_t>(a[0]);
  const int64_t heads = c.number(a[1], INT_MAX, "heads");
  const at::Tensor *q = c.tensor(a[2], "queries"), *key = c.tensor(a[4], "keys");
  c.need(q != nullptr && q->dim() == 3, "queries");
  c.need(key != nullptr && key->dim() == 3, "keys");
  if (!c.ok()) return c.refusal();
  const int64_t tq = q->size(0), tk = key->size(0);
  int64_t qnt, qnh, qpt, qph, knt, knh, vt, vh, ot, oh, pes, per, pec, cu_n[1];
  void* qn = c.bf16_heads(a[2], tq, heads, 128, &qnt, &qnh, false, "queries");
  void* qp = c.bf16_heads(a[3], tq, heads, 64, &qpt, &qph, false, "queries");
  void* kn = c.bf16_heads(a[4], tk, heads, 128, &knt, &knh, false, "keys");
  void* kp = c.rows(a[5], at::kBFloat16, &pes, &per, &pec, "k_pe");
  c.need(pec == 64 && per == tk, "k_pe");
  void* v = c.bf16_heads(a[6], tk, heads, 128, &vt, &vh, false, "values");
  auto* cu_q = c.whole<const int32_t>(a[7], at::kInt, 1, cu_n, "cu_q");
  const int64_t docs = cu_n[0] - 1;
  c.need(docs >= 1 && docs <= INT_MAX, "cu_q");
  auto* cu_k = a[8] == Py_None ? cu_q : c.flat<const int32_t>(a[8], at::kInt, docs + 1, "cu_k");
  const int causal = PyObject_IsTrue(a[9]);
  if (causal < 0) return nullptr;
  auto* prefix = c.flat<const int32_t>(a[10], at::kInt, docs, "prefix");
  const float scale = c.real(a[11], "softmax_scale"), cap = c.real(a[12], "softcap");
  auto* slopes = c.flat<const float>(a[13], at::kFloat, heads, "slopes");
  void* out = c.bf16_heads(a[14], tq, heads, 128, &ot, &oh, true, "out");
  auto* lse = c.flat<float>(a[15], at::kFloat, tq * heads, "lse");
  void* stream = c.stream(a[16]);
  if (!c.ok()) return c.refusal();
  return run([&] { return prompt_attn_c(handle, (int)docs, tq, tk, qn, qnt, qnh, qp, qpt, qph, kn, knt, knh, kp, pes, v, vt,
                              vh, cu_q, cu_k, causal, prefix, scale, cap, slopes, out, ot, oh, lse, stream); });
}

PyObject* bind(PyObject* const* a) {
  void* p[9];
  for (int i = 0; i < 9; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  tables_step_c = reinterpret_cast<decltype(tables_step_c)>(p[0]);
  blocks_mean_c = reinterpret_cast<decltype(blocks_mean_c)>(p[1]);
  blocks_score_c = reinterpret_cast<decltype(blocks_score_c)>(p[2]);
  blocks_select_c = reinterpret_cast<decltype(blocks_select_c)>(p[3]);
  attn_decode_c = reinterpret_cast<decltype(attn_decode_c)>(p[4]);
  rope_apply_c = reinterpret_cast<decltype(rope_apply_c)>(p[5]);
  cache_write_c = reinterpret_cast<decltype(cache_write_c)>(p[6]);
  cache_read_c = reinterpret_cast<decltype(cache_read_c)>(p[7]);
  prompt_attn_c = reinterpret_cast<decltype(prompt_attn_c)>(p[8]);
  Py_RETURN_NONE;
}

template <Py_ssize_t COUNT, PyObject* (*BODY)(PyObject* const*)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<COUNT, BODY>)), METH_FASTCALL,
          nullptr};
}

PyMethodDef methods[] = {
    method<9, bind>("bind"),
    method<14, tables_step>("tables_step"),
    method<9, blocks_mean>("blocks_mean"),
    method<11, blocks_score>("blocks_score"),
    method<8, blocks_select>("blocks_select"),
    method<17, attn_decode>("attn_decode"),
    method<7, rope_apply>("rope_apply"),
    method<15, cache_write>("cache_write"),
    method<9, cache_read>("cache_read"),
    method<17, prompt_attn>("prompt_attn"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_calls() { return PyModule_Create(&module); }
