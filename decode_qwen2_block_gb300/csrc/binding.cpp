// The paged calls from torch tensors: checks of type, device, shape and layout, and
// the call of the library, in one step.  A serving step makes several of these
// calls on a few rows; checked in Python, array by array, and passed through
// ctypes, plan and append took 7.4 us each for kernels of 4 and 2.
//
// The library is the one that the package has loaded: bind() takes its functions'
// addresses, nothing here links to a library of its own.
//
// Every function returns None or raises BlkError.  `stream` is None (the current
// stream of the block's device) or a stream's handle.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/blk.h"

namespace {

struct Refused {};   // a Python exception is set

struct {             // the loaded library's functions
  decltype(&blk_page_plan) page_plan;
  decltype(&blk_page_append) page_append;
  decltype(&blk_attn_paged) attn_paged;
  decltype(&blk_page_append_kv8) page_append_kv8;
  decltype(&blk_page_read_kv8) page_read_kv8;
  decltype(&blk_attn_paged_kv8) attn_paged_kv8;
} lib = {};

[[noreturn]] void refuse(int status, const std::string& what) {
  PyObject* mod = PyImport_ImportModule("decode_qwen2_block_gb300");
  PyObject* cls = mod ? PyObject_GetAttrString(mod, "BlkError") : nullptr;
  PyObject* err = cls ? PyObject_CallFunction(cls, "is", status, what.c_str()) : nullptr;
  if (err) PyErr_SetObject(cls, err);
  Py_XDECREF(err);
  Py_XDECREF(cls);
  Py_XDECREF(mod);
  throw Refused();
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: a tensor is wanted, not %s", what, Py_TYPE(o)->tp_name);
    throw Refused();
  }
  return THPVariable_Unpack(o);
}

// A tensor that the library reads or writes by its raw pointer: of this type and
// shape, on the block's GPU, and contiguous unless the caller looks at its strides.
const at::Tensor& checked(PyObject* o, const char* what, at::ScalarType type, int64_t device,
                          at::IntArrayRef shape, bool contiguous = true,
                          int status = BLK_ERR_SHAPE) {
  const at::Tensor& t = tensor(o, what);
  if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != device || t.sizes() != shape ||
      (contiguous && !t.is_contiguous())) {
    std::ostringstream s;
    s << what << ": " << t.sizes() << " " << t.scalar_type() << " on " << t.device();
    refuse(status, s.str());
  }
  return t;
}

// The stride of dimension i; of one of size 1, which steps nowhere and may have any, `plain`.
int64_t stride_of(const at::Tensor& t, int i, int64_t plain) {
  return t.size(i) == 1 ? plain : t.stride(i);
}

const at::Tensor& workspace(PyObject* o, int64_t device) {
  const at::Tensor& t = tensor(o, "ws");
  if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous()) {
    std::ostringstream s;
    s << "workspace " << t.sizes() << " on " << t.device();
    refuse(BLK_ERR_WORKSPACE, s.str());
  }
  return t;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
void* handle_of(PyObject* o) { return o == Py_None ? nullptr : reinterpret_cast<void*>(integer(o)); }

void* stream_of(PyObject* o, int64_t device) {
  return o == Py_None ? static_cast<void*>(c10::cuda::getCurrentCUDAStream(device).stream())
                      : reinterpret_cast<void*>(integer(o));
}

// The block as its methods pass it: (handle, device, n_heads, n_kv_heads, head_dim).
struct BlockArgs {
  blk_handle h;
  int64_t device, heads, kv_heads, dim;
  explicit BlockArgs(PyObject* o) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 5) {
      PyErr_SetString(PyExc_TypeError, "block");
      throw Refused();
    }
    h = static_cast<blk_handle>(handle_of(PyTuple_GET_ITEM(o, 0)));
    device = integer(PyTuple_GET_ITEM(o, 1));
    heads = integer(PyTuple_GET_ITEM(o, 2));
    kv_heads = integer(PyTuple_GET_ITEM(o, 3));
    dim = integer(PyTuple_GET_ITEM(o, 4));
  }
};

struct Pools {
  const at::Tensor &k, &v;
  Pools(const BlockArgs& b, PyObject* ko, PyObject* vo)
      : k(tensor(ko, "k_pages")), v(tensor(vo, "v_pages")) {
    const auto shape = k.sizes();
    if (shape.size() != 4 || shape[1] != b.kv_heads || shape[3] != b.dim) {
      std::ostringstream s;
      s << "k_pages: " << shape;
      refuse(BLK_ERR_SHAPE, s.str());
    }
    checked(ko, "k_pages", at::kHalf, b.device, shape);
    checked(vo, "v_pages", at::kHalf, b.device, shape);
  }
  int64_t n_pages() const { return k.size(0); }
  int64_t page() const { return k.size(2); }
};

// The codes and scales of an 8-bit cache: a[0 .. 3] are k_pages, v_pages, k_scales, v_scales.
struct Pools8 {
  blk_kv8_pool pool;
  int64_t n_pages, page;
  Pools8(const BlockArgs& b, PyObject* const* a) {
    const at::Tensor& k = tensor(a[0], "k_pages");
    const auto shape = k.sizes();
    if (shape.size() != 4 || shape[1] != b.kv_heads || shape[3] != b.dim) {
      std::ostringstream s;
      s << "k_pages: " << shape;
      refuse(BLK_ERR_SHAPE, s.str());
    }
    n_pages = shape[0];
    page = shape[2];
    const int64_t scales[4] = {n_pages, b.kv_heads, page, b.dim / 32};
    pool.k = checked(a[0], "k_pages", at::kByte, b.device, shape).data_ptr();
    pool.v = checked(a[1], "v_pages", at::kByte, b.device, shape).data_ptr();
    pool.k_scale = checked(a[2], "k_scales", at::kFloat8_e5m2, b.device, scales).data_ptr();
    pool.v_scale = checked(a[3], "v_scales", at::kFloat8_e5m2, b.device, scales).data_ptr();
  }
};

// Rows of K and V [rows, kv_heads, dim] in fp16 with the same strides, the last dimension
// contiguous.
struct Rows {
  void *k, *v;
  int64_t row_stride, head_stride;
  Rows(const BlockArgs& b, int64_t rows, PyObject* ko, PyObject* vo, const char* what) {
    const at::Tensor& kt = checked(ko, "k", at::kHalf, b.device, {rows, b.kv_heads, b.dim}, false);
    const at::Tensor& vt = checked(vo, "v", at::kHalf, b.device, {rows, b.kv_heads, b.dim}, false);
    row_stride = stride_of(kt, 0, b.kv_heads * b.dim);
    head_stride = stride_of(kt, 1, b.dim);
    if (stride_of(vt, 0, b.kv_heads * b.dim) != row_stride ||
        stride_of(vt, 1, b.dim) != head_stride || kt.stride(2) != 1 || vt.stride(2) != 1)
      refuse(BLK_ERR_SHAPE, std::string(what) + ": strides");
    k = kt.data_ptr();
    v = vt.data_ptr();
  }
};

// A ctypes structure's bytes.
struct Batch {
  Py_buffer view;
  explicit Batch(PyObject* o) {
    if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE)) throw Refused();
    if (view.len != (Py_ssize_t)sizeof(blk_paged_batch)) {
      PyBuffer_Release(&view);
      PyErr_SetString(PyExc_TypeError, "batch: a BlkPagedBatch is wanted");
      throw Refused();
    }
  }
  ~Batch() { PyBuffer_Release(&view); }
  Batch(const Batch&) = delete;
  const blk_paged_batch& get() const { return *static_cast<const blk_paged_batch*>(view.buf); }
};

// Runs f with n arguments given; C++ exceptions become Python's.
template <typename F>
PyObject* call(Py_ssize_t given, Py_ssize_t wanted, const char* what, F f) {
  if (given != wanted) return PyErr_Format(PyExc_TypeError, "%s: %zd arguments", what, wanted);
  try {
    const int rc = f();
    if (rc != BLK_OK) refuse(rc, what);
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  Py_RETURN_NONE;
}

template <typename F>
void need_library(F f) {
  if (f) return;
  PyErr_SetString(PyExc_RuntimeError, "_native: no library is bound");
  throw Refused();
}

struct NoGil {       // the library's call may wait for room in the stream's queue
  PyThreadState* s = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(s); }
};

PyObject* page_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 11, "blk_page_plan", [&] {
    const BlockArgs b(a[0]);
    const int64_t page = integer(a[1]);
    const int64_t B = tensor(a[2], "cache_lens").numel(), rows = tensor(a[7], "slot_map").numel();
    const auto vec = [&](int i, const char* what, int64_t k) {
      return checked(a[i], what, at::kLong, b.device, {k}).data_ptr<int64_t>();
    };
    const int64_t* lens = vec(2, "cache_lens", B);
    const int64_t* news = a[3] == Py_None ? nullptr : vec(3, "new_lens", B);
    const int64_t n_free = tensor(a[4], "free_pages").numel();
    const int32_t* free_pages =
        checked(a[4], "free_pages", at::kInt, b.device, {n_free}).data_ptr<int32_t>();
    const at::Tensor& table = tensor(a[5], "block_table");
    const int64_t blocks = table.dim() == 2 ? table.size(1) : 0;
    checked(a[5], "block_table", at::kInt, b.device, {B, blocks});
    int64_t* start = vec(6, "row_start", B + 1);
    int64_t* slots = vec(7, "slot_map", rows);
    int64_t* pos = vec(8, "pos", rows);
    int64_t* used = vec(9, "used", 1);
    int32_t* tab = table.data_ptr<int32_t>();
    void* s = stream_of(a[10], b.device);
    if (page != (int32_t)page) return (int)BLK_ERR_SHAPE;
    need_library(lib.page_plan);
    NoGil g;
    return lib.page_plan(b.h, (int32_t)page, B, lens, news, free_pages, n_free, tab, blocks, rows,
                         start, slots, pos, used, s);
  });
}

PyObject* page_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 7, "blk_page_append", [&] {
    const BlockArgs b(a[0]);
    const Pools p(b, a[4], a[5]);
    const int64_t rows = tensor(a[3], "slot_map").numel();
    const int64_t* slots = checked(a[3], "slot_map", at::kLong, b.device, {rows}).data_ptr<int64_t>();
    const at::Tensor& k = checked(a[1], "k", at::kHalf, b.device, {rows, b.kv_heads, b.dim}, false);
    const at::Tensor& v = checked(a[2], "v", at::kHalf, b.device, {rows, b.kv_heads, b.dim}, false);
    const int64_t rs = stride_of(k, 0, b.kv_heads * b.dim), hs = stride_of(k, 1, b.dim);
    if (stride_of(v, 0, b.kv_heads * b.dim) != rs || stride_of(v, 1, b.dim) != hs ||
        k.stride(2) != 1 || v.stride(2) != 1)
      refuse(BLK_ERR_SHAPE, "page_append: strides");
    const void *kp = k.data_ptr(), *vp = v.data_ptr();
    void *kt = p.k.data_ptr(), *vt = p.v.data_ptr(), *s = stream_of(a[6], b.device);
    need_library(lib.page_append);
    NoGil g;
    return lib.page_append(b.h, kp, vp, rs, hs, slots, rows, (int32_t)p.page(), p.n_pages(), kt, vt,
                           s);
  });
}

PyObject* attn_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 8, "blk_attn_paged", [&] {
    const BlockArgs b(a[0]);
    const Batch batch(a[1]);
    const blk_paged_batch& d = batch.get();
    const Pools p(b, a[3], a[4]);
    if (p.n_pages() != d.n_pages || p.page() != d.page_size)
      refuse(BLK_ERR_SHAPE, "the pools are not those of the batch");
    const at::Tensor& q = checked(a[2], "q", at::kHalf, b.device, {d.n_rows, b.heads, b.dim}, false);
    const at::Tensor& o = checked(a[5], "out", at::kHalf, b.device, {d.n_rows, b.heads, b.dim}, false);
    for (const at::Tensor* t : {&q, &o})
      if (stride_of(*t, 1, b.dim) != b.dim || t->stride(2) != 1)
        refuse(BLK_ERR_SHAPE, "attn_paged: a row's heads must be contiguous");
    const at::Tensor& ws = workspace(a[6], b.device);
    const int64_t width = b.heads * b.dim, qs = stride_of(q, 0, width), os = stride_of(o, 0, width);
    const void *qp = q.data_ptr(), *kp = p.k.data_ptr(), *vp = p.v.data_ptr();
    void *op = o.data_ptr(), *wp = ws.data_ptr(), *s = stream_of(a[7], b.device);
    const size_t bytes = ws.nbytes();
    need_library(lib.attn_paged);
    NoGil g;
    return lib.attn_paged(b.h, &d, qp, qs, kp, vp, op, os, wp, bytes, s);
  });
}

PyObject* page_append_kv8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 9, "blk_page_append_kv8", [&] {
    const BlockArgs b(a[0]);
    const Pools8 p(b, a + 4);
    const int64_t rows = tensor(a[3], "slot_map").numel();
    const int64_t* slots = checked(a[3], "slot_map", at::kLong, b.device, {rows}).data_ptr<int64_t>();
    const Rows r(b, rows, a[1], a[2], "page_append_kv8");
    void* s = stream_of(a[8], b.device);
    need_library(lib.page_append_kv8);
    NoGil g;
    return lib.page_append_kv8(b.h, r.k, r.v, r.row_stride, r.head_stride, slots, rows,
                               (int32_t)p.page, p.n_pages, &p.pool, s);
  });
}

PyObject* page_read_kv8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 9, "blk_page_read_kv8", [&] {
    const BlockArgs b(a[0]);
    const Pools8 p(b, a + 2);
    const int64_t rows = tensor(a[1], "slot_map").numel();
    const int64_t* slots = checked(a[1], "slot_map", at::kLong, b.device, {rows}).data_ptr<int64_t>();
    const Rows r(b, rows, a[6], a[7], "page_read_kv8");
    void* s = stream_of(a[8], b.device);
    need_library(lib.page_read_kv8);
    NoGil g;
    return lib.page_read_kv8(b.h, slots, rows, (int32_t)p.page, p.n_pages, &p.pool, r.k, r.v,
                             r.row_stride, r.head_stride, s);
  });
}

PyObject* attn_paged_kv8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 10, "blk_attn_paged_kv8", [&] {
    const BlockArgs b(a[0]);
    const Batch batch(a[1]);
    const blk_paged_batch& d = batch.get();
    const Pools8 p(b, a + 3);
    if (p.n_pages != d.n_pages || p.page != d.page_size)
      refuse(BLK_ERR_SHAPE, "the pools are not those of the batch");
    const at::Tensor& q = checked(a[2], "q", at::kHalf, b.device, {d.n_rows, b.heads, b.dim}, false);
    const at::Tensor& o = checked(a[7], "out", at::kHalf, b.device, {d.n_rows, b.heads, b.dim}, false);
    for (const at::Tensor* t : {&q, &o})
      if (stride_of(*t, 1, b.dim) != b.dim || t->stride(2) != 1)
        refuse(BLK_ERR_SHAPE, "attn_paged_kv8: a row's heads must be contiguous");
    const at::Tensor& ws = workspace(a[8], b.device);
    const int64_t width = b.heads * b.dim, qs = stride_of(q, 0, width), os = stride_of(o, 0, width);
    const void* qp = q.data_ptr();
    void *op = o.data_ptr(), *wp = ws.data_ptr(), *s = stream_of(a[9], b.device);
    const size_t bytes = ws.nbytes();
    need_library(lib.attn_paged_kv8);
    NoGil g;
    return lib.attn_paged_kv8(b.h, &d, qp, qs, &p.pool, op, os, wp, bytes, s);
  });
}

// bind(page_plan, page_append, attn_paged[, page_append_kv8, page_read_kv8, attn_paged_kv8]):
// the functions' addresses.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* f[6] = {};
  if (n != 3 && n != 6) return PyErr_Format(PyExc_TypeError, "bind: 3 or 6 arguments");
  for (int i = 0; i < n; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (!f[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null address");
      return nullptr;
    }
  }
  lib.page_plan = reinterpret_cast<decltype(lib.page_plan)>(f[0]);
  lib.page_append = reinterpret_cast<decltype(lib.page_append)>(f[1]);
  lib.attn_paged = reinterpret_cast<decltype(lib.attn_paged)>(f[2]);
  lib.page_append_kv8 = reinterpret_cast<decltype(lib.page_append_kv8)>(f[3]);
  lib.page_read_kv8 = reinterpret_cast<decltype(lib.page_read_kv8)>(f[4]);
  lib.attn_paged_kv8 = reinterpret_cast<decltype(lib.attn_paged_kv8)>(f[5]);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL
PyMethodDef methods[] = {
    {"bind", FAST(bind),
     "(page_plan, page_append, attn_paged[, page_append_kv8, page_read_kv8, attn_paged_kv8]): the "
     "library's functions"},
    {"page_plan", FAST(page_plan),
     "(block, page_size, cache_lens, new_lens, free_pages, block_table, row_start, slot_map, pos, "
     "used, stream)"},
    {"page_append", FAST(page_append), "(block, k, v, slot_map, k_pages, v_pages, stream)"},
    {"attn_paged", FAST(attn_paged), "(block, batch, q, k_pages, v_pages, out, ws, stream)"},
    {"page_append_kv8", FAST(page_append_kv8),
     "(block, k, v, slot_map, k_pages, v_pages, k_scales, v_scales, stream)"},
    {"page_read_kv8", FAST(page_read_kv8),
     "(block, slot_map, k_pages, v_pages, k_scales, v_scales, k, v, stream)"},
    {"attn_paged_kv8", FAST(attn_paged_kv8),
     "(block, batch, q, k_pages, v_pages, k_scales, v_scales, out, ws, stream)"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", "The paged calls from torch tensors.", -1,
                      methods};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
