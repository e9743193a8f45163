// The paged-cache operators of include/mk.h on torch tensors: the extension module behind
// paged.py.  It checks tensors (ValueError), fills the C structures, takes outputs and
// workspaces from torch's allocator and calls libmk.so on the current stream; a C status
// other than MK_OK raises the package's MkError.  It is compiled because these calls are
// short: one takes 2 to 10 us on the GPU, the same steps in Python took 31 to 42 us on the
// host.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/core/TensorImpl.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "mk.h"

namespace {

PyObject* g_error = nullptr;  // MkError

struct Refused {};  // a Python exception is set

[[noreturn]] void value_error(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Refused();
}
void need(bool ok, const char* what) {
  if (!ok) value_error(what);
}

void check(mk_status s, const char* where) {
  if (s == MK_OK) return;
  PyObject* args = Py_BuildValue("(is)", (int)s, where);
  if (args) PyErr_SetObject(g_error ? g_error : PyExc_RuntimeError, args);
  Py_XDECREF(args);
  throw Refused();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) value_error(std::string(name) + " must be a tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.layout() != at::kStrided) value_error(std::string(name) + " must be a dense tensor");
  if (t.is_neg()) value_error(std::string(name) + " must not be a negated view (resolve_neg())");
  if (t.requires_grad() && c10::GradMode::is_enabled())
    value_error(std::string(name) + " requires a gradient, and none is recorded here (torch.no_grad())");
  if (t._fw_grad(0).defined() && c10::AutogradState::get_tls_state().get_fw_grad_mode())
    value_error(std::string(name) + " has a forward-mode tangent, and none is computed here");
  return t;
}
// A tensor that the call writes in place counts as changed, as after torch's own operators (one
// of inference mode has no count)
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void written(PyObject* o) {
  if (o != Py_None) written(THPVariable_Unpack(o));
}
template <typename... Objects>
void written(PyObject* o, Objects... more) {
  written(o);
  written(more...);
}
const at::Tensor& on_gpu(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor");
  return t;
}
void same_device(const at::Tensor& t, at::Device dev, const char* name) {
  if (t.device() != dev) value_error(std::string(name) + " must be on " + dev.str());
}

int dtype_of(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kHalf: return MK_F16;
    case at::kBFloat16: return MK_BF16;
    case at::kFloat: return MK_F32;
    default: value_error(std::string(name) + " must be float16, bfloat16 or float32");
  }
}

// a contiguous int32 tensor of one or two dims, or NULL for None where that is allowed
int32_t* int32s(PyObject* o, const char* name, at::Device dev, int64_t n, int64_t m = -1, bool none = false) {
  if (none && o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  const bool shape = m < 0 ? t.dim() == 1 && t.size(0) == n : t.dim() == 2 && t.size(0) == n && t.size(1) == m;
  if (t.scalar_type() != at::kInt || t.device() != dev || !shape || !t.is_contiguous())
    value_error(std::string(name) + " must be a contiguous int32 tensor of " +
                (m < 0 ? std::to_string(n) : std::to_string(n) + " x " + std::to_string(m)) + " on " + dev.str());
  return t.data_ptr<int32_t>();
}
int32_t* status_of(PyObject* o, at::Device dev) { return int32s(o, "status", dev, 4, -1, true); }

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Refused();
  return x;
}
int integer(PyObject* o, const char* name) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Refused();
  if (x < INT32_MIN || x > INT32_MAX) value_error(std::string(name) + " is out of range");
  return (int)x;
}
int size32(int64_t n, const char* name) {
  if (n > INT32_MAX) value_error(std::string(name) + " is too large");
  return (int)n;
}

void* stream_of(at::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// a call's workspace: released to torch's allocator when the call returns, so the next taker
// on the same stream runs after it (in a capture the memory belongs to that graph's pool)
struct Workspace {
  c10::DataPtr p;
  explicit Workspace(size_t bytes) : p(c10::cuda::CUDACachingAllocator::get()->allocate(bytes)) {}
};

// New contiguous tensors of one allocation, without the dispatcher's part of at::empty
struct Fresh {
  c10::Storage storage;
  at::Device dev;
  int64_t at = 0;
  Fresh(int64_t bytes, at::Device d) : dev(d) {
    c10::Allocator* a = c10::cuda::CUDACachingAllocator::get();
    storage = c10::Storage(c10::Storage::use_byte_size_t(), bytes, a->allocate(bytes), a, /*resizable=*/false);
  }
  at::Tensor take(at::IntArrayRef sizes, at::ScalarType type) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(storage), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                            c10::scalarTypeToTypeMeta(type));
    const int64_t e = (int64_t)t.dtype().itemsize();
    t.unsafeGetTensorImpl()->set_storage_offset(at / e);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
    at += t.numel() * e;
    return t;
  }
  static at::Tensor one(at::IntArrayRef sizes, at::ScalarType type, at::Device d) {
    int64_t n = (int64_t)c10::elementSize(type);
    for (int64_t s : sizes) n *= s;
    return Fresh(n, d).take(sizes, type);
  }
};

void table_of(PyObject* o, at::Device dev, int32_t** p, int* rows, int* width, long long* stride) {
  const at::Tensor& t = tensor(o, "table");
  if (t.scalar_type() != at::kInt || t.device() != dev || t.dim() != 2 || (t.stride(1) != 1 && t.size(1) != 1))
    value_error("table must be an int32 [rows, pages] tensor on the pages' device");
  *p = t.data_ptr<int32_t>();
  *rows = size32(t.size(0), "table");
  *width = size32(t.size(1), "table");
  *stride = t.size(0) > 1 ? t.stride(0) : t.size(1);
}

// keys and values: `dims` dims, the last three (a page) contiguous
void pages_of(const at::Tensor& k, const at::Tensor& v, int dims) {
  need(k.dim() == dims && k.sizes() == v.sizes() && k.scalar_type() == v.scalar_type() && k.strides() == v.strides() &&
           k.device() == v.device(),
       "keys and values must be pages of the same shape, type, layout and device");
  const int64_t s = k.size(dims - 2), d = k.size(dims - 1);
  need(k.stride(dims - 1) == 1 && k.stride(dims - 2) == d && k.stride(dims - 3) == s * d,
       "a page's heads, positions and dims must be contiguous");
  need(k.scalar_type() == at::kHalf || k.scalar_type() == at::kBFloat16, "pages must be float16 or bfloat16");
}
mk_page_view view_of(PyObject* ko, PyObject* vo, PyObject* table, at::Device* dev) {
  const at::Tensor &k = on_gpu(ko, "k_pages"), &v = on_gpu(vo, "v_pages");
  pages_of(k, v, 4);
  *dev = k.device();
  mk_page_view w{};
  w.k = k.data_ptr();
  w.v = v.data_ptr();
  w.n_pages = size32(k.size(0), "n_pages");
  w.n_kv_heads = size32(k.size(1), "n_kv_heads");
  w.page_size = size32(k.size(2), "page_size");
  w.head_dim = size32(k.size(3), "head_dim");
  w.page_stride = k.size(0) > 1 ? k.stride(0) : k.size(1) * k.size(2) * k.size(3);
  w.dtype = dtype_of(k, "pages");
  int32_t* p = nullptr;
  table_of(table, *dev, &p, &w.n_rows, &w.table_width, &w.table_stride);
  w.table = p;
  return w;
}

// [n, heads, dim] of one type and device with contiguous dims; its strides
void heads_of(const at::Tensor& t, const char* name, int64_t n, int64_t heads, int64_t dim, at::ScalarType type,
              at::Device dev, long long* s0, long long* s1) {
  if (t.dim() != 3 || t.size(0) != n || t.size(1) != heads || t.size(2) != dim || t.scalar_type() != type ||
      t.device() != dev || t.stride(2) != 1)
    value_error(std::string(name) + " must be [" + std::to_string(n) + ", " + std::to_string(heads) + ", " +
                std::to_string(dim) + "], of the others' type, on " + dev.str() + ", its last dim contiguous");
  *s0 = t.stride(0);
  *s1 = t.stride(1);
}

template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
bool count_is(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", n, want);
  return false;
}
PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }
PyObject* given(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// (q, k, v, k_pages, v_pages, table, positions, rows, freqs, interleaved, mscale, q_out, status)
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!count_is(n_args, 13)) return nullptr;
  return guarded([&]() -> PyObject* {
    at::Device dev(at::kCPU);
    const mk_page_view view = view_of(a[3], a[4], a[5], &dev);
    const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    need(k.dim() == 3, "k must be [tokens, kv heads, head_dim]");
    mk_append_args x{};
    x.dtype = dtype_of(k, "k");
    const int64_t n = k.size(0);
    heads_of(k, "k", n, view.n_kv_heads, view.head_dim, k.scalar_type(), dev, &x.k_token, &x.k_head);
    heads_of(v, "v", n, view.n_kv_heads, view.head_dim, k.scalar_type(), dev, &x.v_token, &x.v_head);
    x.k = k.data_ptr();
    x.v = v.data_ptr();
    x.n_tokens = size32(n, "tokens");
    x.positions = int32s(a[6], "positions", dev, n);
    x.rows = int32s(a[7], "rows", dev, n, -1, true);
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor out;
    if (a[0] != Py_None) {
      const at::Tensor& q = tensor(a[0], "q");
      need(q.dim() == 3, "q must be [tokens, heads, head_dim]");
      heads_of(q, "q", n, q.size(1), view.head_dim, k.scalar_type(), dev, &x.q_token, &x.q_head);
      out = a[11] == Py_None ? Fresh::one(q.sizes(), q.scalar_type(), dev) : tensor(a[11], "q_out");
      heads_of(out, "q_out", n, q.size(1), view.head_dim, k.scalar_type(), dev, &x.o_token, &x.o_head);
      x.n_heads = size32(q.size(1), "heads");
      x.q = q.data_ptr();
      x.q_out = out.data_ptr();
    } else {
      need(a[11] == Py_None, "q_out without q");
    }
    if (a[8] != Py_None) {
      const at::Tensor& f = tensor(a[8], "freqs");
      need(f.scalar_type() == at::kDouble && f.dim() == 1 && f.device() == dev && f.is_contiguous(),
           "freqs must be a contiguous float64 vector on the pages' device");
      x.freqs = f.data_ptr<double>();
      x.n_freqs = size32(f.size(0), "freqs");
    }
    x.interleaved = PyObject_IsTrue(a[9]);
    x.mscale = (float)number(a[10]);
    int32_t* status = status_of(a[12], dev);
    if (n > 0) {
      check(mk_rope_append(&x, &view, status, stream_of(dev)), "mk_rope_append");
      written(a[3], a[4], a[11], a[12]);
    }
    if (a[0] == Py_None) Py_RETURN_NONE;
    return a[11] == Py_None ? wrap(out) : given(a[11]);
  });
}

// (q, k_pages, v_pages, table, lens, rows, scale, softcap, window, len_add, out, return_lse, status)
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!count_is(n_args, 13)) return nullptr;
  return guarded([&]() -> PyObject* {
    at::Device dev(at::kCPU);
    const mk_page_view view = view_of(a[1], a[2], a[3], &dev);
    const at::Tensor& q = tensor(a[0], "q");
    need(q.dim() == 3, "q must be [rows, heads, head_dim]");
    mk_attend_args x{};
    x.dtype = dtype_of(q, "q");
    const int64_t n = q.size(0), hq = q.size(1);
    heads_of(q, "q", n, hq, view.head_dim, q.scalar_type(), dev, &x.q_row, &x.q_head);
    const c10::cuda::CUDAGuard guard(dev);
    const at::Tensor out = a[10] == Py_None ? Fresh::one(q.sizes(), q.scalar_type(), dev) : tensor(a[10], "out");
    heads_of(out, "out", n, hq, view.head_dim, q.scalar_type(), dev, &x.o_row, &x.o_head);
    x.q = q.data_ptr();
    x.out = out.data_ptr();
    x.n_rows = size32(n, "rows");
    x.n_heads = size32(hq, "heads");
    x.lens = int32s(a[4], "lens", dev, n);
    x.rows = int32s(a[5], "rows", dev, n, -1, true);
    x.scale = a[6] == Py_None ? (float)(1.0 / std::sqrt((double)view.head_dim)) : (float)number(a[6]);
    x.softcap = (float)number(a[7]);
    x.window = integer(a[8], "window");
    x.len_add = integer(a[9], "len_add");
    const int with_lse = PyObject_IsTrue(a[11]);
    at::Tensor lse;
    if (with_lse > 0) {
      lse = Fresh::one({n, hq}, at::kFloat, dev);
      x.lse = lse.data_ptr<float>();
    }
    int32_t* status = status_of(a[12], dev);
    if (n > 0) {
      check(mk_paged_attention_workspace(x.n_heads, view.n_kv_heads, view.head_dim, &x.workspace_bytes),
            "mk_paged_attention_workspace");
      const Workspace ws(x.workspace_bytes);
      x.workspace = ws.p.get();
      check(mk_paged_attention(&x, &view, status, stream_of(dev)), "mk_paged_attention");
      written(a[10], a[12]);
    }
    PyObject* o = a[10] == Py_None ? wrap(out) : given(a[10]);
    if (with_lse <= 0 || !o) return o;
    return Py_BuildValue("(NN)", o, wrap(lse));
  });
}

mk_page_pool pool_of(PyObject* ko, PyObject* vo, PyObject* table, PyObject* refs, at::Device* dev) {
  const at::Tensor &k = on_gpu(ko, "k"), &v = on_gpu(vo, "v");
  pages_of(k, v, 5);
  *dev = k.device();
  const int64_t e = k.element_size(), page = k.size(2) * k.size(3) * k.size(4) * e;
  mk_page_pool p{};
  p.k = k.data_ptr();
  p.v = v.data_ptr();
  p.n_layers = size32(k.size(0), "layers");
  p.n_pages = size32(k.size(1), "n_pages");
  p.page_size = size32(k.size(3), "page_size");
  p.page_bytes = page;
  p.page_stride = k.size(1) > 1 ? k.stride(1) * e : page;
  p.layer_stride = k.size(0) > 1 ? k.stride(0) * e : page;
  table_of(table, *dev, &p.table, &p.n_rows, &p.table_width, &p.table_stride);
  p.refs = int32s(refs, "refs", *dev, k.size(1));
  return p;
}

// (k, v, table, lens, refs, parents, reserve, status)
PyObject* update_pages(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!count_is(n_args, 8)) return nullptr;
  return guarded([&]() -> PyObject* {
    at::Device dev(at::kCPU);
    const mk_page_pool pool = pool_of(a[0], a[1], a[2], a[4], &dev);
    mk_update_args x{};
    x.lens = int32s(a[3], "lens", dev, pool.n_rows);
    x.parents = int32s(a[5], "parents", dev, pool.n_rows, -1, true);
    x.reserve = int32s(a[6], "reserve", dev, pool.n_rows, -1, true);
    int32_t* status = status_of(a[7], dev);
    const c10::cuda::CUDAGuard guard(dev);
    check(mk_update_pages_workspace(pool.n_rows, pool.table_width, pool.n_pages, &x.workspace_bytes),
          "mk_update_pages_workspace");
    const Workspace ws(x.workspace_bytes);
    x.workspace = ws.p.get();
    check(mk_update_pages(&x, &pool, status, stream_of(dev)), "mk_update_pages");
    written(a[0], a[1], a[2], a[3], a[4], a[7]);
    Py_RETURN_NONE;
  });
}

// (k, v, table, refs, status)
PyObject* compact_pages(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!count_is(n_args, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    at::Device dev(at::kCPU);
    const mk_page_pool pool = pool_of(a[0], a[1], a[2], a[3], &dev);
    int32_t* status = status_of(a[4], dev);
    const c10::cuda::CUDAGuard guard(dev);
    size_t bytes = 0;
    check(mk_update_pages_workspace(pool.n_rows, pool.table_width, pool.n_pages, &bytes), "mk_update_pages_workspace");
    const Workspace ws(bytes);
    check(mk_compact_pages(&pool, ws.p.get(), bytes, status, stream_of(dev)), "mk_compact_pages");
    written(a[0], a[1], a[2], a[3], a[4]);
    Py_RETURN_NONE;
  });
}

// (logits, scores, ended, eos, status)
PyObject* beam_select(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!count_is(n_args, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &logits = on_gpu(a[0], "logits"), &scores = tensor(a[1], "scores");
    const at::Device dev = logits.device();
    need(logits.dim() == 2 && (logits.stride(1) == 1 || logits.size(1) == 1),
         "logits must be [rows, vocab], each row contiguous");
    need(scores.dim() == 2 && scores.scalar_type() == at::kFloat && scores.device() == dev && scores.is_contiguous(),
         "scores must be a contiguous float32 [groups, beams] tensor on the logits' device");
    const int64_t groups = scores.size(0), beams = scores.size(1);
    need(logits.size(0) == groups * beams, "logits must have groups * beams rows");
    mk_select_args x{};
    x.dtype = dtype_of(logits, "logits");
    x.logits = logits.data_ptr();
    x.groups = size32(groups, "groups");
    x.beams = size32(beams, "beams");
    x.vocab = size32(logits.size(1), "vocab");
    x.row_stride = logits.size(0) > 1 ? logits.stride(0) : logits.size(1);
    x.eos = integer(a[3], "eos");
    x.scores = scores.data_ptr<float>();
    x.ended = int32s(a[2], "ended", dev, groups, beams);
    int32_t* status = status_of(a[4], dev);
    const c10::cuda::CUDAGuard guard(dev);
    check(mk_beam_select_workspace(x.groups, x.beams, x.vocab, &x.workspace_bytes), "mk_beam_select_workspace");
    const Workspace ws(x.workspace_bytes);
    x.workspace = ws.p.get();
    Fresh fresh(4 * 4 * groups * beams, dev);  // the four results share one allocation
    const at::Tensor token = fresh.take({groups, beams}, at::kInt), parent = fresh.take({groups, beams}, at::kInt),
                     done = fresh.take({groups, beams}, at::kInt), best = fresh.take({groups, beams}, at::kFloat);
    x.out_tokens = token.data_ptr<int32_t>();
    x.out_parents = parent.data_ptr<int32_t>();
    x.out_ended = done.data_ptr<int32_t>();
    x.out_scores = best.data_ptr<float>();
    check(mk_beam_select(&x, status, stream_of(dev)), "mk_beam_select");
    written(a[4]);
    return Py_BuildValue("(NNNN)", wrap(token), wrap(parent), wrap(best), wrap(done));
  });
}

// (status)
PyObject* check_status(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!count_is(n_args, 1)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Device dev = on_gpu(a[0], "status").device();
    int32_t* status = int32s(a[0], "status", dev, 4);
    const c10::cuda::CUDAGuard guard(dev);
    mk_status s;
    Py_BEGIN_ALLOW_THREADS
    s = mk_paged_status(status, stream_of(dev));
    Py_END_ALLOW_THREADS
    if (s != MK_OK) written(a[0]);  // cleared
    check(s, "paged status");
    Py_RETURN_NONE;
  });
}

// (MkError): the class raised for a C status
PyObject* set_error(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!count_is(n_args, 1)) return nullptr;
  Py_INCREF(a[0]);
  Py_XSETREF(g_error, a[0]);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(rope_append),   FAST(paged_attention), FAST(update_pages), FAST(compact_pages),
                           FAST(beam_select),   FAST(check_status),    FAST(set_error),    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_mk_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mk_torch(void) { return PyModule_Create(&g_module); }
