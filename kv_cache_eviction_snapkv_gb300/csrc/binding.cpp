// Marshalling of the paged-cache calls: torch tensors in, pointers and strides to the C entry
// points, torch tensors out. A decode step makes these calls once a layer or once a token, where
// the interpreter's checks of a dozen tensors cost several times the kernels (an append of 16
// tokens: 39 us of a caller's time in Python, 3 on the GPU), so they are made here.
//
// The functions take the wrappers' arguments in order (api.py documents them), raise ValueError
// for a tensor of the wrong kind, and return the entry point's status as an int where it is not
// OK. They run on the tensors' device, which the wrapper has made current, and torch's current
// stream; outputs come from torch's allocator, and so does a workspace, given back once the call
// is queued (the allocator orders its reuse on the stream, and keeps a capture's to its graph).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/Allocator.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "kvsel.h"

namespace {

struct Refused {
  std::string what;
};
void need(bool ok, const char* what) {
  if (!ok) throw Refused{what};
}
void need(bool ok, const char* name, const char* what) {
  if (!ok) throw Refused{std::string(name) + what};
}

// The entry points, by the address that the loader has for them.
struct Entry {
  decltype(&kvsel_paged_append) append;
  decltype(&kvsel_paged_attention) attention;
  decltype(&kvsel_paged_attention_bytes) attention_bytes;
  decltype(&kvsel_paged_compact) compact;
  decltype(&kvsel_pages_update) update;
  decltype(&kvsel_pages_update_bytes) update_bytes;
} g_entry{};

const at::Tensor& tensor(PyObject* o, const char* name) {
  need(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}

bool absent(PyObject* o) { return o == Py_None; }

// Address of a contiguous int32 tensor on the cache's device with `n` entries (-1: any number).
int32_t* int32s(PyObject* o, const char* name, const at::Tensor& K, int64_t n, const char* wrong) {
  const at::Tensor& t = tensor(o, name);
  need(t.scalar_type() == at::kInt && t.device() == K.device() && t.is_contiguous(), name,
       " must be a contiguous int32 tensor on the cache's device");
  if (n >= 0) need(t.numel() == n, wrong);
  return static_cast<int32_t*>(t.data_ptr());
}

struct Pool {
  const at::Tensor& K;
  kvsel_pages p;
};

Pool pool_of(PyObject* ko, PyObject* vo) {
  const at::Tensor &K = tensor(ko, "K"), &V = tensor(vo, "V");
  need(K.sizes() == V.sizes() && K.scalar_type() == V.scalar_type() && K.device() == V.device(),
       "K and V must have one shape, type and device");
  need(K.is_cuda(), "K must be a CUDA tensor");
  need(K.scalar_type() == at::kBFloat16 || K.scalar_type() == at::kFloat, "K must be bf16 or fp32");
  const int64_t dims = K.dim();
  need(dims == 4 || dims == 5, "K and V must be [layers, pages, page_size, H_kv, D]");
  const int64_t* n = K.sizes().data() + (dims - 4);
  const int64_t* s = K.strides().data() + (dims - 4);
  const int64_t layers = dims == 5 ? K.size(0) : 1;
  // the stride of a dimension of one entry means nothing
  need(!((s[3] != 1 && n[3] > 1) || (s[2] != n[3] && n[2] > 1) || (s[1] != n[2] * n[3] && n[1] > 1)),
       "K and V must be dense in their last three dimensions");
  for (int64_t i = 0; i < dims; ++i)
    need(K.size(i) <= 1 || K.stride(i) == V.stride(i), "K and V must have the same strides");
  for (int i = 0; i < 4; ++i) need(n[i] <= INT32_MAX, "K is too large");
  need(layers <= INT32_MAX, "K is too large");
  kvsel_pages p{};
  p.num_layers = (int32_t)layers;
  p.num_pages = (int32_t)n[0];
  p.page_size = (int32_t)n[1];
  p.num_kv_heads = (int32_t)n[2];
  p.head_dim = (int32_t)n[3];
  p.dtype = K.scalar_type() == at::kFloat ? KVSEL_F32 : KVSEL_BF16;
  p.layer_stride = layers > 1 ? K.stride(0) : 0;
  p.page_stride = n[0] > 1 ? s[0] : 0;
  p.K = K.data_ptr();
  p.V = V.data_ptr();
  return Pool{K, p};
}

at::Tensor fresh(const at::Tensor& K, at::IntArrayRef sizes, at::ScalarType type) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(K.device()));
}

// A given output, of the wanted shape and type; or a new one (`object` becomes its owner).
at::Tensor output(PyObject*& object, const char* name, const at::Tensor& K, at::IntArrayRef sizes,
                  at::ScalarType type) {
  if (absent(object)) {
    at::Tensor t = fresh(K, sizes, type);
    object = THPVariable_Wrap(t);
    if (!object) throw python_error();
    return t;
  }
  const at::Tensor& t = tensor(object, name);
  need(t.sizes() == sizes && t.scalar_type() == type && t.device() == K.device() && t.is_contiguous(),
       name, " must be contiguous, of the output's shape, type and device");
  Py_INCREF(object);
  return t;
}

// An object that is given up unless released.
struct Owned {
  PyObject* o = nullptr;
  ~Owned() { Py_XDECREF(o); }
  PyObject* release() {
    PyObject* r = o;
    o = nullptr;
    return r;
  }
};

struct Workspace {
  c10::DataPtr own;
  void* data = nullptr;
  int64_t bytes = 0;
};
Workspace workspace_of(PyObject* o, int64_t bytes, const at::Tensor& K) {
  Workspace w;
  if (absent(o)) {
    if (bytes > 0) w.own = c10::GetAllocator(c10::DeviceType::CUDA)->allocate(bytes);
    w.data = w.own.get();
    w.bytes = bytes;
  } else {
    const at::Tensor& t = tensor(o, "workspace");
    need(t.device() == K.device() && t.is_contiguous(),
         "workspace must be a contiguous tensor on the cache's device");
    w.data = t.data_ptr();
    w.bytes = (int64_t)t.nbytes();
  }
  return w;
}

void* stream_of(const at::Tensor& K) {
  return c10::cuda::getCurrentCUDAStream(K.device().index()).stream();
}

kvsel_rows rows_of(PyObject* o, const char* name, const Pool& c, int64_t tokens, int64_t heads) {
  const at::Tensor& t = tensor(o, name);
  const int64_t dims = t.dim();
  need(dims == 3 || dims == 4, name, " must be [layers, tokens, heads, D]");
  const int64_t* n = t.sizes().data() + (dims - 3);
  const int64_t* s = t.strides().data() + (dims - 3);
  const int64_t layers = dims == 4 ? t.size(0) : 1;
  need(layers == c.p.num_layers && n[0] == tokens && n[1] == heads && n[2] == c.p.head_dim, name,
       " must be [layers, tokens, heads, D] with the cache's layers and D, one entry a token, and H_kv "
       "heads for k and v");
  need(t.scalar_type() == c.K.scalar_type() && t.device() == c.K.device(), name,
       " must have the cache's type and device");
  need((heads <= 1 || s[1] == n[2]) && s[2] == 1, name, " must be dense in its last two dimensions");
  return kvsel_rows{t.data_ptr(), layers > 1 ? t.stride(0) : 0, tokens > 1 ? s[0] : 0};
}

const void* weight_of(PyObject* o, const char* name, const Pool& c) {
  if (absent(o)) return nullptr;
  const at::Tensor& w = tensor(o, name);
  need(w.scalar_type() == c.K.scalar_type() && w.device() == c.K.device() && w.is_contiguous() &&
           w.numel() == (int64_t)c.p.num_layers * c.p.head_dim,
       name, " must be a contiguous [layers, D] tensor of the cache's type");
  return w.data_ptr();
}

// table [num_seqs, table_width]
int32_t* table_of(PyObject* o, const at::Tensor& K, int64_t* seqs, int64_t* width) {
  int32_t* p = int32s(o, "table", K, -1, "");
  const at::Tensor& t = THPVariable_Unpack(o);
  need(t.dim() == 2 && t.size(0) <= INT32_MAX && t.size(1) <= INT32_MAX,
       "table must be [num_seqs, table_width]");
  *seqs = t.size(0);
  *width = t.size(1);
  return p;
}

PyObject* status_object(kvsel_status st) { return PyLong_FromLong(st); }

template <typename F>
PyObject* guarded(F&& f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (q, k, v, K, V, cache_pos, positions, table, seqs, q_weight, k_weight, eps, inv_freq,
//  interleaved, scale, q_out)
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    need(n_args == 16, "paged_append takes 16 arguments");
    const Pool c = pool_of(a[3], a[4]);
    PyObject *q = a[0], *k = a[1], *v = a[2], *positions = a[6], *table = a[7], *seqs = a[8],
             *inv_freq = a[12];
    need(!absent(q) || !absent(k), "q or k and v must be given");
    need(absent(k) == absent(v), "k and v go together");
    const at::Tensor& first = tensor(absent(q) ? k : q, absent(q) ? "k" : "q");
    need(first.dim() == 3 || first.dim() == 4, "q, k and v must be [layers, tokens, heads, D]");
    const int64_t tokens = first.size(-3), heads = absent(q) ? 0 : first.size(-2);
    need(tokens <= INT32_MAX && heads <= INT32_MAX, "too many tokens");
    kvsel_rows rq{}, rk{}, rv{};
    if (!absent(q)) rq = rows_of(q, "q", c, tokens, heads);
    int32_t* at = nullptr;
    if (!absent(k)) {
      rk = rows_of(k, "k", c, tokens, c.p.num_kv_heads);
      rv = rows_of(v, "v", c, tokens, c.p.num_kv_heads);
      at = int32s(a[5], "cache_pos", c.K, tokens, "cache_pos must have one entry a token");
    }
    kvsel_rope rope{};
    if (!absent(inv_freq) && tensor(inv_freq, "inv_freq").numel() > 0) {
      const at::Tensor& f = THPVariable_Unpack(inv_freq);
      need(f.scalar_type() == at::kFloat && f.device() == c.K.device() && f.is_contiguous() &&
               f.numel() <= 65535,
           "inv_freq must be a contiguous fp32 tensor on the cache's device");
      need(!absent(positions), "positions must have one entry a token");
      rope.rot_dim = (int32_t)(2 * f.numel());
      rope.interleaved = PyObject_IsTrue(a[13]);
      rope.inv_freq = static_cast<const float*>(f.data_ptr());
      rope.scale = (float)PyFloat_AsDouble(a[14]);
    }
    const float eps = (float)PyFloat_AsDouble(a[11]);
    if (PyErr_Occurred()) throw python_error();
    int32_t* pos = absent(positions) ? nullptr
                                     : int32s(positions, "positions", c.K, tokens,
                                              "positions must have one entry a token");
    int64_t n_seqs = 0, width = 0;
    int32_t* tab = absent(table) ? nullptr : table_of(table, c.K, &n_seqs, &width);
    int32_t* seq = absent(seqs) ? nullptr
                                : int32s(seqs, "seqs", c.K, tokens, "seqs must have one entry a token");
    const void* qw = weight_of(a[9], "q_weight", c);
    const void* kw = weight_of(a[10], "k_weight", c);
    Owned out;
    void* q_out = nullptr;
    if (!absent(q)) {
      PyObject* o = a[15];
      q_out = output(o, "q_out", c.K, first.sizes(), c.K.scalar_type()).data_ptr();
      out.o = o;
    }
    const kvsel_status st = g_entry.append(
        &c.p, (int32_t)tokens, (int32_t)heads, absent(q) ? nullptr : &rq, absent(k) ? nullptr : &rk,
        absent(k) ? nullptr : &rv, rope.rot_dim ? &rope : nullptr, qw, kw, eps, pos, (int32_t)n_seqs, tab,
        (int32_t)width, seq, at, q_out, stream_of(c.K));
    if (st != KVSEL_OK) return status_object(st);
    if (!out.o) Py_RETURN_NONE;
    return out.release();
  });
}

// (q, K, V, table, lens, out, lse, want_lse, workspace)
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    need(n_args == 9, "paged_attention takes 9 arguments");
    const Pool c = pool_of(a[1], a[2]);
    const at::Tensor& q = tensor(a[0], "q");
    need(q.dim() == 3 || q.dim() == 4, "q must be [layers, S, H, D]");
    const int64_t layers = q.dim() == 4 ? q.size(0) : 1, S = q.size(-3), H = q.size(-2);
    need(layers == c.p.num_layers && q.size(-1) == c.p.head_dim && q.scalar_type() == c.K.scalar_type() &&
             q.device() == c.K.device() && q.is_contiguous() && S <= INT32_MAX && H <= INT32_MAX,
         "q must be contiguous [layers, S, H, D] of the cache's layers, D, type and device");
    int64_t seqs = 0, width = 0;
    int32_t* table = table_of(a[3], c.K, &seqs, &width);
    need(seqs == S, "table must be [S, table_width] and lens [S]");
    int32_t* lens = int32s(a[4], "lens", c.K, S, "table must be [S, table_width] and lens [S]");
    Owned out, lse;
    PyObject* o = a[5];
    void* out_at = output(o, "out", c.K, q.sizes(), at::kFloat).data_ptr();
    out.o = o;
    void* lse_at = nullptr;
    o = a[6];
    if (!absent(o) || PyObject_IsTrue(a[7])) {
      lse_at = output(o, "lse", c.K, q.sizes().slice(0, q.dim() - 1), at::kFloat).data_ptr();
      lse.o = o;
    } else {
      Py_INCREF(o);
      lse.o = o;
    }
    const int64_t bytes = g_entry.attention_bytes(&c.p, (int32_t)S, (int32_t)H);
    // where a rule is broken the call says which
    Workspace w = workspace_of(a[8], bytes < 0 ? 0 : bytes, c.K);
    const kvsel_status st = g_entry.attention(
        &c.p, (int32_t)S, (int32_t)H, q.data_ptr(), table, (int32_t)width, lens,
        static_cast<float*>(out_at), static_cast<float*>(lse_at), w.data, w.bytes, stream_of(c.K));
    if (st != KVSEL_OK) return status_object(st);
    PyObject* pair = PyTuple_New(2);
    if (!pair) throw python_error();
    PyTuple_SET_ITEM(pair, 0, out.release());
    PyTuple_SET_ITEM(pair, 1, lse.release());
    return pair;
  });
}

// (K, V, table, lens, keep_idx, keep_offsets, max_keep, ref, slot_pos)
PyObject* paged_compact(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    need(n_args == 9, "paged_compact takes 9 arguments");
    const Pool c = pool_of(a[0], a[1]);
    int64_t S = 0, width = 0;
    int32_t* table = table_of(a[2], c.K, &S, &width);
    int32_t* lens = int32s(a[3], "lens", c.K, S, "lens must have S entries and keep_offsets S + 1");
    int32_t* idx = int32s(a[4], "keep_idx", c.K, -1, "");
    const at::Tensor& keep = THPVariable_Unpack(a[4]);
    need((keep.dim() == 3 ? keep.size(0) == c.p.num_layers : keep.dim() == 2 && c.p.num_layers == 1) &&
             keep.size(-1) == c.p.num_kv_heads,
         "keep_idx must be [layers, keep_rows, H_kv]");
    int32_t* offs = int32s(a[5], "keep_offsets", c.K, S + 1,
                           "lens must have S entries and keep_offsets S + 1");
    const long most = PyLong_AsLong(a[6]);
    if (most == -1 && PyErr_Occurred()) throw python_error();
    need(most >= INT32_MIN && most <= INT32_MAX, "max_keep is too large");
    int32_t* ref = absent(a[7]) ? nullptr
                                : int32s(a[7], "ref", c.K, c.p.num_pages, "ref must have one entry a page");
    Owned pos;
    PyObject* o = a[8];
    void* at = output(o, "slot_pos", c.K, keep.sizes(), at::kInt).data_ptr();
    pos.o = o;
    const kvsel_status st = g_entry.compact(&c.p, (int32_t)S, table, (int32_t)width, lens, idx,
                                            keep.size(-2), offs, (int32_t)most, ref,
                                            static_cast<int32_t*>(at), stream_of(c.K));
    if (st != KVSEL_OK) return status_object(st);
    return pos.release();
  });
}

// (K, V, table, lens, new_lens, parents, table_out, ref, free_pages, workspace)
PyObject* pages_update(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    need(n_args == 10, "pages_update takes 10 arguments");
    const Pool c = pool_of(a[0], a[1]);
    int64_t n_in = 0, width = 0;
    int32_t* table = table_of(a[2], c.K, &n_in, &width);
    const char* counts = "lens must have one entry an old sequence, parents one a new one";
    int32_t* lens = int32s(a[3], "lens", c.K, n_in, counts);
    int32_t* news = int32s(a[4], "new_lens", c.K, -1, "");
    const int64_t n_out = THPVariable_Unpack(a[4]).numel();
    need(n_out <= INT32_MAX, "new_lens is too long");
    int32_t* parents = absent(a[5]) ? nullptr : int32s(a[5], "parents", c.K, n_out, counts);
    Owned t, r, f;
    PyObject* o = a[6];
    void* t_at = output(o, "table_out", c.K, {n_out, width}, at::kInt).data_ptr();
    t.o = o;
    o = a[7];
    void* r_at = output(o, "ref", c.K, {(int64_t)c.p.num_pages}, at::kInt).data_ptr();
    r.o = o;
    o = a[8];
    void* f_at = output(o, "free_pages", c.K, {1}, at::kInt).data_ptr();
    f.o = o;
    const int64_t bytes = g_entry.update_bytes(&c.p, (int32_t)n_out);
    Workspace w = workspace_of(a[9], bytes < 0 ? 0 : bytes, c.K);
    const kvsel_status st = g_entry.update(
        &c.p, (int32_t)n_in, table, (int32_t)width, lens, (int32_t)n_out, parents, news,
        static_cast<int32_t*>(t_at), static_cast<int32_t*>(r_at), static_cast<int32_t*>(f_at), w.data,
        w.bytes, stream_of(c.K));
    if (st != KVSEL_OK) return status_object(st);
    PyObject* three = PyTuple_New(3);
    if (!three) throw python_error();
    PyTuple_SET_ITEM(three, 0, t.release());
    PyTuple_SET_ITEM(three, 1, r.release());
    PyTuple_SET_ITEM(three, 2, f.release());
    return three;
  });
}

// Addresses of the six entry points, in Entry's order.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    need(n_args == 6, "bind takes 6 addresses");
    void* p[6];
    for (int i = 0; i < 6; ++i) {
      p[i] = PyLong_AsVoidPtr(a[i]);
      if (PyErr_Occurred()) throw python_error();
    }
    g_entry = Entry{reinterpret_cast<decltype(Entry::append)>(p[0]),
                    reinterpret_cast<decltype(Entry::attention)>(p[1]),
                    reinterpret_cast<decltype(Entry::attention_bytes)>(p[2]),
                    reinterpret_cast<decltype(Entry::compact)>(p[3]),
                    reinterpret_cast<decltype(Entry::update)>(p[4]),
                    reinterpret_cast<decltype(Entry::update_bytes)>(p[5])};
    Py_RETURN_NONE;
  });
}

#define KVSEL_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {KVSEL_METHOD(paged_append), KVSEL_METHOD(paged_attention),
                           KVSEL_METHOD(paged_compact), KVSEL_METHOD(pages_update), KVSEL_METHOD(bind),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_kvsel_torch", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kvsel_torch(void) { return PyModule_Create(&g_module); }
