// Python entry of the rotary and paged-cache calls: checks tensors, allocates
// what the caller did not give, and calls the C ABI (attn.h) on the current
// stream, like the package's ctypes functions, but compiled: these calls are
// made once per layer and token in decoding, where the time of a call is the
// host's.  Measured on the Grace host, a call after the other with outputs
// allocated: an append of 64 tokens 5.3 to 6.0 us (19.5 with the same checks in
// Python and ctypes), attention of one decoding sequence 6.9 to 7.3 (20).
//
// The functions of libattn.so are handed over by address (init), so that both
// routes use one loaded library.
#include <Python.h>

#include <cmath>
#include <cstdint>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "attn.h"

namespace {

constexpr int kMaxAxes = 8;  // position axes of a rotary table

decltype(&attn_rope) p_rope = nullptr;
decltype(&attn_append_kv) p_append = nullptr;
decltype(&attn_fwd_paged) p_paged = nullptr;
decltype(&attn_fwd_paged_workspace_bytes) p_paged_bytes = nullptr;
PyObject* g_error = nullptr;  // the package's AttnError

[[noreturn]] void fail(PyObject* type, const char* fmt, const char* what = "") {
  PyErr_Format(type, fmt, what);
  throw python_error();
}

void need(bool ok, const char* fmt, const char* what = "") {
  if (!ok) fail(PyExc_ValueError, fmt, what);
}

// A tensor argument; None gives an undefined one.
at::Tensor tensor(PyObject* o, const char* what) {
  if (o == Py_None) return {};
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a tensor", what);
  return THPVariable_Unpack(o);
}

at::Tensor required(PyObject* o, const char* what) {
  at::Tensor t = tensor(o, what);
  if (!t.defined()) fail(PyExc_TypeError, "%s must be a tensor", what);
  return t;
}

bool truth(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw python_error();
  return r != 0;
}

int integer(PyObject* o, const char* what) {
  PyObject* n = PyNumber_Long(o);
  if (n == nullptr) throw python_error();
  int overflow = 0;
  const long v = PyLong_AsLongAndOverflow(n, &overflow);
  Py_DECREF(n);
  need(overflow == 0 && v >= INT32_MIN && v <= INT32_MAX, "%s out of range", what);
  return (int)v;
}

// Sizes the C ABI takes as int.
int size(int64_t n) {
  need(n <= INT32_MAX, "a dimension is too long");
  return (int)n;
}

attn_dtype dtype_of(const at::Tensor& t) {
  if (t.scalar_type() == at::kHalf) return ATTN_F16;
  if (t.scalar_type() == at::kBFloat16) return ATTN_BF16;
  fail(PyExc_TypeError, "tensors must be float16 or bfloat16");
}

bool like(const at::Tensor& a, const at::Tensor& b) {
  return a.scalar_type() == b.scalar_type() && a.device() == b.device();
}

bool ints_on(const at::Tensor& t, at::ScalarType type, const at::Tensor& x) {
  return t.scalar_type() == type && t.device() == x.device() && t.is_contiguous();
}

// Batch (4-D only), head and token strides of a tensor whose rows are read or
// written 16 bytes at a time, 0 for a dimension of size 1.
void row_strides(const at::Tensor& t, const char* what, bool written, int64_t* s) {
  const int64_t n = t.dim();
  need(t.stride(n - 1) == 1, "%s: the last dimension must be contiguous", what);
  for (int64_t i = 0; i < n - 1; ++i) {
    s[i] = t.size(i) > 1 ? t.stride(i) : 0;
    need((s[i] & 7) == 0, "%s: the strides must be multiples of 8 elements", what);
    need(!written || t.size(i) == 1 || s[i] != 0, "%s must not be an expanded tensor", what);
  }
}

// Turning channels of a rotary table for rows of d.
int table_rot(const at::Tensor& table, const at::Tensor& x, int64_t d) {
  need(table.dim() == 2 && table.size(0) == 2 && ints_on(table, at::kLong, x),
       "table must be a contiguous int64 [2, rot/2] tensor (rope_table) on the tensors' device");
  const int64_t rot = 2 * table.size(1);
  need(rot >= 16 && (rot & 15) == 0 && rot <= d,
       "the table must turn a multiple of 16 channels, at most the head dim");
  return (int)rot;
}

void* stream_of(const at::Tensor& x) {
  return c10::cuda::getCurrentCUDAStream(x.get_device()).stream();
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

template <typename T>
T* ptr_as(const at::Tensor& t) {
  return static_cast<T*>(ptr(t));
}

void check(attn_status st, const char* what) {
  if (st == ATTN_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "si", what, (int)st);
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw python_error();
}

void arguments(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) fail(PyExc_TypeError, "wrong number of arguments");
}

// rope(q, k, positions, table, interleaved, out_q, out_k, inverse) -> (q', k')
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 8);
  const at::Tensor q = required(a[0], "q"), k = tensor(a[1], "k");
  const at::Tensor pos = required(a[2], "positions"), table = required(a[3], "table");
  at::Tensor oq = tensor(a[5], "out_q"), ok = tensor(a[6], "out_k");
  const bool inverse = truth(a[7]);
  need(q.dim() == 3 || q.dim() == 4, "tensors must be [B, H, N, d] or packed [H, total, d]");
  const attn_dtype dt = dtype_of(q);
  need(q.is_cuda(), "all tensors must be on the same CUDA device");
  need(q.numel() > 0, "tensors must not be empty");
  const int64_t h = q.dim() - 3;  // dimension of the heads
  const int64_t B = h ? q.size(0) : 1, N = q.size(h + 1), d = q.size(h + 2);
  const int rot = table_rot(table, q, d);
  need(ints_on(pos, at::kInt, q),
       "positions must be a contiguous int32 tensor on the tensors' device");
  const int64_t pd = pos.dim();
  need((pd == 2 || pd == 3) && pos.size(0) >= 1 && pos.size(0) <= kMaxAxes &&
           pos.size(pd - 1) == N && (pd == 2 || pos.size(1) == 1 || pos.size(1) == B),
       "positions must be [axes, N] or [axes, B, N], at most 8 axes");
  need(k.defined() || !ok.defined(), "out_k without k");
  int64_t st[12] = {};
  row_strides(q, "q", false, st + (h ? 0 : 1));
  if (k.defined()) {
    need(k.dim() == q.dim() && like(k, q) && k.numel() > 0 && k.size(h + 1) == N &&
             k.size(h + 2) == d && (!h || k.size(0) == B),
         "q and k must share batch, length, head dim, dtype and device");
    row_strides(k, "k", false, st + 6 + (h ? 0 : 1));
  }
  c10::cuda::CUDAGuard guard(q.device());
  if (!oq.defined()) oq = at::empty(q.sizes(), q.options());
  need(oq.sizes() == q.sizes() && like(oq, q), "out_q must have the shape, dtype and device of q");
  row_strides(oq, "out_q", true, st + 3 + (h ? 0 : 1));
  if (k.defined()) {
    if (!ok.defined()) ok = at::empty(k.sizes(), k.options());
    need(ok.sizes() == k.sizes() && like(ok, k),
         "out_k must have the shape, dtype and device of k");
    row_strides(ok, "out_k", true, st + 9 + (h ? 0 : 1));
  }
  check(p_rope(ptr(q), ptr(k), ptr(oq), ptr(ok), st, ptr_as<int32_t>(pos),
               pd == 3 ? size(pos.size(1)) : 1, (int)pos.size(0), ptr_as<int64_t>(table), rot,
               truth(a[4]), inverse, size(B), size(q.size(h)), k.defined() ? size(k.size(h)) : 0,
               size(N), size(d), dt, stream_of(q)),
        inverse ? "attn_rope_bwd" : "attn_rope");
  PyObject* out = PyTuple_New(2);
  if (out == nullptr) return nullptr;
  PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(oq));
  PyTuple_SET_ITEM(out, 1, k.defined() ? THPVariable_Wrap(ok) : Py_NewRef(Py_None));
  return out;
  END_HANDLE_TH_ERRORS
}

// The cache and the batch of the paged calls.
struct Paged {
  at::Tensor k_pages, v_pages, blocks, cu, kv;

  // x: packed new tokens [H, total, d]
  Paged(PyObject* const* a, const at::Tensor& x)
      : k_pages(required(a[0], "k_pages")), v_pages(required(a[1], "v_pages")),
        blocks(required(a[2], "block_table")), cu(required(a[3], "cu_seqlens")),
        kv(required(a[4], "kv_lens")) {
    need(x.dim() == 3, "packed tensors must be [H, total, d]");
    dtype_of(x);
    need(x.is_cuda() && like(k_pages, x) && like(v_pages, x),
         "tokens and pages must be CUDA tensors of one dtype on one device");
    need(k_pages.dim() == 4 && k_pages.sizes() == v_pages.sizes() && k_pages.size(3) == x.size(2),
         "k_pages, v_pages must be [n_pages, Hkv, page, d] with the tokens' d");
    need(k_pages.is_contiguous() && v_pages.is_contiguous(),
         "k_pages, v_pages must be contiguous");
    need(kv.dim() == 1 && kv.size(0) >= 1 && blocks.dim() == 2 && blocks.size(0) == kv.size(0) &&
             cu.dim() == 1 && cu.size(0) == kv.size(0) + 1,
         "block_table must be [n_seq, max_pages], cu_seqlens [n_seq + 1], kv_lens [n_seq]");
    need(ints_on(blocks, at::kInt, x) && ints_on(cu, at::kInt, x) && ints_on(kv, at::kInt, x),
         "block_table, cu_seqlens and kv_lens must be contiguous int32 tensors on the tokens' "
         "device");
  }
};

// append_kv(k, v, k_pages, v_pages, block_table, cu_seqlens, kv_lens, table,
//           positions, interleaved, q, out_q) -> q' or None
PyObject* append_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 12);
  const at::Tensor k = required(a[0], "k"), v = required(a[1], "v");
  const Paged c(a + 2, k);
  const at::Tensor table = tensor(a[7], "table"), pos = tensor(a[8], "positions");
  const at::Tensor q = tensor(a[10], "q");
  at::Tensor oq = tensor(a[11], "out_q");
  const int64_t Hkv = k.size(0), total = k.size(1), d = k.size(2);
  need(Hkv == c.k_pages.size(1) && v.sizes() == k.sizes() && like(v, k),
       "k and v must be [Hkv, total, d] with the cache's heads");
  need(k.numel() > 0, "tensors must not be empty");
  const int rot = table.defined() ? table_rot(table, k, d) : 0;
  if (pos.defined()) {
    need(table.defined(), "positions without a table");
    need(ints_on(pos, at::kInt, k) && pos.dim() == 2 && pos.size(1) == total &&
             pos.size(0) >= 1 && pos.size(0) <= kMaxAxes,
         "positions must be a contiguous int32 [axes, total] tensor, at most 8 axes");
  }
  int64_t st[6] = {};
  row_strides(k, "k", false, st);
  row_strides(v, "v", false, st + 2);
  need(q.defined() || !oq.defined(), "out_q without q");
  c10::cuda::CUDAGuard guard(k.device());
  if (q.defined()) {
    need(q.dim() == 3 && like(q, k) && q.size(1) == total && q.size(2) == d && q.size(0) >= 1 &&
             q.size(0) % Hkv == 0,
         "q must be [Hq, total, d] with k's total, d, dtype and device, Hq a multiple of Hkv");
    row_strides(q, "q", false, st + 4);
    if (!oq.defined()) oq = at::empty(q.sizes(), q.options());
    need(oq.sizes() == q.sizes() && like(oq, q) && oq.is_contiguous(),
         "out_q must be contiguous with q's shape, dtype and device");
  }
  check(p_append(ptr(k), ptr(v), ptr(q), ptr(oq), st, ptr(c.k_pages), ptr(c.v_pages),
                 ptr_as<int32_t>(c.blocks), ptr_as<int32_t>(c.cu), ptr_as<int32_t>(c.kv),
                 ptr_as<int32_t>(pos), pos.defined() ? (int)pos.size(0) : 1,
                 ptr_as<int64_t>(table), rot, truth(a[9]), size(c.kv.size(0)), size(total),
                 size(c.k_pages.size(0)), size(c.k_pages.size(2)), size(c.blocks.size(1)),
                 q.defined() ? size(q.size(0)) : 0, size(Hkv), size(d), dtype_of(k),
                 stream_of(k)),
        "attn_append_kv");
  if (!q.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(oq);
  END_HANDLE_TH_ERRORS
}

// fwd_paged(q, k_pages, v_pages, block_table, cu_seqlens, kv_lens, max_q, causal,
//           scale, out, lse, workspace) -> (out, lse)
PyObject* fwd_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 12);
  const at::Tensor q = required(a[0], "q");
  const Paged c(a + 1, q);
  const int max_q = integer(a[6], "max_q");
  at::Tensor out = tensor(a[9], "out"), lse = tensor(a[10], "lse");
  at::Tensor ws = tensor(a[11], "workspace");
  const int64_t H = q.size(0), total = q.size(1), d = q.size(2), Hkv = c.k_pages.size(1);
  need(q.is_contiguous(), "q must be contiguous [Hq, total, d]");
  need(Hkv >= 1 && H >= 1 && H % Hkv == 0,
       "the number of key/value heads must divide the query heads");
  need(max_q >= 1 && max_q <= total, "max_q must lie in [1, total]");
  double scale = 1.0 / std::sqrt((double)d);
  if (a[8] != Py_None) {
    scale = PyFloat_AsDouble(a[8]);
    if (scale == -1.0 && PyErr_Occurred()) throw python_error();
  }
  need(!out.defined() || (out.sizes() == q.sizes() && like(out, q) && out.is_contiguous()),
       "out must be a contiguous tensor of q's shape, dtype and device");
  need(!lse.defined() || (lse.dim() == 2 && lse.size(0) == H && lse.size(1) == total &&
                          lse.scalar_type() == at::kFloat && lse.device() == q.device() &&
                          lse.is_contiguous()),
       "lse must be a contiguous float32 [Hq, total] tensor on q's device");
  need(!ws.defined() || ints_on(ws, at::kByte, q),
       "workspace must be a contiguous uint8 tensor on q's device");
  const int n_seq = size(c.kv.size(0)), max_pages = size(c.blocks.size(1));
  const int page = size(c.k_pages.size(2));
  c10::cuda::CUDAGuard guard(q.device());
  if (!out.defined()) out = at::empty(q.sizes(), q.options());
  if (!lse.defined()) lse = at::empty({H, total}, q.options().dtype(at::kFloat));
  if (!ws.defined()) {
    const size_t bytes =
        p_paged_bytes(n_seq, max_q, (int64_t)max_pages * page, size(H), size(Hkv), size(d));
    if (bytes > 0) ws = at::empty({(int64_t)bytes}, q.options().dtype(at::kByte));
  }
  check(p_paged(ptr(q), ptr(c.k_pages), ptr(c.v_pages), ptr(out), ptr_as<float>(lse),
                ptr_as<int32_t>(c.blocks), ptr_as<int32_t>(c.cu), ptr_as<int32_t>(c.kv), ptr(ws),
                ws.defined() ? (size_t)ws.numel() : 0, n_seq, max_q, size(total),
                size(c.k_pages.size(0)), page, max_pages, size(H), size(Hkv), size(d),
                truth(a[7]), (float)scale, dtype_of(q), stream_of(q)),
        "attn_fwd_paged");
  PyObject* pair = PyTuple_New(2);
  if (pair == nullptr) return nullptr;
  PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(out));
  PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(lse));
  return pair;
  END_HANDLE_TH_ERRORS
}

// init(AttnError, addresses of attn_rope, attn_append_kv, attn_fwd_paged,
//      attn_fwd_paged_workspace_bytes)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 5);
  void* f[4];
  for (int i = 0; i < 4; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (f[i] == nullptr) fail(PyExc_TypeError, "function addresses are wanted");
  }
  p_rope = reinterpret_cast<decltype(p_rope)>(f[0]);
  p_append = reinterpret_cast<decltype(p_append)>(f[1]);
  p_paged = reinterpret_cast<decltype(p_paged)>(f[2]);
  p_paged_bytes = reinterpret_cast<decltype(p_paged_bytes)>(f[3]);
  Py_INCREF(a[0]);
  Py_XSETREF(g_error, a[0]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<rope>("rope"), method<append_kv>("append_kv"),
                           method<fwd_paged>("fwd_paged"), method<init>("init"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
