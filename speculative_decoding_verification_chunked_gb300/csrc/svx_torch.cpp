// The binding's per-token calls in native code: checks of torch tensors against the C layouts, then the C call.
//
// A Draft makes these calls once a layer and token, so their cost on the host counts beside kernels of 4 to 10 us: the
// same checks in Python with ctypes took 11 us a call.  Nothing is kept between calls.  Errors become SvxError
// (status, message), as in svx.py, which documents the arguments.
#include <Python.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <initializer_list>
#include <sstream>
#include <string>

#include "svx.h"

namespace {

// Addresses of the C calls: those of the library that svx.py has loaded.
struct Calls {
  decltype(&svx_qk_norm_rope) qk_norm_rope = nullptr;
  decltype(&svx_paged_append) append = nullptr;
  decltype(&svx_paged_decode_workspace) decode_workspace = nullptr;
  decltype(&svx_paged_decode) decode = nullptr;
  decltype(&svx_paged_evict_workspace) evict_workspace = nullptr;
  decltype(&svx_paged_evict) evict = nullptr;
  decltype(&svx_residual_norm) residual_norm = nullptr;
  decltype(&svx_paged_decode_shared_workspace) decode_shared_workspace = nullptr;
  decltype(&svx_paged_decode_shared) decode_shared = nullptr;
  decltype(&svx_cross_attn_workspace) cross_attn_workspace = nullptr;
  decltype(&svx_cross_attn) cross_attn = nullptr;
  decltype(&svx_last_error) last_error = nullptr;
} g;
PyObject* g_error = nullptr;  // svx.SvxError

// What the checks throw; turned into SvxError at the entry points.
struct Refused {
  int status;
  std::string message;
};

[[noreturn]] void refuse(int status, const std::string& message) { throw Refused{status, message}; }

std::string describe(const at::Tensor& t) {
  std::ostringstream s;
  s << t.scalar_type() << " " << t.sizes() << " on " << t.device() << (t.is_contiguous() ? "" : ", not contiguous");
  return s.str();
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(SVX_ERR_INVALID_ARG, std::string(what) + ": a torch tensor is required");
  return THPVariable_Unpack(o);
}

// Address of a dense tensor of exactly this type and shape on this CUDA device.
void* dense(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, int device, const char* what) {
  const at::Tensor& t = tensor(o, what);
  if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape) || !t.is_cuda() || t.get_device() != device ||
      !t.is_contiguous()) {
    std::ostringstream s;
    s << what << ": " << describe(t) << "; expected dense " << type << " " << at::IntArrayRef(shape) << " on cuda:" << device;
    refuse(SVX_ERR_INVALID_ARG, s.str());
  }
  return t.data_ptr();
}

void* optional(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, int device, const char* what) {
  return o == Py_None ? nullptr : dense(o, type, shape, device, what);
}

int type_code(const at::Tensor& t, const char* what) {
  if (t.scalar_type() == at::kBFloat16) return SVX_BF16;
  if (t.scalar_type() == at::kHalf) return SVX_FP16;
  refuse(SVX_ERR_UNSUPPORTED, std::string(what) + ": " + describe(t) + ", expected torch.bfloat16 or torch.float16");
}

at::ScalarType scalar_of(int code) { return code == SVX_BF16 ? at::kBFloat16 : at::kHalf; }

int64_t integer(PyObject* o, const char* what) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(SVX_ERR_INVALID_ARG, std::string(what) + ": an integer is required");
  }
  return v;
}

int32_t integer32(PyObject* o, const char* what) {
  const int64_t v = integer(o, what);
  if (v < INT32_MIN || v > INT32_MAX) refuse(SVX_ERR_INVALID_ARG, std::string(what) + " does not fit 32 bits");
  return static_cast<int32_t>(v);
}

float real(PyObject* o, const char* what) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(SVX_ERR_INVALID_ARG, std::string(what) + ": a number is required");
  }
  return static_cast<float>(v);
}

// Heads [requests][tokens][heads][d], possibly a view of a fused projection: address, elements between tokens.
struct Rows {
  const void* at = nullptr;
  int64_t stride = 0, heads = 0;
};
Rows head_rows(const at::Tensor& t, int64_t n_req, int64_t n_tok, int64_t d, at::ScalarType type, int device, const char* what) {
  if (t.dim() != 4 || t.size(0) != n_req || t.size(1) != n_tok || t.size(3) != d || t.scalar_type() != type || !t.is_cuda() ||
      t.get_device() != device) {
    std::ostringstream s;
    s << what << ": " << describe(t) << ", expected " << type << " [" << n_req << ", " << n_tok << ", heads, " << d << "] on cuda:" << device;
    refuse(SVX_ERR_INVALID_ARG, s.str());
  }
  const int64_t heads = t.size(2);
  if (t.stride(3) != 1 || (heads > 1 && t.stride(2) != d) || (n_tok > 1 && n_req > 1 && t.stride(0) != n_tok * t.stride(1))) {
    std::ostringstream s;
    s << what << ": strides " << t.strides() << ": a token's heads must be dense, and tokens evenly spaced over the requests";
    refuse(SVX_ERR_INVALID_ARG, s.str());
  }
  return Rows{t.data_ptr(), n_tok > 1 ? t.stride(1) : n_req > 1 ? t.stride(0) : heads * d, heads};
}

svx_heads heads_of(PyObject* qo, PyObject* ko, PyObject* vo, PyObject* pos, PyObject* q_norm, PyObject* k_norm, PyObject* eps,
                   PyObject* n_new) {
  const at::Tensor& q = tensor(qo, "q");
  svx_heads h = {};
  h.dtype = type_code(q, "q");
  if (q.dim() != 4 || !q.is_cuda())
    refuse(SVX_ERR_INVALID_ARG, "q: " + describe(q) + ", expected [requests, tokens, heads, head_dim] on a CUDA device");
  const int64_t b = q.size(0), n = q.size(1), d = q.size(3);
  const at::ScalarType type = q.scalar_type();
  const int device = q.get_device();
  const Rows rq = head_rows(q, b, n, d, type, device, "q"), rk = head_rows(tensor(ko, "k"), b, n, d, type, device, "k");
  if (vo != Py_None) {
    const Rows rv = head_rows(tensor(vo, "v"), b, n, d, type, device, "v");
    if (rv.heads != rk.heads) refuse(SVX_ERR_INVALID_ARG, "k and v differ in their number of heads");
    h.v = rv.at;
    h.v_stride = rv.stride;
  }
  if (b > INT32_MAX || n > INT32_MAX || rq.heads > INT32_MAX || rk.heads > INT32_MAX || d > INT32_MAX)
    refuse(SVX_ERR_INVALID_ARG, "q: a dimension does not fit 32 bits");
  h.q = rq.at;
  h.q_stride = rq.stride;
  h.k = rk.at;
  h.k_stride = rk.stride;
  h.q_norm = optional(q_norm, type, {d}, device, "q_norm");
  h.k_norm = optional(k_norm, type, {d}, device, "k_norm");
  h.pos = static_cast<const int32_t*>(dense(pos, at::kInt, {b, n}, device, "pos"));
  h.n_new = static_cast<const int32_t*>(optional(n_new, at::kInt, {b}, device, "n_new"));
  h.n_req = static_cast<int32_t>(b);
  h.n_tok = static_cast<int32_t>(n);
  h.n_q_heads = static_cast<int32_t>(rq.heads);
  h.n_kv_heads = static_cast<int32_t>(rk.heads);
  h.head_dim = static_cast<int32_t>(d);
  h.device = device;
  h.flags = SVX_POINTERS_CHECKED;
  h.eps = -1.f;
  if (eps != Py_None) {
    h.eps = real(eps, "eps");
    if (!(h.eps >= 0.f)) refuse(SVX_ERR_INVALID_ARG, "eps must be >= 0, or None for no norms");
  }
  return h;
}

svx_pages pages_of(PyObject* o) {
  if (!PyBytes_Check(o) || PyBytes_GET_SIZE(o) != static_cast<Py_ssize_t>(sizeof(svx_pages)))
    refuse(SVX_ERR_INVALID_ARG, "not the pages of a PagedCache");
  svx_pages p;
  memcpy(&p, PyBytes_AS_STRING(o), sizeof(p));
  return p;
}

// Puts the call's table into the pages; n_req < 0: any number of requests.  Returns the requests.
int64_t with_table(svx_pages& p, PyObject* o, int64_t n_req) {
  const at::Tensor& t = tensor(o, "table");
  if (t.dim() != 2 || (n_req >= 0 && t.size(0) != n_req) || t.size(1) > INT32_MAX)
    refuse(SVX_ERR_INVALID_ARG, "table: " + describe(t) + ", expected [requests, max_pages]");
  p.table = static_cast<const int32_t*>(dense(o, at::kInt, {t.size(0), t.size(1)}, p.device, "table"));
  p.max_pages = static_cast<int32_t>(t.size(1));
  return t.size(0);
}

void check(svx_status st) {
  if (st != SVX_OK) refuse(st, g.last_error(nullptr));
}

// The caller's workspace, or one from the caching allocator that belongs to the current stream.
struct Workspace {
  at::Tensor own;
  void* at;
  int64_t bytes;
  Workspace(PyObject* o, int64_t need, int device) {
    if (o == Py_None) {
      own = at::empty({need}, at::TensorOptions().dtype(at::kByte).device(at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(device))));
      at = own.data_ptr();
      bytes = need;
      return;
    }
    const at::Tensor& t = tensor(o, "workspace");
    bytes = t.numel() * t.element_size();
    if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous() || bytes < need)
      refuse(SVX_ERR_INVALID_ARG, "workspace: a dense tensor of at least " + std::to_string(need) + " bytes on cuda:" + std::to_string(device) +
                                      " is needed");
    at = t.data_ptr();
  }
};

void* current_stream(int device) {
  return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
}

// Runs f, which makes the C call, and turns what it throws into a Python exception.
template <typename F>
PyObject* guarded(F&& f) {
  try {
    f();
    Py_RETURN_NONE;
  } catch (const Refused& r) {
    PyObject* e = PyObject_CallFunction(g_error, "is", r.status, r.message.c_str());
    if (e) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
  } catch (const c10::OutOfMemoryError& e) {  // no room for a workspace: torch.OutOfMemoryError, as of torch's own calls
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

bool expect(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, got);
  return got == want;
}

template <typename F>
svx_status without_gil(F&& call) {
  svx_status st;
  Py_BEGIN_ALLOW_THREADS st = call();
  Py_END_ALLOW_THREADS return st;
}

const svx_rope* rope_at(PyObject* o) { return reinterpret_cast<const svx_rope*>(integer(o, "rope")); }

PyObject* set_up(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!expect(n, 13)) return nullptr;
  return guarded([&] {
    g_error = a[0];
    Py_INCREF(g_error);
    auto at = [&](int i) { return reinterpret_cast<void*>(integer(a[i], "address")); };
    g.qk_norm_rope = reinterpret_cast<decltype(g.qk_norm_rope)>(at(1));
    g.append = reinterpret_cast<decltype(g.append)>(at(2));
    g.decode_workspace = reinterpret_cast<decltype(g.decode_workspace)>(at(3));
    g.decode = reinterpret_cast<decltype(g.decode)>(at(4));
    g.evict_workspace = reinterpret_cast<decltype(g.evict_workspace)>(at(5));
    g.evict = reinterpret_cast<decltype(g.evict)>(at(6));
    g.residual_norm = reinterpret_cast<decltype(g.residual_norm)>(at(7));
    g.decode_shared_workspace = reinterpret_cast<decltype(g.decode_shared_workspace)>(at(8));
    g.decode_shared = reinterpret_cast<decltype(g.decode_shared)>(at(9));
    g.cross_attn_workspace = reinterpret_cast<decltype(g.cross_attn_workspace)>(at(10));
    g.cross_attn = reinterpret_cast<decltype(g.cross_attn)>(at(11));
    g.last_error = reinterpret_cast<decltype(g.last_error)>(at(12));
  });
}

// pages(k_pages, v_pages, status) -> the C struct as bytes, without a table
PyObject* pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!expect(n, 3)) return nullptr;
  svx_pages p = {};
  PyObject* done = guarded([&] {
    const at::Tensor &k = tensor(a[0], "k_pages"), &v = tensor(a[1], "v_pages");
    p.dtype = type_code(k, "k_pages");
    if (k.dim() != 4 || k.sizes() != v.sizes() || k.strides() != v.strides() || k.scalar_type() != v.scalar_type() ||
        k.device() != v.device() || !k.is_cuda() || (k.size(3) > 1 && k.stride(3) != 1))
      refuse(SVX_ERR_INVALID_ARG, "k_pages: " + describe(k) + ", v_pages: " + describe(v) +
                                      "; expected equal [pages, page_size, KV heads, head_dim] CUDA tensors with dense rows");
    if (k.size(1) > INT32_MAX || k.size(2) > INT32_MAX || k.size(3) > INT32_MAX)
      refuse(SVX_ERR_INVALID_ARG, "k_pages: a dimension does not fit 32 bits");
    p.device = k.get_device();
    p.k = k.data_ptr();
    p.v = v.data_ptr();
    p.status = static_cast<int32_t*>(dense(a[2], at::kInt, {1}, p.device, "status"));
    p.page_stride = k.stride(0);
    p.tok_stride = k.stride(1);
    p.head_stride = k.stride(2);
    p.n_pages = k.size(0);
    p.page_size = static_cast<int32_t>(k.size(1));
    p.n_kv_heads = static_cast<int32_t>(k.size(2));
    p.head_dim = static_cast<int32_t>(k.size(3));
    p.flags = SVX_POINTERS_CHECKED;
  });
  if (!done) return nullptr;
  Py_DECREF(done);
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&p), sizeof(p));
}

// qk_norm_rope(q, k, v, pos, rope, q_out, k_out, v_out, q_norm, k_norm, eps, n_new, status)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!expect(n, 13)) return nullptr;
  return guarded([&] {
    svx_heads h = heads_of(a[0], a[1], a[2], a[3], a[8], a[9], a[10], a[11]);
    const at::ScalarType type = scalar_of(h.dtype);
    void* q_out = dense(a[5], type, {h.n_req, h.n_q_heads, h.n_tok, h.head_dim}, h.device, "q_out");
    void* k_out = dense(a[6], type, {h.n_req, h.n_tok, h.n_kv_heads, h.head_dim}, h.device, "k_out");
    void* v_out = optional(a[7], type, {h.n_req, h.n_tok, h.n_kv_heads, h.head_dim}, h.device, "v_out");
    h.status = static_cast<int32_t*>(optional(a[12], at::kInt, {1}, h.device, "status"));
    const svx_rope* rope = rope_at(a[4]);
    void* stream = current_stream(h.device);
    check(without_gil([&] { return g.qk_norm_rope(&h, rope, q_out, k_out, v_out, stream); }));
  });
}

// append(pages, q, k, v, pos, rope, table, start, q_out, q_norm, k_norm, eps, n_new, acc, slot_pos)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!expect(n, 15)) return nullptr;
  return guarded([&] {
    svx_pages p = pages_of(a[0]);
    if (a[3] == Py_None) refuse(SVX_ERR_INVALID_ARG, "v is required");
    const svx_heads h = heads_of(a[1], a[2], a[3], a[4], a[9], a[10], a[11], a[12]);
    if (h.device != p.device) refuse(SVX_ERR_INVALID_ARG, "q and the cache are on different devices");
    with_table(p, a[6], h.n_req);
    const int64_t room = static_cast<int64_t>(p.max_pages) * p.page_size;
    const int32_t* start = static_cast<const int32_t*>(dense(a[7], at::kInt, {h.n_req}, p.device, "start"));
    void* q_out = dense(a[8], scalar_of(h.dtype), {h.n_req, h.n_q_heads, h.n_tok, h.head_dim}, p.device, "q_out");
    float* acc = static_cast<float*>(optional(a[13], at::kFloat, {h.n_req, p.n_kv_heads, room}, p.device, "acc"));
    int32_t* slot_pos = static_cast<int32_t*>(optional(a[14], at::kInt, {h.n_req, p.n_kv_heads, room}, p.device, "slot_pos"));
    const svx_rope* rope = rope_at(a[5]);
    void* stream = current_stream(p.device);
    check(without_gil([&] { return g.append(&h, rope, &p, start, q_out, acc, slot_pos, stream); }));
  });
}

// decode(pages, q, table, lens, o, lse, max_len, scale, acc_in, acc_out, workspace)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!expect(n, 11)) return nullptr;
  return guarded([&] {
    svx_pages p = pages_of(a[0]);
    const at::Tensor& q = tensor(a[1], "q");
    if (q.dim() != 4 || q.size(0) > INT32_MAX || q.size(1) > INT32_MAX)
      refuse(SVX_ERR_INVALID_ARG, "q: " + describe(q) + ", expected [requests, heads, 1, head_dim]");
    const int64_t b = q.size(0), hq = q.size(1);
    const at::ScalarType type = scalar_of(p.dtype);
    with_table(p, a[2], b);
    const int64_t room = static_cast<int64_t>(p.max_pages) * p.page_size;
    const void* qp = dense(a[1], type, {b, hq, 1, p.head_dim}, p.device, "q");
    const int32_t* lens = static_cast<const int32_t*>(dense(a[3], at::kInt, {b}, p.device, "lens"));
    void* o = dense(a[4], type, {b, hq, 1, p.head_dim}, p.device, "o");
    float* lse = static_cast<float*>(dense(a[5], at::kFloat, {b, hq, 1}, p.device, "lse"));
    const int64_t max_len = integer(a[6], "max_len");
    const float scale = real(a[7], "scale");
    const float* acc_in = static_cast<const float*>(optional(a[8], at::kFloat, {b, p.n_kv_heads, room}, p.device, "acc_in"));
    float* acc_out = static_cast<float*>(optional(a[9], at::kFloat, {b, p.n_kv_heads, room}, p.device, "acc_out"));
    int64_t need = 0;
    check(g.decode_workspace(&p, static_cast<int32_t>(b), static_cast<int32_t>(hq), max_len, acc_in != nullptr, &need));
    const Workspace ws(a[10], need, p.device);
    void* stream = current_stream(p.device);
    check(without_gil([&] {
      return g.decode(&p, static_cast<int32_t>(b), static_cast<int32_t>(hq), qp, lens, max_len, scale, o, lse, acc_in, acc_out, ws.at,
                      ws.bytes, stream);
    }));
  });
}

// decode_shared(pages, q, prefix_table, prefix_lens, first, table, lens, o, lse, max_prefix, max_len, scale, workspace)
PyObject* decode_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!expect(n, 13)) return nullptr;
  return guarded([&] {
    svx_pages p = pages_of(a[0]);
    const at::Tensor& q = tensor(a[1], "q");
    if (q.dim() != 4 || q.size(0) > INT32_MAX || q.size(1) > INT32_MAX)
      refuse(SVX_ERR_INVALID_ARG, "q: " + describe(q) + ", expected [requests, heads, 1, head_dim]");
    const int64_t b = q.size(0), hq = q.size(1);
    const at::ScalarType type = scalar_of(p.dtype);
    with_table(p, a[5], b);
    svx_prefixes f = {};
    const at::Tensor& far = tensor(a[2], "prefix_table");
    if (far.dim() != 2 || far.size(0) > INT32_MAX || far.size(1) > INT32_MAX)
      refuse(SVX_ERR_INVALID_ARG, "prefix_table: " + describe(far) + ", expected [prefixes, max_pages]");
    f.n_prefix = static_cast<int32_t>(far.size(0));
    f.max_pages = static_cast<int32_t>(far.size(1));
    f.table = static_cast<const int32_t*>(dense(a[2], at::kInt, {far.size(0), far.size(1)}, p.device, "prefix_table"));
    f.len = static_cast<const int32_t*>(dense(a[3], at::kInt, {far.size(0)}, p.device, "prefix_lens"));
    f.first = static_cast<const int32_t*>(dense(a[4], at::kInt, {far.size(0) + 1}, p.device, "first"));
    f.max_len = integer(a[9], "max_prefix");
    const void* qp = dense(a[1], type, {b, hq, 1, p.head_dim}, p.device, "q");
    const int32_t* lens = static_cast<const int32_t*>(dense(a[6], at::kInt, {b}, p.device, "lens"));
    void* o = dense(a[7], type, {b, hq, 1, p.head_dim}, p.device, "o");
    float* lse = static_cast<float*>(dense(a[8], at::kFloat, {b, hq, 1}, p.device, "lse"));
    const int64_t max_len = integer(a[10], "max_len");
    const float scale = real(a[11], "scale");
    int64_t need = 0;
    check(g.decode_shared_workspace(&p, static_cast<int32_t>(b), static_cast<int32_t>(hq), &f, max_len, &need));
    const Workspace ws(a[12], need, p.device);
    void* stream = current_stream(p.device);
    check(without_gil([&] {
      return g.decode_shared(&p, static_cast<int32_t>(b), static_cast<int32_t>(hq), qp, &f, lens, max_len, scale, o, lse, ws.at, ws.bytes,
                             stream);
    }));
  });
}

// cross_attn(q, k, v, o, lse, lens, mask, scale, status, workspace)
PyObject* cross_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!expect(n, 10)) return nullptr;
  return guarded([&] {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &o = tensor(a[3], "o");
    svx_cross c = {};
    c.dtype = type_code(q, "q");
    const at::ScalarType type = q.scalar_type();
    if (q.dim() != 4 || !q.is_cuda())
      refuse(SVX_ERR_INVALID_ARG, "q: " + describe(q) + ", expected [requests, heads, tokens, head_dim] on a CUDA device");
    c.device = q.get_device();
    for (int64_t i = 0; i < 4; ++i)
      if (q.size(i) > INT32_MAX || (k.dim() == 4 && k.size(i) > INT32_MAX))
        refuse(SVX_ERR_INVALID_ARG, "q or k: a dimension does not fit 32 bits");
    auto rows_dense = [&](const at::Tensor& t, const char* what) {
      if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != c.device || t.dim() != 4 || (t.size(3) > 1 && t.stride(3) != 1)) {
        std::ostringstream s;
        s << what << ": " << describe(t) << "; expected " << type << " with four dimensions, the last dense, on cuda:" << c.device;
        refuse(SVX_ERR_INVALID_ARG, s.str());
      }
    };
    rows_dense(q, "q");
    rows_dense(k, "k");
    rows_dense(v, "v");
    rows_dense(o, "o");
    if (o.sizes() != q.sizes()) refuse(SVX_ERR_INVALID_ARG, "o: " + describe(o) + ", expected q's shape");
    bool alike = v.sizes() == k.sizes();
    for (int64_t i = 0; alike && i < 3; ++i) alike = k.size(i) <= 1 || v.stride(i) == k.stride(i);  // (one entry: never stepped over)
    if (!alike) {
      std::ostringstream s;
      s << "v: " << describe(v) << ", strides " << v.strides() << "; expected k's shape and strides: " << describe(k) << ", strides " << k.strides();
      refuse(SVX_ERR_INVALID_ARG, s.str());
    }
    if (k.size(0) != q.size(0) || k.size(3) != q.size(3))
      refuse(SVX_ERR_INVALID_ARG, "k: " + describe(k) + ", expected [requests, states, KV heads, head_dim] of q's requests and head_dim");
    c.n_req = static_cast<int32_t>(q.size(0));
    c.n_q_heads = static_cast<int32_t>(q.size(1));
    c.n_tok = static_cast<int32_t>(q.size(2));
    c.head_dim = static_cast<int32_t>(q.size(3));
    c.n_states = static_cast<int32_t>(k.size(1));
    c.n_kv_heads = static_cast<int32_t>(k.size(2));
    c.q = q.data_ptr();
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.o = o.data_ptr();
    c.q_req = q.stride(0), c.q_head = q.stride(1), c.q_tok = q.stride(2);
    c.kv_req = k.stride(0), c.kv_state = k.stride(1), c.kv_head = k.stride(2);
    c.o_req = o.stride(0), c.o_head = o.stride(1), c.o_tok = o.stride(2);
    c.lse = static_cast<float*>(optional(a[4], at::kFloat, {c.n_req, c.n_q_heads, c.n_tok}, c.device, "lse"));
    c.len = static_cast<const int32_t*>(optional(a[5], at::kInt, {c.n_req}, c.device, "lens"));
    if (a[6] != Py_None) {
      const at::Tensor& m = tensor(a[6], "mask");
      if (m.scalar_type() != at::kBool || m.dim() != 2 || m.size(0) != c.n_req || m.size(1) != c.n_states || !m.is_cuda() ||
          m.get_device() != c.device || (c.n_states > 1 && m.stride(1) != 1)) {
        std::ostringstream s;
        s << "mask: " << describe(m) << "; expected bool [" << c.n_req << ", " << c.n_states << "] with dense rows on cuda:" << c.device;
        refuse(SVX_ERR_INVALID_ARG, s.str());
      }
      c.mask = static_cast<const uint8_t*>(m.data_ptr());
      c.mask_req = c.n_req > 1 ? m.stride(0) : 0;
    }
    c.scale = real(a[7], "scale");
    c.status = static_cast<int32_t*>(optional(a[8], at::kInt, {1}, c.device, "status"));
    c.flags = SVX_POINTERS_CHECKED;
    int64_t need = 0;
    check(g.cross_attn_workspace(&c, &need));
    const Workspace ws(a[9], need, c.device);
    void* stream = current_stream(c.device);
    check(without_gil([&] { return g.cross_attn(&c, ws.at, ws.bytes, stream); }));
  });
}

// evict(pages, table, lens, budget, sink, recent, next_pos, acc_in, pos_in, acc_out, pos_out, len_out, max_len, workspace)
PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!expect(n, 14)) return nullptr;
  return guarded([&] {
    svx_pages p = pages_of(a[0]);
    const int64_t b = with_table(p, a[1], -1);
    if (b > INT32_MAX) refuse(SVX_ERR_INVALID_ARG, "table: too many requests");
    const int64_t room = static_cast<int64_t>(p.max_pages) * p.page_size;
    const int32_t budget = integer32(a[3], "budget"), sink = integer32(a[4], "sink"), recent = integer32(a[5], "recent");
    const int64_t max_len = integer(a[12], "max_len");
    const int32_t* lens = static_cast<const int32_t*>(dense(a[2], at::kInt, {b}, p.device, "lens"));
    const int32_t* next_pos = static_cast<const int32_t*>(dense(a[6], at::kInt, {b}, p.device, "next_pos"));
    const float* acc_in = static_cast<const float*>(dense(a[7], at::kFloat, {b, p.n_kv_heads, room}, p.device, "acc_in"));
    const int32_t* pos_in = static_cast<const int32_t*>(dense(a[8], at::kInt, {b, p.n_kv_heads, room}, p.device, "pos_in"));
    float* acc_out = static_cast<float*>(dense(a[9], at::kFloat, {b, p.n_kv_heads, room}, p.device, "acc_out"));
    int32_t* pos_out = static_cast<int32_t*>(dense(a[10], at::kInt, {b, p.n_kv_heads, room}, p.device, "pos_out"));
    int32_t* len_out = static_cast<int32_t*>(dense(a[11], at::kInt, {b}, p.device, "len_out"));
    int64_t need = 0;
    check(g.evict_workspace(&p, static_cast<int32_t>(b), max_len, budget, &need));
    const Workspace ws(a[13], need, p.device);
    void* stream = current_stream(p.device);
    check(without_gil([&] {
      return g.evict(&p, static_cast<int32_t>(b), lens, max_len, budget, sink, recent, next_pos, acc_in, pos_in, acc_out, pos_out,
                     len_out, ws.at, ws.bytes, stream);
    }));
  });
}

// Elements between the rows of a tensor [..., dim], evenly spaced over its leading dimensions; 0: one row.
int64_t row_stride(const at::Tensor& t, const char* what) {
  int64_t stride = 0, next = 0;  // of the last dimension with more than one entry, and what the one before it needs
  bool any = false, even = t.dim() >= 1 && (t.size(-1) <= 1 || t.stride(-1) == 1);
  for (int64_t i = t.dim() - 2; i >= 0; --i) {
    if (t.size(i) <= 1) continue;
    if (!any) stride = t.stride(i);
    else even = even && t.stride(i) == next;
    any = true;
    next = t.stride(i) * t.size(i);
  }
  if (!even) {
    std::ostringstream s;
    s << what << ": strides " << t.strides() << ": rows must be dense, and evenly spaced over the leading dimensions";
    refuse(SVX_ERR_INVALID_ARG, s.str());
  }
  return stride;
}

// residual_norm(h, y, h_out, x_out, norm, eps, post_norm, post_eps, gate, act, alpha, beta)
PyObject* residual_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!expect(n, 12)) return nullptr;
  return guarded([&] {
    const at::Tensor& h = tensor(a[0], "h");
    if (!h.is_cuda() || h.dim() < 1 || h.numel() == 0 || h.size(-1) > INT32_MAX)
      refuse(SVX_ERR_INVALID_ARG, "h: " + describe(h) + ", expected [..., dim] on a CUDA device");
    svx_residual r = {};
    r.device = h.get_device();
    r.dim = static_cast<int32_t>(h.size(-1));
    r.rows = h.numel() / r.dim;
    // the type of everything but the stream: that of the first of these that is given
    const int of = a[1] != Py_None ? 1 : a[3] != Py_None ? 3 : 0;
    r.dtype = type_code(tensor(a[of], of == 1 ? "y" : of == 3 ? "x_out" : "h"), of == 1 ? "y" : of == 3 ? "x_out" : "h");
    const at::ScalarType type = scalar_of(r.dtype), stream_type = h.scalar_type();
    if (stream_type != type && stream_type != at::kFloat)
      refuse(SVX_ERR_UNSUPPORTED, "h: " + describe(h) + "; expected the type of the block's output or torch.float32");
    r.stream_dtype = stream_type == at::kFloat ? SVX_FP32 : r.dtype;
    auto rows = [&](int i, at::ScalarType t, const char* what, int64_t* stride) -> void* {
      if (a[i] == Py_None) return nullptr;
      const at::Tensor& x = tensor(a[i], what);
      if (x.scalar_type() != t || x.sizes() != h.sizes() || !x.is_cuda() || x.get_device() != r.device) {
        std::ostringstream s;
        s << what << ": " << describe(x) << "; expected " << t << " " << h.sizes() << " on cuda:" << r.device;
        refuse(SVX_ERR_INVALID_ARG, s.str());
      }
      *stride = row_stride(x, what);
      return x.data_ptr();
    };
    r.h = rows(0, stream_type, "h", &r.h_stride);
    r.y = rows(1, type, "y", &r.y_stride);
    r.h_out = rows(2, stream_type, "h_out", &r.h_out_stride);
    r.x_out = rows(3, type, "x_out", &r.x_stride);
    r.norm = optional(a[4], type, {r.dim}, r.device, "norm");
    r.eps = real(a[5], "eps");
    r.post_norm = optional(a[6], type, {r.dim}, r.device, "post_norm");
    r.post_eps = -1.f;
    if (a[7] != Py_None) {
      r.post_eps = real(a[7], "post_eps");
      if (!(r.post_eps >= 0.f)) refuse(SVX_ERR_INVALID_ARG, "post_eps must be >= 0, or None for no norm after the block");
    }
    if (a[8] != Py_None) {
      const at::Tensor& gate = tensor(a[8], "gate");
      if (gate.dim() == 1 && gate.size(0) == 1) {
        r.gate_kind = SVX_GATE_SCALAR;
        r.gate = dense(a[8], type, {1}, r.device, "gate");
      } else if (gate.dim() == 1) {
        r.gate_kind = SVX_GATE_CHANNEL;
        r.gate = dense(a[8], type, {r.dim}, r.device, "gate");
      } else {
        r.gate_kind = SVX_GATE_ELEMENT;
        r.gate = rows(8, type, "gate", &r.gate_stride);
      }
    }
    r.act = integer32(a[9], "act");
    r.alpha = real(a[10], "alpha");
    r.beta = real(a[11], "beta");
    r.flags = SVX_POINTERS_CHECKED;
    void* stream = current_stream(r.device);
    check(without_gil([&] { return g.residual_norm(&r, stream); }));
  });
}

#define SVX_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {SVX_METHOD(set_up), SVX_METHOD(pages), SVX_METHOD(qk_norm_rope), SVX_METHOD(append), SVX_METHOD(decode),
                         SVX_METHOD(evict), SVX_METHOD(residual_norm),
                         SVX_METHOD(decode_shared), SVX_METHOD(cross_attn), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "svx_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_svx_torch() { return PyModule_Create(&module); }
