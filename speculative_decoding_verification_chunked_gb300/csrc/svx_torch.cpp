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
  if (!expect(n, 8)) return nullptr;
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
    g.last_error = reinterpret_cast<decltype(g.last_error)>(at(7));
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

#define SVX_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {SVX_METHOD(set_up), SVX_METHOD(pages), SVX_METHOD(qk_norm_rope), SVX_METHOD(append), SVX_METHOD(decode),
                         SVX_METHOD(evict), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "svx_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_svx_torch() { return PyModule_Create(&module); }
