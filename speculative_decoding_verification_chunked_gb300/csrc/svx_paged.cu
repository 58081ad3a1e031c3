// Host side shared by the paged-cache entry points: argument checks, and the rotation's fixed-point phases.
#include "svx_paged.h"

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

namespace svx {

void set_thread_error(const char* msg);  // svx_runtime.cu: message for svx_last_error(NULL)

svx_status paged_fail(svx_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  try {
    set_thread_error(buf);
  } catch (const std::bad_alloc&) {  // no memory for the message: the status still tells
  }
  return st;
}

bool on_device(const void* p, int device) {
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return a.type == cudaMemoryTypeManaged || (a.type == cudaMemoryTypeDevice && a.device == device);
}

int sm_count(int device) {
  static std::atomic<int> known[64];  // a property of the device: asked once
  if (device >= 0 && device < 64) {
    const int n = known[device].load(std::memory_order_relaxed);
    if (n > 0) return n;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (device >= 0 && device < 64) known[device].store(n, std::memory_order_relaxed);
  return n;
}

svx_status paged_view(const svx_pages* c, int32_t n_req, PageView* out) {
  if (!c) return paged_fail(SVX_ERR_INVALID_ARG, "cache is NULL");
  if (n_req < 1 || n_req > kMaxReq) return paged_fail(SVX_ERR_INVALID_ARG, "n_req must be in [1, %d]", kMaxReq);
  if (c->dtype != SVX_BF16 && c->dtype != SVX_FP16)
    return paged_fail(SVX_ERR_UNSUPPORTED, "dtype must be SVX_BF16 or SVX_FP16");
  if (c->head_dim != 64 && c->head_dim != 128) return paged_fail(SVX_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (c->n_kv_heads < 1 || c->n_kv_heads > 4096)
    return paged_fail(SVX_ERR_INVALID_ARG, "n_kv_heads must be in [1, 4096]");
  if (c->page_size < 1 || c->max_pages < 1 ||
      static_cast<int64_t>(c->page_size) * c->max_pages > 0x7fffffffLL)
    return paged_fail(SVX_ERR_INVALID_ARG, "page_size and max_pages must be positive with a product below 2^31");
  if (c->n_pages < 1 || c->n_pages > 0x7fffffffLL)
    return paged_fail(SVX_ERR_INVALID_ARG, "n_pages must be in [1, 2^31)");
  const int64_t s[3] = {c->page_stride, c->tok_stride, c->head_stride}, n[3] = {c->n_pages, c->page_size, c->n_kv_heads};
  int64_t extent = c->head_dim;
  for (int i = 0; i < 3; ++i) {
    // (a stride over a dimension of one entry is never stepped over)
    if (n[i] > 1 && (s[i] < c->head_dim || s[i] % 8 || s[i] > (int64_t{1} << 46) / n[i]))
      return paged_fail(SVX_ERR_INVALID_ARG, "page, slot and head strides must be multiples of 8 elements, at least head_dim");
    extent += (n[i] - 1) * s[i];
  }
  if (!c->k || !c->v || !is_aligned(c->k, 16) || !is_aligned(c->v, 16))
    return paged_fail(SVX_ERR_INVALID_ARG, "k and v pages must be 16-byte aligned device pointers");
  if (!c->table || !c->status || !is_aligned(c->table, 4) || !is_aligned(c->status, 4))
    return paged_fail(SVX_ERR_INVALID_ARG, "table and status must be device pointers");
  *out = PageView{c->k,
                  c->v,
                  c->table,
                  c->status,
                  s[0],
                  s[1],
                  s[2],
                  extent,
                  static_cast<int32_t>(c->n_pages),
                  c->page_size,
                  c->max_pages,
                  c->n_kv_heads,
                  n_req,
                  c->page_size * c->max_pages,
                  0,
                  0};
  // round-up multiplication: with 2^l >= page_size, mul = floor(2^32 (2^l - page_size) / page_size) + 1
  uint32_t l = 0;
  while ((int64_t{1} << l) < c->page_size) ++l;
  out->div_shift = l;
  out->div_mul = static_cast<uint32_t>(((uint64_t{1} << 32) * ((uint64_t{1} << l) - c->page_size)) / c->page_size + 1);
  return SVX_OK;
}

namespace {
thread_local int64_t t_clip[kClips] = {-1, -1, -1};
thread_local bool t_expire = false;
}

bool expire_waits() { return t_expire; }

int64_t clipped(PagedBuffer kind, int64_t extent) {
  return t_clip[kind] >= 0 && t_clip[kind] < extent ? t_clip[kind] : extent;
}

namespace {

// True if a row that begins `off` elements behind a row of the pool shares elements with one of the first `dims` dimensions'
// rows (strides ascending, each at least the span of those before it, so that only the two nearest multiples of the largest
// can come within reach).
bool meets_a_row(int64_t off, const int64_t* stride, const int64_t* n, int dims, int64_t d) {
  if (dims == 0) return off < d && -off < d;
  const int64_t s = stride[dims - 1], most = n[dims - 1] - 1;
  int64_t a = off / s;
  if (off < 0 && a * s != off) --a;  // rounded down
  for (int i = 0; i < 2; ++i, ++a)
    if (a <= most && -a <= most && meets_a_row(off - a * s, stride, n, dims - 1, d)) return true;
  return false;
}

}  // namespace

bool pools_collide(const svx_pages* c, bool same_pool_too) {
  int64_t stride[3], n[3];
  int dims = 0;
  const int64_t s[3] = {c->page_stride, c->tok_stride, c->head_stride}, count[3] = {c->n_pages, c->page_size, c->n_kv_heads};
  for (int i = 0; i < 3; ++i) {
    if (count[i] == 1) continue;
    int at = dims++;
    for (; at > 0 && stride[at - 1] > s[i]; --at) {
      stride[at] = stride[at - 1];
      n[at] = n[at - 1];
    }
    stride[at] = s[i];
    n[at] = count[i];
  }
  int64_t span = c->head_dim;
  for (int i = 0; i < dims; ++i) {
    if (stride[i] < span) return true;  // rows of one pool overlap
    span += (n[i] - 1) * stride[i];
  }
  if (c->k == c->v) return same_pool_too;
  // (16-byte aligned pointers: whole elements apart)
  const int64_t apart = (static_cast<const char*>(c->v) - static_cast<const char*>(c->k)) / 2;
  return apart < span && -apart < span && meets_a_row(apart, stride, n, dims, c->head_dim);
}

// f / (2 pi) mod 1 in units of 2^-64, rounded down (a negative one up), for |f| < 2^20: whole turns drop out, since positions
// are whole numbers.  f = m 2^e with a whole m < 2^53, so m times 1 / (2 pi) in 128 bits, shifted, is the fraction to its last
// bit; a product in double has lost it for the fast pairs (f = 1e5 at position 2^31: 2^-9 of a turn).
static uint64_t turn_fraction(double f) {
  constexpr uint64_t kHigh = 0x28be60db9391054aull, kLow = 0x7f09d5f47d4d3770ull;  // 2^128 / (2 pi)
  int e = 0;
  const double scaled = std::frexp(std::fabs(f), &e);
  const uint64_t m = static_cast<uint64_t>(std::ldexp(scaled, 53));
  // f = m 2^(e - 53): shift the product's 128 fraction bits to 64 and by the exponent
  const int shift = 64 + 53 - e;
  if (shift >= 192) return 0;  // below 2^-64 of a turn (the product has 181 bits)
  const unsigned __int128 low = static_cast<unsigned __int128>(m) * kLow;
  const unsigned __int128 high = static_cast<unsigned __int128>(m) * kHigh + (low >> 64);  // in units of 2^64
  const uint64_t turns = static_cast<uint64_t>(high >> (shift - 64));  // shift - 64 = 53 - e >= 33
  return f < 0 ? 0 - turns : turns;
}

}  // namespace svx

extern "C" svx_status svx_debug_clip_paged(int32_t buffer, int64_t elements) {
  if (buffer < 0 || buffer >= svx::kClips) return svx::paged_fail(SVX_ERR_INVALID_ARG, "buffer must be 0, 1 or 2");
  svx::t_clip[buffer] = elements < 0 ? -1 : elements;
  return SVX_OK;
}

extern "C" svx_status svx_debug_expire_rows(int32_t on) {
  svx::t_expire = on != 0;
  return SVX_OK;
}

extern "C" svx_status svx_rope_init(svx_rope* rope, int32_t rot_dim, int32_t neighbours, const double* inv_freq,
                                    float scale) {
  using svx::paged_fail;
  if (!rope) return paged_fail(SVX_ERR_INVALID_ARG, "rope is NULL");
  if (rot_dim < 0 || rot_dim > 128 || rot_dim % 16)
    return paged_fail(SVX_ERR_INVALID_ARG, "rot_dim must be a multiple of 16 in [0, 128]");
  if (rot_dim && !inv_freq) return paged_fail(SVX_ERR_INVALID_ARG, "inv_freq is NULL");
  if (!std::isfinite(scale)) return paged_fail(SVX_ERR_INVALID_ARG, "scale must be finite");
  svx_rope r = {};
  for (int i = 0; i < rot_dim / 2; ++i) {
    if (!(std::fabs(inv_freq[i]) < 1048576.0))
      return paged_fail(SVX_ERR_INVALID_ARG, "inv_freq[%d] must be finite, below 2^20 in magnitude", i);
    r.turns[i] = svx::turn_fraction(inv_freq[i]);
  }
  r.scale = scale;
  r.rot_dim = rot_dim;
  r.neighbours = neighbours ? 1 : 0;
  *rope = r;
  return SVX_OK;
}
