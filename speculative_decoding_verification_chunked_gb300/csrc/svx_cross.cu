// Attention of a decoder's tokens to an encoder's states: the entry point, its checks and launches.
//
//   O[b, h, j] = sum_t p_t v_t / sum_t p_t,  p_t = e^(scale q[b, h, j].k_t - m),  t < len[b] with mask[b, t],  LSE = m + ln sum_t p_t
//
// There is no order among states, so the tokens of a request and the query heads of a KV head are alike: rows of one product
// with the same keys.
//
// Up to 16 rows (one token, few query heads to a KV head) attend_kernel brings K and V in once and its products are small beside them;
// with more, rows_kernel.  A request whose states are all hidden costs its keys' words of the mask and nothing of K and V.
// Measured: one token x 1500 states of 16 heads 9.0 us (two launches and their latencies); 32 requests of one token, 32 heads over 8 KV heads,
// up to 6404 states of which 20% are hidden 59 us (the bytes of all states below the lengths: 63); 4 x 448 tokens x 701 to 1500
// states of 16 heads 23 us; 8192 x 16384 1334 us among other passes, 1204 alone.
#include "svx_rows.cuh"

namespace svx {
namespace {

constexpr int64_t kMaxBlocks = 65535;

struct CrossView {
  bool many;  // rows of a request and KV head: more than one-token attention's kernels take at a time
  Sizes z;
  RowSizes rz;
  size_t total;
  AttendParams p;
};

bool stride_ok(int64_t n, int64_t s) { return n <= 1 || (s >= 0 && s % 8 == 0 && s <= (int64_t{1} << 46) / n); }

int64_t span_of(std::initializer_list<int64_t> n, std::initializer_list<int64_t> s, int64_t d) {
  int64_t e = d;
  for (size_t i = 0; i < n.size(); ++i)
    if (n.begin()[i] > 1) e += (n.begin()[i] - 1) * s.begin()[i];
  return e;
}

// True if no two rows of d elements meet: sorted, each stride is at least the span of the dimensions below it.
bool rows_apart(int64_t (&n)[3], int64_t (&s)[3], int64_t d) {
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (s[j] < s[i]) {
        std::swap(s[i], s[j]);
        std::swap(n[i], n[j]);
      }
  int64_t span = d;
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (s[i] < span) return false;
    span += (n[i] - 1) * s[i];
  }
  return true;
}

// Everything but the pointers, and but for the sizes that hang on the SMs.
svx_status cross_view(const svx_cross* c, CrossView* out) {
  if (!c) return paged_fail(SVX_ERR_INVALID_ARG, "the arguments are NULL");
  const svx_cross& a = *c;
  if (a.dtype != SVX_BF16 && a.dtype != SVX_FP16)
    return paged_fail(SVX_ERR_UNSUPPORTED, "dtype must be SVX_BF16 or SVX_FP16");
  if (a.head_dim != 64 && a.head_dim != 128) return paged_fail(SVX_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (a.n_req < 1 || a.n_req > kMaxReq) return paged_fail(SVX_ERR_INVALID_ARG, "n_req must be in [1, %d]", kMaxReq);
  if (a.n_tok < 1 || a.n_states < 0 || a.n_states > 0x7fffffff - 256)
    return paged_fail(SVX_ERR_INVALID_ARG, "n_tok must be at least 1, n_states in [0, 2^31 - 256)");
  if (a.n_kv_heads < 1 || a.n_q_heads < a.n_kv_heads || a.n_q_heads % a.n_kv_heads || a.n_q_heads > 4096)
    return paged_fail(SVX_ERR_INVALID_ARG, "n_q_heads must be a positive multiple of n_kv_heads, at most 4096");
  const int64_t B = a.n_req, N = a.n_tok, S = a.n_states, Hq = a.n_q_heads, Hkv = a.n_kv_heads;
  if (!stride_ok(B, a.q_req) || !stride_ok(Hq, a.q_head) || !stride_ok(N, a.q_tok) || !stride_ok(B, a.kv_req) ||
      !stride_ok(Hkv, a.kv_head) || !stride_ok(S, a.kv_state) || !stride_ok(B, a.o_req) || !stride_ok(Hq, a.o_head) ||
      !stride_ok(N, a.o_tok))
    return paged_fail(SVX_ERR_INVALID_ARG, "strides must be multiples of 8 elements, not negative");
  int64_t n[3] = {B, Hq, N}, s[3] = {a.o_req, a.o_head, a.o_tok};
  if (!rows_apart(n, s, a.head_dim)) return paged_fail(SVX_ERR_INVALID_ARG, "rows of o overlap");
  if (a.mask && (a.mask_req < 0 || (B > 1 && a.mask_req > (int64_t{1} << 46) / B)))
    return paged_fail(SVX_ERR_INVALID_ARG, "mask_req must not be negative");
  const int64_t rows = N * (Hq / Hkv), blocks = (rows + kRowsMax - 1) / kRowsMax;
  const int ct = kChunkBytes / (2 * a.head_dim);
  const int64_t per_item = (S + ct - 1) / ct, chunks = B * Hkv * blocks * per_item;
  if (blocks > kMaxBlocks || chunks > 0x7fffffff)
    return paged_fail(SVX_ERR_UNSUPPORTED, "n_req * heads * n_tok * n_states is too large (%lld chunks, at most 2^31 - 1)",
                      static_cast<long long>(chunks));
  // (8 requests of 32 heads and 8 KV heads, 16384 states: 16 rows 93 us by attend_kernel, 94 by rows_kernel; 20 rows 172 and 95; 1500
  // states 21 and 22, 26 and 22)
  out->many = rows > kRowsMax;
  out->z.max_len = static_cast<int32_t>(S);
  out->z.blocks = static_cast<int32_t>(blocks);
  AttendParams& p = out->p;
  p.pages.page_stride = B > 1 ? a.kv_req : 0;
  p.pages.tok_stride = S > 1 ? a.kv_state : 0;
  p.pages.head_stride = Hkv > 1 ? a.kv_head : 0;
  p.pages.extent = span_of({B, S, Hkv}, {a.kv_req, a.kv_state, a.kv_head}, a.head_dim);
  p.pages.n_pages = a.n_req;
  p.pages.page_size = std::max(a.n_states, 1);
  p.pages.max_pages = 1;
  p.pages.n_kv_heads = a.n_kv_heads;
  p.pages.n_req = a.n_req;
  p.pages.cap = p.pages.page_size;
  p.mask_stride = a.mask_req;
  p.q_b = B > 1 ? a.q_req : 0;
  p.q_h = Hq > 1 ? a.q_head : 0;
  p.q_n = N > 1 ? a.q_tok : 0;
  p.o_b = B > 1 ? a.o_req : 0;
  p.o_h = Hq > 1 ? a.o_head : 0;
  p.o_n = N > 1 ? a.o_tok : 0;
  p.n_tok = a.n_tok;
  p.rows = static_cast<int32_t>(rows);
  p.n_q = a.n_q_heads;
  p.group = a.n_q_heads / a.n_kv_heads;
  return SVX_OK;
}

svx_status cross_sizes(const svx_cross& a, CrossView* v) {
  const int sms = sm_count(a.device);
  if (sms <= 0) return paged_fail(SVX_ERR_CUDA, "cannot read the SM count");
  const int64_t items = static_cast<int64_t>(a.n_req) * a.n_kv_heads;
  if (v->many) {
    const int item_rows = item_rows_for(v->p.rows);
    size_rows(&v->rz, items * ((v->p.rows + item_rows - 1) / item_rows), (static_cast<int64_t>(a.n_states) + kKeyTile - 1) / kKeyTile, item_rows,
              a.head_dim, sms, 0, true);
    v->total = v->rz.total;
    return SVX_OK;
  }
  const int ct = kChunkBytes / (2 * a.head_dim);
  const int64_t per_item = (static_cast<int64_t>(a.n_states) + ct - 1) / ct, chunks = items * v->z.blocks * per_item;
  v->z.whole = per_item <= kWholeItem && chunks <= sms * per_item;  // as in one-token attention over pages
  size_pieces(&v->z, chunks, a.head_dim, sms);
  v->total = v->z.total;
  return SVX_OK;
}

template <typename T, int D>
cudaError_t launch_cross(const AttendParams& p, bool many, int device, cudaStream_t s) {
  if (many) {
    const cudaError_t e = launch_rows<T, kDense, D>(p, device, s);
    if (e != cudaSuccess || p.row_ctas == 1 || p.row_whole) return e;
    const int jobs = (p.row_ctas - 1) * (p.item_rows / 32) * (D / 32);
    return launch_pdl(join_rows<T, kDense, D>, dim3(std::min(jobs, 3 * p.row_ctas)), dim3(kWarps * 32), 0, s, p);  // (3 an SM are resident)
  }
  const cudaError_t e =
      p.rows > 8 ? launch_attend<T, kDense, D, true, false>(p, device, s) : launch_attend<T, kDense, D, false, false>(p, device, s);
  if (e != cudaSuccess || p.whole) return e;
  return launch_pdl(join_kernel<T, kDense, D, false>, dim3(p.pages.n_req * p.pages.n_kv_heads, p.blocks), dim3(kWarps * 32), 0, s, p);
}

}  // namespace
}  // namespace svx

extern "C" svx_status svx_cross_attn_workspace(const svx_cross* c, int64_t* bytes) {
  if (!bytes) return svx::paged_fail(SVX_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = 0;
  svx::CrossView v = {};
  svx_status st = svx::cross_view(c, &v);
  if (st == SVX_OK) st = svx::cross_sizes(*c, &v);
  if (st == SVX_OK) *bytes = static_cast<int64_t>(v.total);
  return st;
}

extern "C" svx_status svx_cross_attn(const svx_cross* c, void* workspace, int64_t workspace_bytes, void* stream) {
  using svx::paged_fail;
  svx::CrossView v = {};
  svx_status st = svx::cross_view(c, &v);
  if (st != SVX_OK) return st;
  const svx_cross& a = *c;
  svx::AttendParams& p = v.p;
  if (!a.q || !a.o || !svx::is_aligned(a.q, 16) || !svx::is_aligned(a.o, 16))
    return paged_fail(SVX_ERR_INVALID_ARG, "q and o must be 16-byte aligned device pointers");
  if (a.n_states && (!a.k || !a.v || !svx::is_aligned(a.k, 16) || !svx::is_aligned(a.v, 16)))
    return paged_fail(SVX_ERR_INVALID_ARG, "k and v must be 16-byte aligned device pointers");
  if (!svx::words_aligned({a.lse, a.len, a.status}))
    return paged_fail(SVX_ERR_INVALID_ARG, "lse, len and status must be 4-byte aligned");
  if (!svx::log2_scale(a.scale, a.head_dim, &p.scale))
    return paged_fail(SVX_ERR_INVALID_ARG, "scale must be positive and below 2^128 ln 2, or 0");
  const int64_t B = a.n_req, N = a.n_tok, Hq = a.n_q_heads;
  const size_t states = a.n_states ? static_cast<size_t>(p.pages.extent) * 2 : 0;
  const svx::Span q = {a.q, static_cast<size_t>(svx::span_of({B, Hq, N}, {a.q_req, a.q_head, a.q_tok}, a.head_dim)) * 2},
                  o = {a.o, static_cast<size_t>(svx::span_of({B, Hq, N}, {a.o_req, a.o_head, a.o_tok}, a.head_dim)) * 2},
                  lse = {a.lse, static_cast<size_t>(B * Hq * N) * 4}, len = {a.len, static_cast<size_t>(B) * 4},
                  mask = {a.mask, a.n_states ? static_cast<size_t>((B - 1) * a.mask_req + a.n_states) : 0}, status = {a.status, 4},
                  k = {a.n_states ? a.k : nullptr, states}, v_span = {a.n_states ? a.v : nullptr, states};
  if (svx::any_overlap({o, lse, status}, {q, k, v_span, len, mask}))
    return paged_fail(SVX_ERR_INVALID_ARG, "an output overlaps an input or another output");
  st = svx::cross_sizes(a, &v);
  if (st != SVX_OK) return st;
  if (!workspace || !svx::is_aligned(workspace, 256) || workspace_bytes < static_cast<int64_t>(v.total))
    return paged_fail(SVX_ERR_INVALID_ARG, "workspace must be 256-byte aligned, of at least %zu bytes", v.total);
  if (svx::any_overlap({{workspace, v.total}}, {q, k, v_span, len, mask, o, lse, status}))
    return paged_fail(SVX_ERR_INVALID_ARG, "the workspace overlaps another buffer");
  svx::PagedDevice dev(a.device);
  if (!dev.ok) return paged_fail(SVX_ERR_CUDA, "cannot use device %d", a.device);
  const void* ptrs[] = {a.q, k.p, v_span.p, a.o, a.lse, a.len, a.mask, a.status, workspace};
  for (const void* x : ptrs)
    if (x && !(a.flags & SVX_POINTERS_CHECKED) && !svx::on_device(x, a.device))
      return paged_fail(SVX_ERR_INVALID_ARG, "a pointer is not memory of device %d", a.device);

  p.pages.k = const_cast<void*>(a.k);
  p.pages.v = const_cast<void*>(a.v);
  p.pages.status = a.status;
  p.pages.extent = svx::clipped(svx::kClipPool, p.pages.extent);
  p.q = a.q;
  p.len = a.len;
  p.mask = a.mask;
  p.o = a.o;
  p.lse = a.lse;
  svx::place_pieces(p, v.z, static_cast<char*>(workspace));  // (with many rows: the bounds alone)
  if (v.many) svx::place_rows(p, v.rz, static_cast<char*>(workspace));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a.dtype == SVX_BF16)
    e = a.head_dim == 128 ? svx::launch_cross<__nv_bfloat16, 128>(p, v.many, a.device, s) : svx::launch_cross<__nv_bfloat16, 64>(p, v.many, a.device, s);
  else
    e = a.head_dim == 128 ? svx::launch_cross<__half, 128>(p, v.many, a.device, s) : svx::launch_cross<__half, 64>(p, v.many, a.device, s);
  if (e != cudaSuccess) return paged_fail(SVX_ERR_CUDA, "cross attention launch failed: %s", cudaGetErrorString(e));
  return SVX_OK;
}
