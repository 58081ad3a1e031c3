// Attention of one new token per request over a paged cache: the entry point and its join's sizes (the kernels and the reasons
// for their shape: svx_attend.cuh).
#include "svx_attend.cuh"

namespace svx {
namespace {

constexpr int64_t kMaxGridY = 65535;
svx_status sizes(const svx_pages* c, int32_t n_req, int32_t n_q, int64_t max_len, bool weights, Sizes* z) {
  if (n_q < c->n_kv_heads || n_q % c->n_kv_heads || n_q > 4096)
    return paged_fail(SVX_ERR_INVALID_ARG, "n_q_heads must be a positive multiple of n_kv_heads, at most 4096");
  const int64_t cap = static_cast<int64_t>(c->page_size) * c->max_pages;
  if (max_len < 0 || max_len > cap) return paged_fail(SVX_ERR_INVALID_ARG, "max_len must be in [0, max_pages * page_size]");
  if (max_len == 0) max_len = cap;
  const int sms = sm_count(c->device);
  if (sms <= 0) return paged_fail(SVX_ERR_CUDA, "cannot read the SM count");
  const int group = n_q / c->n_kv_heads;
  const int ct = kChunkBytes / (2 * c->head_dim);
  z->max_len = static_cast<int32_t>(max_len);
  z->blocks = (group + kRowsMax - 1) / kRowsMax;
  const int64_t chunks = static_cast<int64_t>(n_req) * c->n_kv_heads * z->blocks * ((max_len + ct - 1) / ct);
  if (weights && max_len > kMaxGridY * kWeightSlots)
    return paged_fail(SVX_ERR_UNSUPPORTED, "max_len must be at most %lld with weights",
                      static_cast<long long>(kMaxGridY * kWeightSlots));
  if (chunks > 0x7fffffff)
    return paged_fail(SVX_ERR_UNSUPPORTED, "n_req * heads * max_len is too large (%lld chunks of %d slots, at most 2^31 - 1)",
                      static_cast<long long>(chunks), ct);
  // Whole items to the CTAs where they are few and short: the longest takes a CTA kWholeItem / 8 chunks a warp, and the join's
  // launch and wait go.  Split and whole: one KV head of 64, 512 slots, 6.2 and 5.9 us; 8 KV heads of 128, 8 requests of 1 to 512
  // slots 9.4 and 8.7, 8 of 256 slots 6.9 and 6.7; 2 of 1024 slots (64 chunks, and so split) 8.0 and 11.7.  At the limit itself, 8 of
  // 512 slots, all as long as max_len, 8.3 and 8.5: the host knows the bound only, and ragged lengths below it gain more.
  const int64_t per_item = (max_len + ct - 1) / ct;
  z->whole = !weights && per_item <= kWholeItem && chunks <= sms * per_item;
  z->score_stride = (max_len + ct - 1) / ct * ct;
  size_pieces(z, chunks, c->head_dim, sms);
  z->row_ml = z->total;
  z->scores = z->row_ml + (weights ? up256(static_cast<size_t>(n_req) * n_q * 8) : 0);
  z->total = z->scores + (weights ? up256(static_cast<size_t>(n_req) * n_q * z->score_stride * 4) : 0);
  return SVX_OK;
}


template <typename T, int D>
cudaError_t launch_all(const AttendParams& p, int device, cudaStream_t s) {
  const bool wide = p.group > 8, scores = p.scores != nullptr;
  const cudaError_t e =
      wide ? (scores ? launch_attend<T, kPaged, D, true, true>(p, device, s) : launch_attend<T, kPaged, D, true, false>(p, device, s))
           : (scores ? launch_attend<T, kPaged, D, false, true>(p, device, s) : launch_attend<T, kPaged, D, false, false>(p, device, s));
  if (e != cudaSuccess || p.whole) return e;
  const int slots = scores ? (p.max_len + kWeightSlots - 1) / kWeightSlots : 1;
  const dim3 grid(p.pages.n_req * p.pages.n_kv_heads, std::max(p.blocks, slots));
  return scores ? launch_pdl(join_kernel<T, kPaged, D, true>, grid, dim3(kWarps * 32), 0, s, p)
                : launch_pdl(join_kernel<T, kPaged, D, false>, grid, dim3(kWarps * 32), 0, s, p);
}

}  // namespace
}  // namespace svx

extern "C" svx_status svx_paged_decode_workspace(const svx_pages* cache, int32_t n_req, int32_t n_q_heads,
                                                 int64_t max_len, int32_t weights, int64_t* bytes) {
  if (!bytes) return svx::paged_fail(SVX_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = 0;
  svx::PageView v;
  svx_status st = svx::paged_view(cache, n_req, &v);
  if (st != SVX_OK) return st;
  svx::Sizes z = {};
  st = svx::sizes(cache, n_req, n_q_heads, max_len, weights != 0, &z);
  if (st != SVX_OK) return st;
  *bytes = static_cast<int64_t>(z.total);
  return SVX_OK;
}

extern "C" svx_status svx_paged_decode(const svx_pages* cache, int32_t n_req, int32_t n_q_heads, const void* q,
                                       const int32_t* len, int64_t max_len, float scale, void* o, float* lse,
                                       const float* acc_in, float* acc_out, void* workspace, int64_t workspace_bytes,
                                       void* stream) {
  using svx::paged_fail;
  svx::AttendParams p = {};
  svx_status st = svx::paged_view(cache, n_req, &p.pages);
  if (st != SVX_OK) return st;
  if ((acc_in == nullptr) != (acc_out == nullptr))
    return paged_fail(SVX_ERR_INVALID_ARG, "give both acc_in and acc_out, or neither");
  if (!q || !o || !lse || !len || !svx::is_aligned(q, 16) || !svx::is_aligned(o, 16))
    return paged_fail(SVX_ERR_INVALID_ARG, "q, len, o and lse must be device pointers, q and o 16-byte aligned");
  if (!svx::words_aligned({len, lse, acc_in, acc_out}))
    return paged_fail(SVX_ERR_INVALID_ARG, "len, lse and acc must be 4-byte aligned");
  // (scores are held in log2 units: the scale times log2 e has to be finite in fp32)
  if (!svx::log2_scale(scale, cache->head_dim, &p.scale))
    return paged_fail(SVX_ERR_INVALID_ARG, "scale must be positive and below 2^128 ln 2, or 0");
  const size_t n_rows = static_cast<size_t>(n_req) * std::max(n_q_heads, 0), per_req = static_cast<size_t>(n_req) * 4;
  const size_t row = static_cast<size_t>(cache->head_dim) * 2, acc = per_req * p.pages.n_kv_heads * p.pages.cap;
  const svx::Span q_span = {q, n_rows * row}, o_span = {o, n_rows * row}, lse_span = {lse, n_rows * 4}, out_span = {acc_out, acc},
                  in_span = {acc_in == acc_out ? nullptr : acc_in, acc}, len_span = {len, per_req},
                  table_span = {cache->table, per_req * cache->max_pages};
  // (a strided pool takes what lies between its rows along)
  const size_t pool = static_cast<size_t>(p.pages.extent) * 2;
  const svx::Span k_span = {cache->k, pool}, v_span = {cache->v, pool};
  if (svx::any_overlap({o_span, lse_span, out_span, {cache->status, 4}}, {q_span, len_span, table_span, in_span, k_span, v_span}))
    return paged_fail(SVX_ERR_INVALID_ARG, "an output overlaps an input or another output (acc_out may be acc_in)");
  svx::Sizes z = {};
  st = svx::sizes(cache, n_req, n_q_heads, max_len, acc_in != nullptr, &z);
  if (st != SVX_OK) return st;
  if (!workspace || !svx::is_aligned(workspace, 256) || workspace_bytes < static_cast<int64_t>(z.total))
    return paged_fail(SVX_ERR_INVALID_ARG, "workspace must be 256-byte aligned, of at least %zu bytes", z.total);
  if (svx::any_overlap({{workspace, z.total}}, {q_span, o_span, lse_span, in_span, out_span, len_span, table_span, k_span, v_span, {cache->status, 4}}))
    return paged_fail(SVX_ERR_INVALID_ARG, "the workspace overlaps another buffer");
  svx::PagedDevice dev(cache->device);
  if (!dev.ok) return paged_fail(SVX_ERR_CUDA, "cannot use device %d", cache->device);
  const void* ptrs[] = {cache->k, cache->v, cache->table, cache->status, q, len, o, lse, acc_in, acc_out, workspace};
  for (const void* x : ptrs)
    if (x && !(cache->flags & SVX_POINTERS_CHECKED) && !svx::on_device(x, cache->device))
      return paged_fail(SVX_ERR_INVALID_ARG, "a pointer is not memory of device %d", cache->device);

  p.pages.extent = svx::clipped(svx::kClipPool, p.pages.extent);
  char* ws = static_cast<char*>(workspace);
  p.q = q;
  p.len = len;
  p.o = o;
  p.lse = lse;
  p.acc_in = acc_in;
  p.acc_out = acc_out;
  svx::place_pieces(p, z, ws);
  p.row_ml = acc_in ? reinterpret_cast<float2*>(ws + z.row_ml) : nullptr;
  p.scores = acc_in ? reinterpret_cast<float*>(ws + z.scores) : nullptr;
  p.score_stride = z.score_stride;
  p.n_q = n_q_heads;
  p.group = n_q_heads / cache->n_kv_heads;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cache->dtype == SVX_BF16)
    e = cache->head_dim == 128 ? svx::launch_all<__nv_bfloat16, 128>(p, cache->device, s)
                               : svx::launch_all<__nv_bfloat16, 64>(p, cache->device, s);
  else
    e = cache->head_dim == 128 ? svx::launch_all<__half, 128>(p, cache->device, s)
                               : svx::launch_all<__half, 64>(p, cache->device, s);
  if (e != cudaSuccess) return paged_fail(SVX_ERR_CUDA, "decode kernel launch failed: %s", cudaGetErrorString(e));
  return SVX_OK;
}
