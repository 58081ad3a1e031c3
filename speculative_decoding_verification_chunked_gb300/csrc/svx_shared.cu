// Attention of one new token per request over a paged cache, for requests that share prefixes: a prefix's K and V are read once
// for all its requests, whose tokens' query heads are the rows of one product with them.
//
// With few rows to a prefix two kinds of sequences lie in one flat range of chunks (attend_kernel, svx_attend.cuh): the prefixes, with
// the rows of all their requests, and the requests' own slots.  With many rows the prefixes are rows_kernel's work (svx_rows.cuh) and
// attend_kernel beside it takes the requests' own slots.  Every row then has two lots of states (m, l, O), which join_shared merges.
//
// Measured (32 heads, 8 KV heads, d = 128, bf16): 16 samples of a 32768-slot prompt with up to 512 slots of their own 44 us (the bytes 22);
// 256 requests behind 65536 slots, read once, 243 us (the products 144; the requests' own slots are brought in by SMs of their
// own meanwhile).  Four branches of 2048 slots, 4 heads of d = 64: 11.7 us, two launches and their trips to memory.
#include "svx_rows.cuh"

namespace svx {
namespace {

constexpr int kBatch = 64;  // pieces of a row whose factors are worked out at a time

// A CTA takes every gridDim.x-th of the requests' KV heads, block of 16 query heads y, and of the dimensions part z of gridDim.z.
// APART: the prefixes were rows_kernel's work.
template <typename T, int D, bool APART>
__global__ void __launch_bounds__(kWarps * 32, 4) join_shared(const __grid_constant__ AttendParams P) {
  constexpr int CT = kChunkBytes / (2 * D);
  // Where the pieces of a row's lot lie: one is a finished state; else piece c is in slot 0 of CTA first + c, or (c = 0) slot 1.
  struct Lot {
    int32_t first, pieces, row;  // row: in the pieces' blocks, or of the finished states
  };
  __shared__ Plan<kShared> plan;
  __shared__ float s_f[kBatch * kRowsMax];
  __shared__ float2 s_ml[kRowsMax];
  __shared__ Lot s_lots[kWarps][2][kRowsMax];  // of the next heads, a warp's work each
  __shared__ float4 s_o[kWarps * 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // (the lengths were there before the attention kernel began, which had waited for whoever wrote them)
  const int T_all = build_plan<kShared, CT>(P, plan, false, APART);
  const Split split(P, T_all);
  const RowSplit row_split(P, APART ? plan.row_tiles : 0);
  const int blk = blockIdx.y, rows = min(P.group - blk * kRowsMax, kRowsMax);
  // the outputs over the threads: several share one where there are more of them than outputs
  const int quads = D / 4 / gridDim.z, outs = rows * quads, share = max(kWarps * 32 / outs, 1);
  const int part = share > 1 ? tid / outs : 0;
  const Lot(*s_lot)[kRowsMax] = s_lots[0];
  auto ml_at = [&](int r, int c) {
    const int lot = c < s_lot[0][r].pieces ? 0 : 1;
    if (lot) c -= s_lot[0][r].pieces;
    const Lot x = s_lot[lot][r];
    if (x.pieces == 1) return __ldcg(P.state_ml + x.row);
    const int slot = (x.first + c) * 2 + (c == 0 ? 1 : 0);
    return __ldcg(APART && lot == 0 ? P.rows_ml + slot * P.item_rows + x.row : P.part_ml + slot * kRowsMax + x.row);
  };
  auto o_at = [&](int r, int c, int d4) {
    const int lot = c < s_lot[0][r].pieces ? 0 : 1;
    if (lot) c -= s_lot[0][r].pieces;
    const Lot x = s_lot[lot][r];
    const int slot = (x.first + c) * 2 + (c == 0 ? 1 : 0);
    if (APART && lot == 0 && x.pieces > 1)
      return __ldcg(P.rows_o + (static_cast<int64_t>(slot) * (D / 4) + d4 / 4) * P.item_rows + x.row);
    const float* at = x.pieces == 1 ? P.state_o + static_cast<int64_t>(x.row) * D : P.part_o + static_cast<int64_t>(slot * kRowsMax + x.row) * D;
    return __ldcg(reinterpret_cast<const float4*>(at + d4));
  };
  auto add = [](float4& o, const float4& x, float f) {
    o.x = fmaf(x.x, f, o.x);
    o.y = fmaf(x.y, f, o.y);
    o.z = fmaf(x.z, f, o.z);
    o.w = fmaf(x.w, f, o.w);
  };
  const int heads = P.pages.n_req * P.pages.n_kv_heads;
  bool waited = false;
  for (int bh0 = blockIdx.x; bh0 < heads; bh0 += kWarps * gridDim.x) {
    if (waited) __syncthreads();  // (the last ones are done with)
    {
      const int bh = bh0 + warp * gridDim.x, b = bh / P.pages.n_kv_heads, h = bh - b * P.pages.n_kv_heads;
      const int r = lane % kRowsMax, lot = lane / kRowsMax;  // 0: the prefix, 1: the request's own
      int prefix = 0;  // the first that ends behind the request
      for (int i = 0; i < P.n_prefix; i += 32)
        prefix += __popc(__ballot_sync(0xffffffffu, i + lane < P.n_prefix && plan.req0[i + lane + 1] <= b));
      Lot x{0, 0, 0};
      int seq = kMaxReq + b, block = blk, blocks = P.blocks;
      x.row = r;
      bool any = r < rows && bh < heads;
      if (lot == 0) {
        any = any && prefix < P.n_prefix && plan.req0[prefix] <= b;
        if (any) {
          const int R = (b - plan.req0[prefix]) * P.group + blk * kRowsMax + r;
          seq = prefix;
          const int per = APART ? P.item_rows : kRowsMax;
          block = R / per;
          blocks = (seq_rows(P, plan, prefix) + per - 1) / per;
          x.row = R % per;
        }
      }
      const int n = any ? plan.n[seq] : 0;
      if (n > 0) {
        const int first = plan.first[seq] + (h * blocks + block) * n;
        const bool far = APART && lot == 0;
        x.first = far ? row_split.of(first) : split.of(first);
        x.pieces = (far ? row_split.of(first + n - 1) : split.of(first + n - 1)) - x.first + 1;
        if (x.pieces == 1) x.row = (lot * P.pages.n_req + b) * P.n_q + h * P.group + blk * kRowsMax + r;
      }
      s_lots[warp][lot][r] = x;
    }
    __syncthreads();
    if (!waited) {
      grid_dependency_wait();
      allow_dependents();
      waited = true;
    }
    for (int nth = 0; nth < kWarps && bh0 + nth * gridDim.x < heads; ++nth) {
      const int bh = bh0 + nth * gridDim.x, b = bh / P.pages.n_kv_heads, h = bh - b * P.pages.n_kv_heads;
      s_lot = s_lots[nth];
      if (nth > 0) __syncthreads();  // (the last one's states and factors are done with)
      int most = 0;  // pieces of any row
      for (int r = 0; r < rows; ++r) most = max(most, s_lot[0][r].pieces + s_lot[1][r].pieces);
      for (int i0 = 0; i0 < outs; i0 += kWarps * 32) {  // (once, unless there are more outputs than threads)
        const int i = share > 1 ? tid - part * outs : i0 + tid;
        // (rows_kernel's pieces have a row's neighbours beside it, the others its dimensions)
        const int r = APART ? i % rows : i / quads, d4 = ((APART ? i / rows : i - r * quads) + blockIdx.z * quads) * 4;
        const bool mine = i < outs && part < share;
        const int pieces = mine ? s_lot[0][r].pieces + s_lot[1][r].pieces : 0;
        // this thread's first pieces are fetched along with the states
        constexpr int kAhead = 4;
        float4 ahead[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (part + u * share < pieces) ahead[u] = o_at(r, part + u * share, d4);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c0 = 0; c0 < max(most, 1); c0 += kBatch) {
          if (c0 > 0 || i0 > 0) __syncthreads();  // (the last batch's factors have been used)
          if (i0 == 0 || most > kBatch)
            for (int q = warp; q < rows; q += kWarps) {
              const int all = s_lot[0][q].pieces + s_lot[1][q].pieces, end = min(all, c0 + kBatch);
              float2 ml = c0 + lane < end ? ml_at(q, c0 + lane) : make_float2(kNegInf, 0.f);
              float M = ml.x, L = 0.f;
              if (c0 == 0 && i0 == 0) {
                for (int c = lane + 32; c < all; c += 32) M = fmaxf(M, ml_at(q, c).x);
#pragma unroll
                for (int k = 16; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
              } else {
                M = s_ml[q].x;
                L = s_ml[q].y;
              }
              const float less = M == kNegInf ? 0.f : -M;
              float sum = 0.f;
              for (int c = c0 + lane; c < end; c += 32) {
                if (c != c0 + lane) ml = ml_at(q, c);
                const float f = ex2(ml.x + less);
                s_f[(c - c0) * kRowsMax + q] = f;
                sum = fmaf(ml.y, f, sum);
              }
#pragma unroll
              for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
              if (lane == 0 && i0 == 0) s_ml[q] = make_float2(M, L + sum);
            }
          __syncthreads();
          const int end = min(pieces, c0 + kBatch);
          int c = c0 + part;
          if (c0 == 0) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u, c += share)
              if (c < end) add(o, ahead[u], s_f[c * kRowsMax + r]);
          }
#pragma unroll 4
          for (; c < end; c += share) add(o, o_at(r, c, d4), s_f[(c - c0) * kRowsMax + r]);
        }
        if (share > 1) {
          s_o[tid] = o;
          __syncthreads();
          if (part == 0)
            for (int p = 1; p < share; ++p) {
              const float4 x = s_o[p * outs + i];
              o = make_float4(o.x + x.x, o.y + x.y, o.z + x.z, o.w + x.w);
            }
        }
        if (mine && part == 0) write_row<T>(P, place<kShared, D>(P, plan, kMaxReq + b, h, blk, r), d4, s_ml[r].x, s_ml[r].y, o);
      }
    }
  }
}

struct SharedSizes {
  Sizes z;
  RowSizes rz;
  bool many;
  int32_t max_prefix;
};

// What can be told without the device.
svx_status shared_check(const svx_pages* c, int32_t n_q, const svx_prefixes* f, int64_t max_len) {
  if (n_q < c->n_kv_heads || n_q % c->n_kv_heads || n_q > 4096)
    return paged_fail(SVX_ERR_INVALID_ARG, "n_q_heads must be a positive multiple of n_kv_heads, at most 4096");
  if (!f) return paged_fail(SVX_ERR_INVALID_ARG, "prefixes is NULL");
  if (f->n_prefix < 1 || f->n_prefix > kMaxReq) return paged_fail(SVX_ERR_INVALID_ARG, "n_prefix must be in [1, %d]", kMaxReq);
  const int64_t cap = static_cast<int64_t>(c->page_size) * c->max_pages, room = static_cast<int64_t>(c->page_size) * f->max_pages;
  if (f->max_pages < 1 || room > 0x7fffffffLL)
    return paged_fail(SVX_ERR_INVALID_ARG, "the prefixes' max_pages must be positive, its product with page_size below 2^31");
  if (max_len < 0 || max_len > cap) return paged_fail(SVX_ERR_INVALID_ARG, "max_len must be in [0, max_pages * page_size]");
  if (f->max_len < 0 || f->max_len > room)
    return paged_fail(SVX_ERR_INVALID_ARG, "the prefixes' max_len must be in [0, their max_pages * page_size]");
  return SVX_OK;
}

// (after shared_check)
svx_status shared_sizes(const svx_pages* c, int32_t n_req, int32_t n_q, const svx_prefixes* f, int64_t max_len, SharedSizes* out) {
  if (max_len == 0) max_len = static_cast<int64_t>(c->page_size) * c->max_pages;
  const int64_t max_prefix = f->max_len ? f->max_len : static_cast<int64_t>(c->page_size) * f->max_pages;
  const int sms = sm_count(c->device);
  if (sms <= 0) return paged_fail(SVX_ERR_CUDA, "cannot read the SM count");
  const int group = n_q / c->n_kv_heads, ct = kChunkBytes / (2 * c->head_dim);
  Sizes& z = out->z;
  z.max_len = static_cast<int32_t>(max_len);
  out->max_prefix = static_cast<int32_t>(max_prefix);
  z.blocks = (group + kRowsMax - 1) / kRowsMax;
  // (a prefix's last block of rows may not be full)
  const int64_t all_rows = static_cast<int64_t>(n_req) * group, used = std::min(f->n_prefix, n_req);
  const int64_t own = static_cast<int64_t>(n_req) * c->n_kv_heads * z.blocks * ((max_len + ct - 1) / ct);
  const int64_t far = c->n_kv_heads * (all_rows / kRowsMax + used) * ((max_prefix + ct - 1) / ct);
  // By the rows to a prefix, on average (32 heads, 8 KV heads, one prefix of 16384 slots: 16 rows 24.3 us by attend_kernel alone, 24.9 with
  // rows_kernel; 32 rows 34 and 26; 64 rows and 32768 slots 87 and 48; eight prefixes of 4096 slots with 8 rows each 38 and 43).  `first` is
  // on the device, so prefixes without requests count too (256 requests of one prompt in a call for 1 prefix 230 us, for 16 440, for 64,
  // where attend_kernel takes them, 2230).
  out->many = all_rows > static_cast<int64_t>(kRowsMax) * f->n_prefix;
  if (own + far > 0x7fffffff)
    return paged_fail(SVX_ERR_UNSUPPORTED, "heads times lengths are too large (%lld chunks of %d slots, at most 2^31 - 1)",
                      static_cast<long long>(own + far), ct);
  const int64_t chunks = own + (out->many ? 0 : far);
  // With many rows the SMs are shared out over the two kernels by their work, so that they end together: a CTA of attend_kernel brings in
  // some 45 GB/s of short sequences, and begins and ends an item in 0.18 us (84 requests of one slot each, 8 KV heads: 43 us without that
  // term, 30); a tile of rows_kernel takes 1.4 us with two row tiles, 1.0 with one.  By the bounds known here: where lengths are
  // far below them, the kernel that has the work has few CTAs (256 requests of up to 512 slots behind 65536: bounds of 512 own slots 230
  // us, of 2048 360, of 8192 1350, of 65536 5300; 16 of them behind 32768: 45, 59, 119, 544; prefix bounds 4 times too wide 670 and 61).
  int own_ctas = sms;
  if (out->many) {
    // (of a prefix, on average; 8 of 16 requests' 64 rows, 4096 slots, d = 64: in items of 128 rows 39 us, of 256 44; 16 such of 2048 slots,
    // d = 128: 64 and 60)
    const int item_rows = item_rows_for((all_rows + used - 1) / used);
    const int64_t items = c->n_kv_heads * (all_rows / item_rows + used), per = (max_prefix + kKeyTile - 1) / kKeyTile;
    const double own_us = static_cast<double>(n_req) * c->n_kv_heads * max_len * c->head_dim * 4 / 45e3 + 0.18 * n_req * c->n_kv_heads * z.blocks;
    const double far_us = static_cast<double>(items) * per * (item_rows > kRowTile ? 1.4 : 1.0);
    own_ctas = std::min(std::max(static_cast<int>(sms * own_us / (own_us + far_us) + 0.5), 8), sms - 4);
    // Where a prefix's rows are several items, as many CTAs as make the items' halves whole: then the CTAs of a KV head's items go
    // through the same keys at a time, and find them in L2 (256 requests behind 65536 slots, 32 such items: 107 CTAs 251 us, 112 233).
    const int64_t blocks = (all_rows + used * item_rows - 1) / (used * item_rows), half = c->n_kv_heads * used * blocks / 2;
    if (blocks > 1) {
      const int64_t near = (sms - own_ctas + half / 2) / half * half;
      if (near >= 4 && near <= sms - 4 && std::abs(near - (sms - own_ctas)) * 8 <= sms) own_ctas = sms - static_cast<int>(near);
    }
    size_rows(&out->rz, items, per, item_rows, c->head_dim, sms - own_ctas, 0, false);
  }
  size_pieces(&z, chunks, c->head_dim, own_ctas);
  const size_t rows = static_cast<size_t>(2) * n_req * n_q;
  z.state_o = z.total;
  z.state_ml = z.state_o + up256(rows * c->head_dim * 4);
  z.total = z.state_ml + up256(rows * 8);
  if (out->many) {
    out->rz.rows_o += z.total;
    out->rz.rows_ml += z.total;
    out->rz.sums += z.total;
    out->rz.refs += z.total;
    z.total += out->rz.total;
  }
  return SVX_OK;
}

template <typename T, int D>
cudaError_t launch_shared(const AttendParams& p, int device, cudaStream_t s) {
  const int sms = sm_count(device);
  // the join: CTAs that are resident at a time (4 an SM); where the heads are fewer, several to a head, on parts of its dimensions
  const int heads = p.pages.n_req * p.pages.n_kv_heads, ctas = heads * p.blocks;
  const dim3 grid(std::min(heads, std::max(4 * sms / p.blocks, 1)), p.blocks, ctas * 4 <= 4 * sms ? 4 : ctas * 2 <= 4 * sms ? 2 : 1);
  cudaError_t e;
  if (p.prefix_apart) {
    e = p.group > 8 ? launch_attend<T, kShared, D, true, false>(p, device, s) : launch_attend<T, kShared, D, false, false>(p, device, s);
    if (e != cudaSuccess) return e;
    e = launch_rows<T, kShared, D>(p, device, s);
    return e != cudaSuccess ? e : launch_pdl(join_shared<T, D, true>, grid, dim3(kWarps * 32), 0, s, p);
  }
  // (rows of a prefix: those of all its requests)
  const bool wide = static_cast<int64_t>(p.group) * p.pages.n_req > 8;
  e = wide ? launch_attend<T, kShared, D, true, false>(p, device, s) : launch_attend<T, kShared, D, false, false>(p, device, s);
  return e != cudaSuccess ? e : launch_pdl(join_shared<T, D, false>, grid, dim3(kWarps * 32), 0, s, p);
}

}  // namespace
}  // namespace svx

extern "C" svx_status svx_paged_decode_shared_workspace(const svx_pages* cache, int32_t n_req, int32_t n_q_heads,
                                                        const svx_prefixes* prefixes, int64_t max_len, int64_t* bytes) {
  if (!bytes) return svx::paged_fail(SVX_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = 0;
  svx::PageView v;
  svx_status st = svx::paged_view(cache, n_req, &v);
  if (st != SVX_OK) return st;
  svx::SharedSizes z = {};
  st = svx::shared_check(cache, n_q_heads, prefixes, max_len);
  if (st == SVX_OK) st = svx::shared_sizes(cache, n_req, n_q_heads, prefixes, max_len, &z);
  if (st == SVX_OK) *bytes = static_cast<int64_t>(z.z.total);
  return st;
}

extern "C" svx_status svx_paged_decode_shared(const svx_pages* cache, int32_t n_req, int32_t n_q_heads, const void* q,
                                              const svx_prefixes* prefixes, const int32_t* len, int64_t max_len, float scale,
                                              void* o, float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
  using svx::paged_fail;
  svx::AttendParams p = {};
  svx_status st = svx::paged_view(cache, n_req, &p.pages);
  if (st != SVX_OK) return st;
  st = svx::shared_check(cache, n_q_heads, prefixes, max_len);
  if (st != SVX_OK) return st;
  const svx_prefixes& f = *prefixes;
  if (!q || !o || !lse || !len || !svx::is_aligned(q, 16) || !svx::is_aligned(o, 16))
    return paged_fail(SVX_ERR_INVALID_ARG, "q, len, o and lse must be device pointers, q and o 16-byte aligned");
  if (!f.table || !f.len || !f.first || !svx::words_aligned({f.table, f.len, f.first, len, lse}))
    return paged_fail(SVX_ERR_INVALID_ARG, "the prefixes' table, len and first, and len and lse, must be 4-byte aligned device pointers");
  if (!svx::log2_scale(scale, cache->head_dim, &p.scale))
    return paged_fail(SVX_ERR_INVALID_ARG, "scale must be positive and below 2^128 ln 2, or 0");
  const size_t n_rows = static_cast<size_t>(n_req) * n_q_heads, row = static_cast<size_t>(cache->head_dim) * 2;
  const size_t per_req = static_cast<size_t>(n_req) * 4, per_prefix = static_cast<size_t>(f.n_prefix) * 4;
  const size_t pool = static_cast<size_t>(p.pages.extent) * 2;
  const svx::Span q_span = {q, n_rows * row}, o_span = {o, n_rows * row}, lse_span = {lse, n_rows * 4}, len_span = {len, per_req},
                  table_span = {cache->table, per_req * cache->max_pages}, far_table = {f.table, per_prefix * f.max_pages},
                  far_len = {f.len, per_prefix}, first_span = {f.first, per_prefix + 4}, k_span = {cache->k, pool},
                  v_span = {cache->v, pool}, status = {cache->status, 4};
  if (svx::any_overlap({o_span, lse_span, status}, {q_span, len_span, table_span, far_table, far_len, first_span, k_span, v_span}))
    return paged_fail(SVX_ERR_INVALID_ARG, "an output overlaps an input or another output");
  svx::SharedSizes z = {};
  st = svx::shared_sizes(cache, n_req, n_q_heads, prefixes, max_len, &z);
  if (st != SVX_OK) return st;
  if (!workspace || !svx::is_aligned(workspace, 256) || workspace_bytes < static_cast<int64_t>(z.z.total))
    return paged_fail(SVX_ERR_INVALID_ARG, "workspace must be 256-byte aligned, of at least %zu bytes", z.z.total);
  if (svx::any_overlap({{workspace, z.z.total}},
                       {q_span, o_span, lse_span, len_span, table_span, far_table, far_len, first_span, k_span, v_span, status}))
    return paged_fail(SVX_ERR_INVALID_ARG, "the workspace overlaps another buffer");
  svx::PagedDevice dev(cache->device);
  if (!dev.ok) return paged_fail(SVX_ERR_CUDA, "cannot use device %d", cache->device);
  const void* ptrs[] = {cache->k, cache->v, cache->table, cache->status, q, f.table, f.len, f.first, len, o, lse, workspace};
  for (const void* x : ptrs)
    if (!(cache->flags & SVX_POINTERS_CHECKED) && !svx::on_device(x, cache->device))
      return paged_fail(SVX_ERR_INVALID_ARG, "a pointer is not memory of device %d", cache->device);

  p.pages.extent = svx::clipped(svx::kClipPool, p.pages.extent);
  char* ws = static_cast<char*>(workspace);
  svx::place_pieces(p, z.z, ws);
  p.state_o = reinterpret_cast<float*>(ws + z.z.state_o);
  p.state_ml = reinterpret_cast<float2*>(ws + z.z.state_ml);
  p.prefix_apart = z.many;
  p.q = q;
  p.len = len;
  p.o = o;
  p.lse = lse;
  p.n_q = n_q_heads;
  p.group = n_q_heads / cache->n_kv_heads;
  if (z.many) svx::place_rows(p, z.rz, ws);
  p.prefix_table = f.table;
  p.prefix_len = f.len;
  p.first = f.first;
  p.n_prefix = f.n_prefix;
  p.prefix_max_pages = f.max_pages;
  p.max_prefix = z.max_prefix;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cache->dtype == SVX_BF16)
    e = cache->head_dim == 128 ? svx::launch_shared<__nv_bfloat16, 128>(p, cache->device, s)
                               : svx::launch_shared<__nv_bfloat16, 64>(p, cache->device, s);
  else
    e = cache->head_dim == 128 ? svx::launch_shared<__half, 128>(p, cache->device, s)
                               : svx::launch_shared<__half, 64>(p, cache->device, s);
  if (e != cudaSuccess) return paged_fail(SVX_ERR_CUDA, "shared-prefix kernel launch failed: %s", cudaGetErrorString(e));
  return SVX_OK;
}
