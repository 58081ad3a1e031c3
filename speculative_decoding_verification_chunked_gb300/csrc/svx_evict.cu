// Eviction from a paged cache by accumulated attention weight.
//
// Per (request, KV head) row of L slots, n = min(L, budget) are kept: those whose position is protected (sinks and the
// most recent), then the largest weights, equal ones by the lower slot.  The kept slots >= n (spares) fill the evicted
// ones < n (holes), both in order of slot.  Sources and destinations are disjoint, so rows move inside the pages in any
// order and without a staging copy, and only as many as there are holes: after a step that went one page over its
// budget that is at most a page, where a compaction in order would move nearly every row.
//
// select_kernel: a cluster of CTAs per row holds the row's slots in registers as 32-bit keys whose unsigned order is
// the order of preference (weights >= 0 or not, NaN as -inf, protected slots above all).  The n-th largest key is found
// by bisection over the key's bits: a count per step, no histogram, so equal weights cost nothing extra and nothing
// depends on the order of atomics.  Ties, holes and spares are numbered by ballots and one scan over the warps each.
// move_kernel: a warp copies a row's K and V (512 bytes at d = 128) at a time, four rows in flight.
// Floor: 8 bytes a slot read, 8 a kept slot written, 8 d bytes a moved slot.
#include <cooperative_groups.h>

#include <algorithm>

#include "svx_paged.h"

namespace cg = cooperative_groups;

namespace svx {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxKeys = 32;    // per thread
constexpr int kMaxCluster = 8;  // portable
static_assert(kThreads * kMaxKeys * kMaxCluster == SVX_EVICT_MAX_LEN, "the longest row a cluster holds");

struct EvictParams {
  PageView pages;
  const int32_t* len;
  const int32_t* next_pos;
  const float* acc_in;
  const int32_t* pos_in;
  float* acc_out;
  int32_t* pos_out;
  int32_t* len_out;
  int32_t* moves;   // [rows]: moved slots of each row
  int32_t* kept;    // [n_req]: new lengths
  int32_t* holes;   // [rows][most]
  int32_t* spares;  // [rows][most]
  int32_t max_len, budget, sink, recent;
  int32_t most;     // moves a row can need
  int32_t cluster;
};

// Unsigned order = float order; NaN as -inf, -0 as +0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (isnan(w)) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u ^ ((u & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}

struct Counts {
  int32_t warp[2][kWarps];
  int32_t peer[2][kMaxCluster];
};

// Sum over the row's cluster of one value per warp (the same in all lanes); `turn` alternates between calls, so
// that one barrier (two in a cluster) separates a call's writes from the last reads of the same buffer.
__device__ __forceinline__ int cluster_sum(int v, Counts& s, int turn, int n_cta, int rank) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) s.warp[turn][warp] = v;
  __syncthreads();
  int sum = __reduce_add_sync(0xffffffffu, s.warp[turn][lane]);
  if (n_cta > 1) {
    cg::cluster_group cl = cg::this_cluster();
    if (threadIdx.x < n_cta) *cl.map_shared_rank(&s.peer[turn][rank], threadIdx.x) = sum;
    cl.sync();
    sum = 0;
    for (int i = 0; i < n_cta; ++i) sum += s.peer[turn][i];
  }
  return sum;
}

// Sum of the values of the warps before this one, in the order (CTA of the cluster, warp); `total` gets all.
__device__ __forceinline__ int cluster_scan(int v, Counts& s, int turn, int n_cta, int rank, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) s.warp[turn][warp] = v;
  __syncthreads();
  const int x = s.warp[turn][lane];
  int before = __reduce_add_sync(0xffffffffu, lane < warp ? x : 0);
  int sum = __reduce_add_sync(0xffffffffu, x);
  if (n_cta > 1) {
    cg::cluster_group cl = cg::this_cluster();
    if (threadIdx.x < n_cta) *cl.map_shared_rank(&s.peer[turn][rank], threadIdx.x) = sum;
    cl.sync();
    sum = 0;
    for (int i = 0; i < n_cta; ++i) {
      if (i < rank) before += s.peer[turn][i];
      sum += s.peer[turn][i];
    }
  }
  *total = sum;
  return before;
}

template <int KEYS>
__global__ void __launch_bounds__(kThreads, 1) select_kernel(const __grid_constant__ EvictParams P) {
  __shared__ Counts s;
  grid_dependency_wait();
  allow_dependents();
  const int n_cta = P.cluster, rank = static_cast<int>(blockIdx.x) % n_cta;
  const int row = static_cast<int>(blockIdx.x) / n_cta;
  const int b = row / P.pages.n_kv_heads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int raw = P.len[b];
  const int L = min(max(raw, 0), P.max_len);
  const int n = min(L, P.budget);
  if (threadIdx.x == 0 && rank == 0 && row == b * P.pages.n_kv_heads) {
    if (raw != L) atomicOr(P.pages.status, kErrInput);
    P.kept[b] = n;
  }
  const int64_t meta = static_cast<int64_t>(row) * P.pages.cap;
  const int first = (rank * kWarps + warp) * (32 * KEYS) + lane;  // this lane's slots: first + 32 i
  uint32_t key[KEYS];
  const int64_t recent_from = static_cast<int64_t>(P.next_pos[b]) - P.recent;
#pragma unroll
  for (int i = 0; i < KEYS; ++i) {
    const int t = first + 32 * i;
    key[i] = 0;
    if (t < L) {
      const int32_t pos = P.pos_in[meta + t];
      key[i] = pos < P.sink || pos >= recent_from ? 0xffffffffu : order_key(P.acc_in[meta + t]);
    }
  }
  // the n-th largest key: the largest `cut` with at least n keys >= cut
  int turn = 0;
  uint32_t cut = 0;
  int above = 0;  // keys > cut, if not exact
  bool exact = L <= P.budget;
  if (n_cta > 1) cg::this_cluster().sync();  // every CTA runs before another writes to its shared memory
  if (!exact) {
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t tryc = cut | (1u << bit);
      int c = 0;
#pragma unroll
      for (int i = 0; i < KEYS; ++i) c += key[i] >= tryc;
      c = cluster_sum(__reduce_add_sync(0xffffffffu, c), s, turn, n_cta, rank);
      turn ^= 1;
      if (c >= n) {
        cut = tryc;
        exact = c == n;
        if (exact) break;
      } else {
        above = c;
      }
    }
  } else {
    cut = 1;  // every slot's key
  }
  uint32_t keep = 0;  // bit i: slot first + 32 i is kept
  if (exact) {
#pragma unroll
    for (int i = 0; i < KEYS; ++i) keep |= static_cast<uint32_t>(key[i] >= cut) << i;
  } else {
    // after the last bit the trials that followed the last failing one all held, so that one was cut + 1 and
    // `above` counts the keys > cut (none failed: cut is the largest key, above 0)
    int mine = 0;
#pragma unroll
    for (int i = 0; i < KEYS; ++i) mine += __popc(__ballot_sync(0xffffffffu, key[i] == cut));
    int ties;
    int at = cluster_scan(mine, s, turn, n_cta, rank, &ties);
    turn ^= 1;
    const int need = n - above;
#pragma unroll
    for (int i = 0; i < KEYS; ++i) {
      const bool tie = key[i] == cut;
      const uint32_t m = __ballot_sync(0xffffffffu, tie);
      const int mine_at = at + __popc(m & ((1u << lane) - 1u));
      at += __popc(m);
      keep |= static_cast<uint32_t>(key[i] > cut || (tie && mine_at < need)) << i;
    }
  }
  // holes and spares, numbered in order of slot
  int nh = 0, ns = 0;
#pragma unroll
  for (int i = 0; i < KEYS; ++i) {
    const int t = first + 32 * i;
    const bool k = (keep >> i) & 1u;
    nh += __popc(__ballot_sync(0xffffffffu, t < n && !k));
    ns += __popc(__ballot_sync(0xffffffffu, t >= n && k));
  }
  int all_h, all_s;
  int ah = cluster_scan(nh, s, turn, n_cta, rank, &all_h);
  turn ^= 1;
  int as = cluster_scan(ns, s, turn, n_cta, rank, &all_s);
  turn ^= 1;
  if (threadIdx.x == 0 && rank == 0) P.moves[row] = min(min(all_h, all_s), P.most);
  int32_t* holes = P.holes + static_cast<int64_t>(row) * P.most;
  int32_t* spares = P.spares + static_cast<int64_t>(row) * P.most;
  const bool copy_acc = P.acc_out != P.acc_in, copy_pos = P.pos_out != P.pos_in;
  const uint32_t before = (1u << lane) - 1u;
#pragma unroll
  for (int i = 0; i < KEYS; ++i) {
    const int t = first + 32 * i;
    const bool k = (keep >> i) & 1u;
    const bool hole = t < n && !k, spare = t >= n && k;
    const uint32_t mh = __ballot_sync(0xffffffffu, hole), ms = __ballot_sync(0xffffffffu, spare);
    const int ih = ah + __popc(mh & before), is = as + __popc(ms & before);
    ah += __popc(mh);
    as += __popc(ms);
    if (hole && ih < P.most) holes[ih] = t;
    if (spare && is < P.most) spares[is] = t;
    if (t < n && k) {
      if (copy_acc) P.acc_out[meta + t] = P.acc_in[meta + t];
      if (copy_pos) P.pos_out[meta + t] = P.pos_in[meta + t];
    }
  }
  if (n_cta > 1) cg::this_cluster().sync();  // no CTA leaves while another may still write to its shared memory
}

constexpr int kMoveWarps = 8;
constexpr int kMoveBatch = 4;

template <int D>
__global__ void __launch_bounds__(kMoveWarps * 32) move_kernel(const __grid_constant__ EvictParams P) {
  using T = uint16_t;                    // rows move as bits, whatever the type
  constexpr int PIECES = D / 8;          // 16-byte pieces of a row
  constexpr int SIDE = 32 / (2 * PIECES);  // moves of a warp at a time: K on one half of the lanes, V on the other
  grid_dependency_wait();
  allow_dependents();
  const int row = blockIdx.y, b = row / P.pages.n_kv_heads, h = row - b * P.pages.n_kv_heads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) P.len_out[b] = P.kept[b];
  const int M = P.moves[row];
  const int32_t* holes = P.holes + static_cast<int64_t>(row) * P.most;
  const int32_t* spares = P.spares + static_cast<int64_t>(row) * P.most;
  const int64_t meta = static_cast<int64_t>(row) * P.pages.cap;
  const int32_t* table = P.pages.table + static_cast<int64_t>(b) * P.pages.max_pages;
  const bool is_v = lane >= 16;
  uint4* pool = static_cast<uint4*>(is_v ? P.pages.v : P.pages.k);
  const int piece = lane % PIECES, side = (lane % 16) / PIECES;
  const int step = gridDim.x * kMoveWarps * SIDE * kMoveBatch;
  for (int i0 = (blockIdx.x * kMoveWarps + warp) * SIDE * kMoveBatch; i0 < M; i0 += step) {
    int64_t to[kMoveBatch];
    uint4 v[kMoveBatch];
    int32_t hole[kMoveBatch], spare[kMoveBatch];
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u) {
      const int i = i0 + u * SIDE + side;
      hole[u] = spare[u] = -1;
      if (i < M) {
        hole[u] = holes[i];
        spare[u] = spares[i];
      }
    }
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u) {
      to[u] = -1;
      if (hole[u] < 0) continue;
      const uint32_t ps = P.pages.page_size;
      const uint32_t pt = static_cast<uint32_t>(hole[u]) / ps, pf = static_cast<uint32_t>(spare[u]) / ps;
      const int64_t ot = slot_offset(P.pages, table[pt], hole[u] - pt * ps);
      const int64_t of = slot_offset(P.pages, table[pf], spare[u] - pf * ps);
      if (ot < 0 || of < 0) {
        atomicOr(P.pages.status, kErrInput);
        continue;
      }
      const int64_t from = of + static_cast<int64_t>(h) * P.pages.head_stride;
      to[u] = ot + static_cast<int64_t>(h) * P.pages.head_stride;
      const T* base = reinterpret_cast<const T*>(pool);
      if (!in_bounds(base + from, D, base, P.pages.extent, P.pages.status, kSitePool) ||
          !in_bounds(base + to[u], D, base, P.pages.extent, P.pages.status, kSitePool)) {
        to[u] = -1;
        continue;
      }
      v[u] = pool[from / 8 + piece];
    }
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u)
      if (to[u] >= 0) pool[to[u] / 8 + piece] = v[u];
    if (piece == 0) {
#pragma unroll
      for (int u = 0; u < kMoveBatch; ++u)
        if (hole[u] >= 0) {
          if (is_v) P.pos_out[meta + hole[u]] = P.pos_in[meta + spare[u]];
          else P.acc_out[meta + hole[u]] = P.acc_in[meta + spare[u]];
        }
    }
  }
}

// ------------------------------------------------------------------ host

struct Sizes {
  int32_t max_len, most;
  size_t kept, holes, spares, total;
};

svx_status sizes(const svx_pages* c, int32_t n_req, int64_t max_len, int32_t budget, Sizes* z) {
  const int64_t cap = static_cast<int64_t>(c->page_size) * c->max_pages;
  if (max_len < 0 || max_len > cap) return paged_fail(SVX_ERR_INVALID_ARG, "max_len must be in [0, max_pages * page_size]");
  if (max_len == 0) max_len = std::min<int64_t>(cap, SVX_EVICT_MAX_LEN);
  if (max_len > SVX_EVICT_MAX_LEN)
    return paged_fail(SVX_ERR_UNSUPPORTED, "max_len must be at most %d (SVX_EVICT_MAX_LEN)", SVX_EVICT_MAX_LEN);
  if (budget < 1) return paged_fail(SVX_ERR_INVALID_ARG, "budget must be >= 1");
  z->max_len = static_cast<int32_t>(max_len);
  z->most = static_cast<int32_t>(std::max<int64_t>(0, std::min<int64_t>(budget, max_len - budget)));
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t rows = static_cast<size_t>(n_req) * c->n_kv_heads;
  z->kept = up(rows * 4);
  z->holes = z->kept + up(static_cast<size_t>(n_req) * 4);
  z->spares = z->holes + up(rows * z->most * 4);
  z->total = z->spares + up(rows * z->most * 4);
  return SVX_OK;
}

template <int KEYS>
cudaError_t launch_select(const EvictParams& p, int rows, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * p.cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, select_kernel<KEYS>, p);
}

}  // namespace
}  // namespace svx

extern "C" svx_status svx_paged_evict_workspace(const svx_pages* cache, int32_t n_req, int64_t max_len, int32_t budget,
                                                int64_t* bytes) {
  if (!bytes) return svx::paged_fail(SVX_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = 0;
  svx::PageView v;
  svx_status st = svx::paged_view(cache, n_req, &v);
  if (st != SVX_OK) return st;
  svx::Sizes z = {};
  st = svx::sizes(cache, n_req, max_len, budget, &z);
  if (st != SVX_OK) return st;
  *bytes = static_cast<int64_t>(z.total);
  return SVX_OK;
}

extern "C" svx_status svx_paged_evict(const svx_pages* cache, int32_t n_req, const int32_t* len, int64_t max_len,
                                      int32_t budget, int32_t sink, int32_t recent, const int32_t* next_pos,
                                      const float* acc_in, const int32_t* pos_in, float* acc_out, int32_t* pos_out,
                                      int32_t* len_out, void* workspace, int64_t workspace_bytes, void* stream) {
  using svx::paged_fail;
  svx::EvictParams p = {};
  svx_status st = svx::paged_view(cache, n_req, &p.pages);
  if (st != SVX_OK) return st;
  svx::Sizes z = {};
  st = svx::sizes(cache, n_req, max_len, budget, &z);
  if (st != SVX_OK) return st;
  if (sink < 0 || recent < 0 || static_cast<int64_t>(sink) + recent > budget)
    return paged_fail(SVX_ERR_INVALID_ARG, "sink and recent must be >= 0, with a sum of at most budget");
  if (!len || !next_pos || !acc_in || !pos_in || !acc_out || !pos_out || !len_out)
    return paged_fail(SVX_ERR_INVALID_ARG, "len, next_pos, acc, pos and len_out must be device pointers");
  const size_t meta = static_cast<size_t>(n_req) * p.pages.n_kv_heads * p.pages.cap * 4;
  auto meets = [](const void* a, const void* b, size_t n) {
    const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
    return x != y && x < y + n && y < x + n;
  };
  if (meets(acc_in, acc_out, meta) || meets(pos_in, pos_out, meta) || meets(len, len_out, static_cast<size_t>(n_req) * 4))
    return paged_fail(SVX_ERR_INVALID_ARG, "acc_out, pos_out and len_out must be their inputs or not overlap them");
  if (!workspace || !svx::is_aligned(workspace, 256) || workspace_bytes < static_cast<int64_t>(z.total))
    return paged_fail(SVX_ERR_INVALID_ARG, "workspace must be 256-byte aligned, of at least %zu bytes", z.total);
  svx::PagedDevice dev(cache->device);
  if (!dev.ok) return paged_fail(SVX_ERR_CUDA, "cannot use device %d", cache->device);
  const void* ptrs[] = {cache->k, cache->v, cache->table, cache->status, len,     next_pos, acc_in,
                        pos_in,   acc_out,  pos_out,      len_out,       workspace};
  for (const void* x : ptrs)
    if (!svx::on_device(x, cache->device))
      return paged_fail(SVX_ERR_INVALID_ARG, "a pointer is not memory of device %d", cache->device);
  const int sms = svx::sm_count(cache->device);
  if (sms <= 0) return paged_fail(SVX_ERR_CUDA, "cannot read the SM count");

  char* ws = static_cast<char*>(workspace);
  p.len = len;
  p.next_pos = next_pos;
  p.acc_in = acc_in;
  p.pos_in = pos_in;
  p.acc_out = acc_out;
  p.pos_out = pos_out;
  p.len_out = len_out;
  p.moves = reinterpret_cast<int32_t*>(ws);
  p.kept = reinterpret_cast<int32_t*>(ws + z.kept);
  p.holes = reinterpret_cast<int32_t*>(ws + z.holes);
  p.spares = reinterpret_cast<int32_t*>(ws + z.spares);
  p.max_len = z.max_len;
  p.budget = budget;
  p.sink = sink;
  p.recent = recent;
  p.most = z.most;
  const int rows = n_req * p.pages.n_kv_heads;
  p.cluster = 1;
  while (p.cluster * svx::kThreads * svx::kMaxKeys < z.max_len) p.cluster *= 2;
  const int per = (z.max_len + p.cluster * svx::kThreads - 1) / (p.cluster * svx::kThreads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = per <= 2    ? svx::launch_select<2>(p, rows, s)
                  : per <= 4  ? svx::launch_select<4>(p, rows, s)
                  : per <= 8  ? svx::launch_select<8>(p, rows, s)
                  : per <= 16 ? svx::launch_select<16>(p, rows, s)
                              : svx::launch_select<32>(p, rows, s);
  if (e == cudaSuccess) {
    // enough CTAs for a row's most moves, no more than about eight per SM over all rows
    const int side = cache->head_dim == 128 ? 1 : 2;
    const int per_cta = svx::kMoveWarps * svx::kMoveBatch * side;
    const int want = (z.most + per_cta - 1) / per_cta, room = std::max(1, 8 * sms / rows);
    const dim3 grid(static_cast<unsigned>(std::max(1, std::min(want, room))), static_cast<unsigned>(rows));
    e = cache->head_dim == 128 ? svx::launch_pdl(svx::move_kernel<128>, grid, dim3(svx::kMoveWarps * 32), 0, s, p)
                               : svx::launch_pdl(svx::move_kernel<64>, grid, dim3(svx::kMoveWarps * 32), 0, s, p);
  }
  if (e != cudaSuccess) return paged_fail(SVX_ERR_CUDA, "evict kernel launch failed: %s", cudaGetErrorString(e));
  return SVX_OK;
}
