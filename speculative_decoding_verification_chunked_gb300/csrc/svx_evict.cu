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
// by histograms of 256 bins: first of the range that the keys span (which spreads them, where their top bits would
// not), then of the bin that holds it, two or three passes as a rule.  The counts are sums of ones: no order of the
// atomics changes a result.  Ties, holes and spares are numbered by ballots and one scan over the warps each.
// move_kernel: a lane works out a move, then the warp brings up to 32 rows of K and V (512 bytes each at d = 128) into
// shared memory with asynchronous copies and writes them out, so a warp has 16 KiB in flight without holding registers.
// Floor: 8 bytes a slot read, 8 a kept slot written, 8 d bytes a moved slot.
// Measured, d = 128, 64 rows: 2112 to 2048 slots 8.0 us (latency: lengths, keys, four histogram passes of 0.7 us, pages,
// rows); 32768 to 4096 61 us, of which selection 18 us (6 to load, 6 for three passes, each with a cluster barrier) and the
// moves 40 us, 235 MB at 5.9 TB/s.  Before: bisection over 32 bits in place of the histograms 137 us in all.
#include <cooperative_groups.h>

#include <algorithm>

#include "svx_paged.h"

namespace cg = cooperative_groups;

namespace svx {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kMaxKeys = 32;    // per thread
constexpr int kMaxCluster = 8;  // portable
constexpr int kSplitKeys = 16;  // a thread's keys above which a row takes more CTAs, where SMs are free: a barrier of the
                                // cluster costs 0.45 us a pass (8 rows of 8192 slots: 8 keys in 2 CTAs 17.6 us, 16 in 1 15.8)
constexpr int kFewThreads = 512;  // up to so many, a CTA makes its row's moves too, if they are few
constexpr int kFewMoves = 8;  // of a warp
static_assert(kMaxThreads * kMaxKeys * kMaxCluster == SVX_EVICT_MAX_LEN, "the longest row a cluster holds");

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
  int32_t chunk;    // moves of a warp at a time, <= 32
  int32_t fused;    // select_kernel makes the moves too
  int32_t head_dim;
};

// Unsigned order = float order; NaN as -inf, -0 as +0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (isnan(w)) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u ^ ((u & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}

constexpr int kBins = 256;
constexpr int kPasses = 4;  // 8 bits of a 32-bit range each

struct Shared {
  int32_t hist[kPasses][kBins];  // a pass has its own, so that none is cleared while a peer may still read it
  int3 found[kPasses];           // bin, its keys, how many of them are kept
  uint2 warp_range[32];
  uint2 peer_range;
  int32_t warp_protected[32];
  int32_t peer_protected;
  int2 warp_scan[2][32];
  int2 peer_scan[2];
};

// Sum of the lower lanes' values.
__device__ __forceinline__ int warp_before(int v, int lane) {
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x - v;
}

// Sums of the values of the warps before this one, in the order (CTA of the cluster, warp); `total` gets all.
// `turn`: a buffer of its own for each use.  In a cluster, every look into a peer's shared memory follows a
// cluster barrier, so the peer has started and has written what is read.
template <int WARPS>
__device__ __forceinline__ int2 cluster_scan(int2 v, Shared& s, int turn, int n_cta, int rank, int2* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) s.warp_scan[turn][warp] = v;
  __syncthreads();
  const int2 x = lane < WARPS ? s.warp_scan[turn][lane] : make_int2(0, 0);
  int2 before = make_int2(__reduce_add_sync(0xffffffffu, lane < warp ? x.x : 0),
                          __reduce_add_sync(0xffffffffu, lane < warp ? x.y : 0));
  int2 sum = make_int2(__reduce_add_sync(0xffffffffu, x.x), __reduce_add_sync(0xffffffffu, x.y));
  if (n_cta > 1) {
    cg::cluster_group cl = cg::this_cluster();
    if (threadIdx.x == 0) s.peer_scan[turn] = sum;
    cl.sync();
    const int2 y = lane < n_cta ? *cl.map_shared_rank(&s.peer_scan[turn], lane) : make_int2(0, 0);
    before.x += __reduce_add_sync(0xffffffffu, lane < rank ? y.x : 0);
    before.y += __reduce_add_sync(0xffffffffu, lane < rank ? y.y : 0);
    sum = make_int2(__reduce_add_sync(0xffffffffu, y.x), __reduce_add_sync(0xffffffffu, y.y));
  }
  *total = sum;
  return before;
}

// One move: where a row of the request's head comes from and where it goes (element offsets; -1: left out).
struct Move {
  int64_t from, to;
};
template <typename T, int D>
__device__ __forceinline__ Move look_up(const EvictParams& P, const int32_t* table, int h, const T* pool, int hole, int spare) {
  const uint32_t ps = P.pages.page_size;
  const uint32_t pt = page_of(P.pages, static_cast<uint32_t>(hole)), pf = page_of(P.pages, static_cast<uint32_t>(spare));
  const int32_t page_to = table[pt], page_from = table[pf];
  Move m{slot_offset(P.pages, page_from, spare - pf * ps), slot_offset(P.pages, page_to, hole - pt * ps)};
  if (m.to < 0 || m.from < 0) {
    atomicOr(P.pages.status, kErrInput);
    return Move{-1, -1};
  }
  const int64_t head = static_cast<int64_t>(h) * P.pages.head_stride;
  m.to += head;
  m.from += head;
  if (!in_bounds(pool + m.from, D, pool, P.pages.extent, P.pages.status, kSitePool) ||
      !in_bounds(pool + m.to, D, pool, P.pages.extent, P.pages.status, kSitePool))
    return Move{-1, -1};
  return m;
}

template <int KEYS, int THREADS>
__global__ void __launch_bounds__(THREADS) select_kernel(const __grid_constant__ EvictParams P) {
  constexpr int kWarps = THREADS / 32;
  __shared__ Shared s;
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
  constexpr int LOADS = KEYS <= 10 ? KEYS : KEYS == 12 ? 6 : 8;  // slots in flight at a time
  static_assert(KEYS % LOADS == 0, "whole turns");
#pragma unroll
  for (int i0 = 0; i0 < KEYS; i0 += LOADS) {
    int32_t pos[LOADS];
    float w[LOADS];
#pragma unroll
    for (int u = 0; u < LOADS; ++u) {
      const int t = first + 32 * (i0 + u);
      pos[u] = t < L ? P.pos_in[meta + t] : 0;
      w[u] = t < L ? P.acc_in[meta + t] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < LOADS; ++u) {
      const uint32_t k = pos[u] < P.sink || pos[u] >= recent_from ? 0xffffffffu : order_key(w[u]);
      key[i0 + u] = first + 32 * (i0 + u) < L ? k : 0u;
    }
  }
  // Keep the keys > cut, and of those equal to it the first `need`.
  uint32_t cut = 0;
  int need = 0;
  if (L > P.budget) {
    // range of the keys that are not protected, and how many are
    uint32_t lo = 0xffffffffu, hi = 0;
    int prot = 0;
#pragma unroll
    for (int i = 0; i < KEYS; ++i) {
      prot += key[i] == 0xffffffffu;
      if (key[i] != 0 && key[i] != 0xffffffffu) {
        lo = min(lo, key[i]);
        hi = max(hi, key[i]);
      }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    prot = __reduce_add_sync(0xffffffffu, prot);
    for (int i = threadIdx.x; i < kPasses * kBins; i += THREADS) (&s.hist[0][0])[i] = 0;
    if (lane == 0) {
      s.warp_range[warp] = make_uint2(lo, hi);
      s.warp_protected[warp] = prot;
    }
    __syncthreads();
    uint2 r = lane < kWarps ? s.warp_range[lane] : make_uint2(0xffffffffu, 0u);
    int q = lane < kWarps ? s.warp_protected[lane] : 0;
    if (n_cta > 1) {
      r = make_uint2(__reduce_min_sync(0xffffffffu, r.x), __reduce_max_sync(0xffffffffu, r.y));
      q = __reduce_add_sync(0xffffffffu, q);
      cg::cluster_group cl = cg::this_cluster();
      if (threadIdx.x == 0) {
        s.peer_range = r;
        s.peer_protected = q;
      }
      cl.sync();
      r = lane < n_cta ? *cl.map_shared_rank(&s.peer_range, lane) : make_uint2(0xffffffffu, 0u);
      q = lane < n_cta ? *cl.map_shared_rank(&s.peer_protected, lane) : 0;
    }
    lo = __reduce_min_sync(0xffffffffu, r.x);
    hi = __reduce_max_sync(0xffffffffu, r.y);
    need = n - __reduce_add_sync(0xffffffffu, q);
    if (need <= 0) {  // only among the protected: the first n of them
      cut = 0xffffffffu;
      need = n;
    } else {
      // up to 256 equal bins, a power of two wide, of [lo, hi], then of the bin in which the need-th largest lies, until
      // all of a bin is kept or it holds one value.  (As L > n, some key is not protected: lo <= hi.)
      uint32_t span = hi - lo;  // the keys in question: lo .. lo + span
      for (int pass = 0;; ++pass) {
        const int shift = max(24 - __clz(span), 0);
#pragma unroll
        for (int i = 0; i < KEYS; ++i) {
          const uint32_t d = key[i] - lo;  // keys below lo wrap to more than span
          if (d <= span) atomicAdd(&s.hist[pass][d >> shift], 1);
        }
        __syncthreads();
        if (n_cta > 1) cg::this_cluster().sync();
        if (warp == 0) {  // lane l has bins 8 l .. 8 l + 7; keys above a bin = suffix sums
          int c[8] = {};
#pragma unroll 2
          for (int peer = 0; peer < n_cta; ++peer) {
            const int32_t* bins = n_cta > 1 ? cg::this_cluster().map_shared_rank(s.hist[pass], peer) : s.hist[pass];
            const int4 x = reinterpret_cast<const int4*>(bins)[2 * lane], y = reinterpret_cast<const int4*>(bins)[2 * lane + 1];
            c[0] += x.x, c[1] += x.y, c[2] += x.z, c[3] += x.w, c[4] += y.x, c[5] += y.y, c[6] += y.z, c[7] += y.w;
          }
          int above = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) above += c[i];
          const int mine = above;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_down_sync(0xffffffffu, above, o);
            if (lane + o < 32) above += y;
          }
          above -= mine;  // keys in the bins of higher lanes
#pragma unroll
          for (int i = 7; i >= 0; --i) {
            // one bin of one lane, as the counts reach need
            if (above < need && above + c[i] >= need) s.found[pass] = make_int3(lane * 8 + i, c[i], need - above);
            above += c[i];
          }
        }
        __syncthreads();
        const int held = s.found[pass].y;
        need = s.found[pass].z;
        lo += static_cast<uint32_t>(s.found[pass].x) << shift;
        if (held == need) {  // the whole bin is kept: the cut lies below it
          cut = lo - 1;
          need = 0;
          break;
        }
        if (shift == 0 || pass == kPasses - 1) {  // (the last pass has shift 0)
          cut = lo;
          break;
        }
        span = min((1u << shift) - 1u, hi - lo);  // (protected keys lie above hi, and the wrap behind them)
      }
    }
  }
  // From here lane i speaks for the 32 slots base .. base + 31, of which lane j held the j-th in key[i]: bit j of its
  // words.  So ties, holes and spares are counted once a word, and one scan over the lanes numbers them.
  const int base = first - lane + 32 * lane;
  uint32_t keep = 0, tie = 0;
#pragma unroll
  for (int i = 0; i < KEYS; ++i) {
    const uint32_t m = __ballot_sync(0xffffffffu, key[i] > cut);
    if (lane == i) keep = m;
  }
  int2 all;
  if (need > 0) {  // the same in all threads of the row
#pragma unroll
    for (int i = 0; i < KEYS; ++i) {
      const uint32_t m = __ballot_sync(0xffffffffu, key[i] == cut);
      if (lane == i) tie = m;
    }
    const int mine = __popc(tie);
    int at = warp_before(mine, lane);
    at += cluster_scan<kWarps>(make_int2(__shfl_sync(0xffffffffu, at + mine, 31), 0), s, 0, n_cta, rank, &all).x;
    // the first need - at of them
    for (int left = need - at; __popc(tie) > max(left, 0);) tie &= ~(0x80000000u >> __clz(tie));
    keep |= tie;
  }
  const int in_front = min(max(n - base, 0), 32);
  const uint32_t front = in_front == 32 ? 0xffffffffu : (1u << in_front) - 1u;  // slots < n
  // weights and positions of the slots that stay where they are
  const bool copy_acc = P.acc_out != P.acc_in, copy_pos = P.pos_out != P.pos_in;
  if (copy_acc || copy_pos) {
#pragma unroll
    for (int i0 = 0; i0 < KEYS; i0 += LOADS) {
      if (first - lane + 32 * i0 >= n) break;  // the same for the warp
      float w[LOADS];
      int32_t pos[LOADS];
      uint32_t stays = 0;
#pragma unroll
      for (int u = 0; u < LOADS; ++u) {  // together, ahead of the stores
        const int64_t t = meta + first + 32 * (i0 + u);
        stays |= (__shfl_sync(0xffffffffu, keep & front, i0 + u) >> lane & 1u) << u;
        if (copy_acc && (stays >> u & 1u)) w[u] = P.acc_in[t];
        if (copy_pos && (stays >> u & 1u)) pos[u] = P.pos_in[t];
      }
#pragma unroll
      for (int u = 0; u < LOADS; ++u) {
        const int64_t t = meta + first + 32 * (i0 + u);
        if (copy_acc && (stays >> u & 1u)) P.acc_out[t] = w[u];
        if (copy_pos && (stays >> u & 1u)) P.pos_out[t] = pos[u];
      }
    }
  }
  uint32_t hole = lane < KEYS ? front & ~keep : 0u, spare = keep & ~front;
  int ah = warp_before(__popc(hole), lane), as = warp_before(__popc(spare), lane);
  const int2 warp_all = make_int2(__shfl_sync(0xffffffffu, ah + __popc(hole), 31), __shfl_sync(0xffffffffu, as + __popc(spare), 31));
  const int2 start = cluster_scan<kWarps>(warp_all, s, 1, n_cta, rank, &all);
  ah += start.x;
  as += start.y;
  if (threadIdx.x == 0 && rank == 0) P.moves[row] = min(min(all.x, all.y), P.most);
  int32_t* holes = P.holes + static_cast<int64_t>(row) * P.most;
  int32_t* spares = P.spares + static_cast<int64_t>(row) * P.most;
  const uint32_t before = (1u << lane) - 1u;
#pragma unroll
  for (int i = 0; i < KEYS; ++i) {
    const uint32_t mh = __shfl_sync(0xffffffffu, hole, i), ms = __shfl_sync(0xffffffffu, spare, i);
    if (mh) {  // the same in all lanes
      const int ih = __shfl_sync(0xffffffffu, ah, i) + __popc(mh & before);
      if ((mh >> lane & 1u) && ih < P.most) holes[ih] = first + 32 * i;
    }
    if (ms) {
      const int is = __shfl_sync(0xffffffffu, as, i) + __popc(ms & before);
      if ((ms >> lane & 1u) && is < P.most) spares[is] = first + 32 * i;
    }
  }
  if (n_cta > 1) cg::this_cluster().sync();  // no CTA leaves while another may still read its shared memory
  if constexpr (THREADS > kFewThreads) return;
  if (!P.fused) return;
  // Few moves, one small CTA to the row: they are made here, without another kernel.
  if (threadIdx.x == 0 && row == b * P.pages.n_kv_heads) P.len_out[b] = n;
  __syncthreads();  // holes and spares are written
  const int M = min(min(all.x, all.y), P.most);
  const int32_t* table = P.pages.table + static_cast<int64_t>(b) * P.pages.max_pages;
  const int h = row - b * P.pages.n_kv_heads;
  using T = uint16_t;
  T *pk = static_cast<T*>(P.pages.k), *pv = static_cast<T*>(P.pages.v);
  // A lane looks up a move, eight to a warp; then d / 8 lanes copy a row of K and as many its row of V.
  constexpr int kFew = 8;
  const int pieces = P.head_dim / 8, side = 16 / pieces;  // side: moves of a warp at a time
  const int piece = lane % pieces, mine = (lane % 16) / pieces;
  T* pool = lane >= 16 ? pv : pk;
  for (int i0 = warp * kFew; i0 < M; i0 += kWarps * kFew) {
    Move m{-1, -1};
    if (lane < kFew && i0 + lane < M) {
      const int hole = holes[i0 + lane], spare = spares[i0 + lane];
      const float w = P.acc_in[meta + spare];
      const int32_t pos = P.pos_in[meta + spare];
      m = P.head_dim == 128 ? look_up<T, 128>(P, table, h, pk, hole, spare) : look_up<T, 64>(P, table, h, pk, hole, spare);
      P.acc_out[meta + hole] = w;
      P.pos_out[meta + hole] = pos;
    }
    int64_t to[kFew];
    uint4 v[kFew];
#pragma unroll
    for (int u = 0; u < kFew; ++u) {
      const int k = u * side + mine;  // (with two at a time, four turns do)
      const int64_t from = __shfl_sync(0xffffffffu, m.from, k & 7);
      to[u] = __shfl_sync(0xffffffffu, m.to, k & 7);
      if (k >= kFew) to[u] = -1;
      if (to[u] >= 0) v[u] = reinterpret_cast<const uint4*>(pool + from)[piece];
    }
#pragma unroll
    for (int u = 0; u < kFew; ++u)
      if (to[u] >= 0) reinterpret_cast<uint4*>(pool + to[u])[piece] = v[u];
  }
}

constexpr int kMoveWarps = 2;

template <int D>
__global__ void __launch_bounds__(kMoveWarps * 32) move_kernel(const __grid_constant__ EvictParams P) {
  using T = uint16_t;                      // rows move as bits, whatever the type
  constexpr int PIECES = D / 8;            // 16-byte pieces of a row
  constexpr int SIDE = 32 / (2 * PIECES);  // moves of a warp at a time: K on one half of the lanes, V on the other
  grid_dependency_wait();
  allow_dependents();
  const int row = blockIdx.x, b = row / P.pages.n_kv_heads, h = row - b * P.pages.n_kv_heads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.y == 0 && h == 0 && threadIdx.x == 0) P.len_out[b] = P.kept[b];
  const int M = P.moves[row];
  const int32_t* holes = P.holes + static_cast<int64_t>(row) * P.most;
  const int32_t* spares = P.spares + static_cast<int64_t>(row) * P.most;
  const int64_t meta = static_cast<int64_t>(row) * P.pages.cap;
  const int32_t* table = P.pages.table + static_cast<int64_t>(b) * P.pages.max_pages;
  const bool is_v = lane >= 16;
  const int piece = lane % PIECES, side = (lane % 16) / PIECES;
  T* pool = static_cast<T*>(is_v ? P.pages.v : P.pages.k);
  __shared__ uint4 buf[kMoveWarps][32 / SIDE][32];
  const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(&buf[warp][0][lane]));
  const int step = gridDim.y * kMoveWarps * P.chunk;
  for (int i0 = (blockIdx.y * kMoveWarps + warp) * P.chunk; i0 < M; i0 += step) {
    // one lane works out one move: where from, where to; and moves the slot's weight and position
    int64_t from = -1, to = -1;
    if (lane < P.chunk && i0 + lane < M) {
      const int hole = holes[i0 + lane], spare = spares[i0 + lane];
      const float w = P.acc_in[meta + spare];
      const int32_t pos = P.pos_in[meta + spare];
      const Move move = look_up<T, D>(P, table, h, pool, hole, spare);
      from = move.from;
      to = move.to;
      P.acc_out[meta + hole] = w;
      P.pos_out[meta + hole] = pos;
    }
    // the rows come in together, 16 bytes a lane and copy, and leave together
    const int n = min(P.chunk, M - i0);
#pragma unroll 4
    for (int c = 0; c < n; c += SIDE) {
      const int m = c + side;
      const int64_t f = __shfl_sync(0xffffffffu, from, m & 31);
      if (m < n && f >= 0)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(mine + (c / SIDE) * 512u),
                     "l"(reinterpret_cast<const uint4*>(pool + f) + piece)
                     : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // a lane reads back what it copied itself
#pragma unroll 4
    for (int c = 0; c < n; c += SIDE) {
      const int m = c + side;
      const int64_t t = __shfl_sync(0xffffffffu, to, m & 31);
      if (m < n && t >= 0) reinterpret_cast<uint4*>(pool + t)[piece] = buf[warp][c / SIDE][lane];
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

template <int KEYS, int THREADS>
cudaError_t launch_select(const EvictParams& p, int rows, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * p.cluster);
  cfg.blockDim = dim3(THREADS);
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
  return cudaLaunchKernelEx(&cfg, select_kernel<KEYS, THREADS>, p);
}

// Threads and CTAs of a row: few warps where few slots need them, since every histogram pass waits for all; a cluster of
// CTAs where one does not hold the row, or where there are SMs for it and it shortens a thread's part.  (64 rows of 2112
// slots: 256 threads 7.9 us, 512 8.5; of 4096: 512 threads 8.9 us, 256 9.9.)
constexpr int kSmallRow = 256 * 10, kMiddleRow = 512 * 16;
cudaError_t launch_selects(EvictParams& p, int rows, int sms, cudaStream_t s) {
  const int threads = p.max_len <= kSmallRow ? 256 : p.max_len <= kMiddleRow ? kFewThreads : kMaxThreads;
  p.cluster = 1;
  auto keys = [&](int c) { return (p.max_len + c * threads - 1) / (c * threads); };
  while (p.cluster < kMaxCluster &&
         (keys(p.cluster) > kMaxKeys || (keys(p.cluster) > kSplitKeys && rows * p.cluster * 2 <= sms)))
    p.cluster *= 2;
  // Moves in the same kernel where a small CTA has one turn of its warps of them, which saves a launch and a trip through
  // memory: 64 rows of 2112 slots to 2048 take 8.0 us so and 8.7 us in two kernels.  With two turns it is slower: 64 rows of
  // 2176 to 2048 9.8 and 9.2 us, 256 rows of 1152 to 1024 14.6 and 13.0; 64 rows of 4352 to 4096 15.6 and 12.7.  Not
  // where the new lengths go over the old, which other heads' CTAs may still have to read.
  p.fused = threads <= kFewThreads && p.cluster == 1 && p.most <= kFewMoves * (threads / 32) && p.len_out != p.len;
  const int per = keys(p.cluster);
  if (threads == 256)
    return per <= 4   ? launch_select<4, 256>(p, rows, s)
           : per <= 8 ? launch_select<8, 256>(p, rows, s)
                      : launch_select<10, 256>(p, rows, s);
  if (threads == kFewThreads)
    return per <= 8    ? launch_select<8, kFewThreads>(p, rows, s)
           : per <= 12 ? launch_select<12, kFewThreads>(p, rows, s)
                       : launch_select<16, kFewThreads>(p, rows, s);
  return per <= 12   ? launch_select<12, kMaxThreads>(p, rows, s)
         : per <= 16 ? launch_select<16, kMaxThreads>(p, rows, s)
                     : launch_select<32, kMaxThreads>(p, rows, s);
}

cudaError_t launch_moves(EvictParams& p, int head_dim, int rows, int sms, cudaStream_t s) {
  // moves of a warp: as many as it looks up at a time, fewer where that leaves SMs without a warp
  p.chunk = 32;
  while (p.chunk > 8 && static_cast<int64_t>(rows) * p.most < static_cast<int64_t>(p.chunk) * sms * kMoveWarps) p.chunk /= 2;
  const int per_cta = kMoveWarps * p.chunk;
  const int want = (p.most + per_cta - 1) / per_cta, room = std::max(1, 40 * sms / rows);
  const dim3 grid(static_cast<unsigned>(rows), static_cast<unsigned>(std::max(1, std::min(want, room))));
  return head_dim == 128 ? launch_pdl(move_kernel<128>, grid, dim3(kMoveWarps * 32), 0, s, p)
                         : launch_pdl(move_kernel<64>, grid, dim3(kMoveWarps * 32), 0, s, p);
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
  if (!svx::words_aligned({len, next_pos, acc_in, pos_in, acc_out, pos_out, len_out}))
    return paged_fail(SVX_ERR_INVALID_ARG, "len, next_pos, acc, pos and len_out must be 4-byte aligned");
  const size_t meta = static_cast<size_t>(n_req) * p.pages.n_kv_heads * p.pages.cap * 4;
  const size_t per_req = static_cast<size_t>(n_req) * 4;
  if (!workspace || !svx::is_aligned(workspace, 256) || workspace_bytes < static_cast<int64_t>(z.total))
    return paged_fail(SVX_ERR_INVALID_ARG, "workspace must be 256-byte aligned, of at least %zu bytes", z.total);
  // The pools are written too (a strided one takes what lies between its rows along).
  const size_t pool = static_cast<size_t>(p.pages.extent) * 2;
  const svx::Span k_span = {cache->k, pool}, v_span = {cache->v, pool}, next_span = {next_pos, per_req},
                  table_span = {cache->table, per_req * cache->max_pages};
  auto meets_pool = [&](const svx::Span& s) { return svx::any_overlap({s}, {k_span, v_span}); };
  if (svx::any_overlap({{acc_out, meta}, {pos_out, meta}, {len_out, per_req}, {workspace, z.total}, {cache->status, 4}},
                       {{acc_in == acc_out ? nullptr : acc_in, meta},
                        {pos_in == pos_out ? nullptr : pos_in, meta},
                        {len == len_out ? nullptr : len, per_req},
                        next_span,
                        table_span,
                        k_span,
                        v_span}) ||
      meets_pool({acc_in, meta}) || meets_pool({pos_in, meta}) || meets_pool({len, per_req}) || meets_pool(next_span) ||
      meets_pool(table_span))
    return paged_fail(SVX_ERR_INVALID_ARG, "an output or the workspace overlaps an input, another output or the pools "
                                           "(acc_out, pos_out and len_out may be their inputs)");
  // (one buffer for K and V moves its rows twice, to the same places: no harm)
  if (svx::pools_collide(cache, false)) return paged_fail(SVX_ERR_INVALID_ARG, "rows of the K and V pages share memory");
  svx::PagedDevice dev(cache->device);
  if (!dev.ok) return paged_fail(SVX_ERR_CUDA, "cannot use device %d", cache->device);
  const void* ptrs[] = {cache->k, cache->v, cache->table, cache->status, len,     next_pos, acc_in,
                        pos_in,   acc_out,  pos_out,      len_out,       workspace};
  for (const void* x : ptrs)
    if (!(cache->flags & SVX_POINTERS_CHECKED) && !svx::on_device(x, cache->device))
      return paged_fail(SVX_ERR_INVALID_ARG, "a pointer is not memory of device %d", cache->device);
  const int sms = svx::sm_count(cache->device);
  if (sms <= 0) return paged_fail(SVX_ERR_CUDA, "cannot read the SM count");

  p.pages.extent = svx::clipped(svx::kClipPool, p.pages.extent);
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
  p.head_dim = cache->head_dim;
  const int rows = n_req * p.pages.n_kv_heads;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = svx::launch_selects(p, rows, sms, s);
  if (e == cudaSuccess && !p.fused) e = svx::launch_moves(p, cache->head_dim, rows, sms, s);
  if (e != cudaSuccess) return paged_fail(SVX_ERR_CUDA, "evict kernel launch failed: %s", cudaGetErrorString(e));
  return SVX_OK;
}
