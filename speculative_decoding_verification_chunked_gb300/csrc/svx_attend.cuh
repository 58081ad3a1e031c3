// Attention of few rows to the same keys: one new token per request over a paged cache (kPaged, which the figures below are of), a few
// rows against an encoder's states (kDense), and rows of shared prefixes beside the requests' own slots (kShared).
//
//   s_t = scale q.k_t,  m = max s,  p_t = e^(s_t - m),  l = sum p,  O = sum p v / l,  LSE = m + ln l
//
// Every K and V row is used by the G query heads of its KV head and never again: 4 G flops an element read, so
// the bytes of K and V are the floor, and the kernel's task is to keep enough of them in flight.
//
// Work.  The slots of every (request, KV head, block of 16 query heads) - an item - are cut into chunks of
// 4 KiB of K; all items' chunks form one flat range, which is cut evenly over the CTAs and again over a CTA's warps
// ("stream-K"), so a ragged batch loads every warp alike, and one long request uses all of them.  The lengths are read on
// the device.  A warp is its own pipeline: it brings its chunks in with 16-byte cp.async (rows found through the page
// table, the next entry fetched a chunk ahead), kStages deep, through the ends of items and with no barrier shared with
// the other warps.  8 warps x 2 chunks in flight are 128 KiB an SM.
// An item that lies in one warp is finished there.  Of the others a warp keeps the piece that ends in its range in global
// memory (lead) and the one that goes on behind it in its emptied stages (tail); when all warps of the CTA are done
// they merge the pieces that belong together, finish the items that lie in the CTA, and leave (m, l, O) of the others in the
// CTA's slot 0 (the item began before the CTA's range) or 1 (it goes on behind it), which join_kernel merges.
// (Where the warps of a CTA shared an item's chunks in turn and merged at its end, every item stopped the CTA: 16 requests
// of 1 to 8192 slots, 8 KV heads, took 70 us and take 48 us so; 64 of 100 to 1000 slots 58 and 31 us.)
// What bounds it: the copy rate.  8 x 32768 slots (8 KV heads, d = 128, 1.07 GB) 159 us = 6750 GB/s, 99.5% of the
// measured copy rate; 1 x 131072 slots 86 us = 6260 GB/s; below some 200 MB the fixed cost shows, about 5 us until the
// first chunk is in (lengths, split, page table, chunk: four trips to memory in a row) and 5 us of joining.
//
// Products: mma.sync m16n8k16, query heads on M.  They cost a few percent of the time (32 a chunk), so the
// tensor memory path, which wants 64 rows or more on M and a second trip through it, gains nothing here.  With up to 8
// query heads per KV head the upper 8 rows would be idle: they carry what is left of p after its rounding to a 16-bit type,
// so P.V has p to 2^-16 of itself (bf16) or better at no extra product, far within the output's own rounding.  With 9 to
// 16 the remainder is a second product.
// Softmax state, scores and sums are fp32.  m is not the maximum but a reference that moves only when a score passes it
// by more than kTau, so most chunks need no exchange between lanes; every merge takes (m, l, O) with any reference.
#pragma once

#include "svx_paged.h"

#include <algorithm>
#include <atomic>
#include <cfloat>

namespace svx {
namespace {

constexpr int kWarps = 8;
constexpr int kStages = 3;
constexpr uint32_t kMinChunks = 2 * kWarps;  // a CTA takes at least so many chunks, if there are
constexpr int kChunkBytes = 4096;  // of K (and as much of V)
constexpr int kRowsMax = 16;       // query heads of an item
constexpr float kTau = 8.0f;       // p stays below 2^8
constexpr float kLn2 = 0.69314718055994530942f;
#define kNegInf (-INFINITY)

// What the kernels attend to.
enum Source : int {
  kPaged = 0,   // a request's pages: one token per request (svx_paged_decode)
  kDense = 1,   // an encoder's states [request][state][KV head][d], any tokens of the request, a mask (svx_cross_attn)
  kShared = 2,  // the pages of prefixes, each for the rows of several requests, and behind them the requests' own (svx_paged_decode_shared)
};

struct AttendParams {
  PageView pages;
  const void* q;
  const int32_t* len;
  void* o;
  float* lse;
  const float* acc_in;
  float* acc_out;
  float* lead;      // [ctas][8 warps][16][D]
  float2* lead_ml;  // [ctas][8 warps][16]
  float* part_o;    // [ctas][2][16][D]
  float2* part_ml;  // [ctas][2][16]
  float2* row_ml;   // [n_req * n_q]: final (m, l), for the weights
  float* scores;    // [n_req * n_q][score_stride], log2 units
  int64_t score_stride;
  float scale;      // softmax scale * log2(e)
  int32_t max_len;
  int32_t n_q, group, blocks;  // blocks of 16 query heads per KV head
  int32_t whole;               // no item is split over CTAs: there is nothing to join
  int32_t ctas;                // of the attention kernel
  // kDense (pages: one of max_len slots per request, and no table)
  const uint8_t* mask;  // [n_req][mask_stride]: 0: hidden; or NULL
  int64_t mask_stride;
  int64_t q_b, q_h, q_n, o_b, o_h, o_n;  // elements between requests, heads and tokens
  int32_t n_tok, rows;                   // tokens of a request; group * n_tok
  // kShared
  const int32_t* prefix_table;  // [n_prefix][prefix_max_pages]
  const int32_t* prefix_len;
  const int32_t* first;         // [n_prefix + 1]: the requests of each prefix
  int32_t n_prefix, prefix_max_pages, max_prefix;
  int32_t prefix_apart;         // the prefixes are another kernel's work
  float* state_o;               // [2][n_req * n_q][D]: finished states, of the prefix and of the request's own slots
  float2* state_ml;             // [2][n_req * n_q]
  // of rows_kernel (svx_rows.cuh)
  float4* rows_o;               // [row_ctas][2][D / 4][item_rows]: states of items that more than one CTA works on
  float2* rows_ml;              // [row_ctas][2][item_rows]
  float4* row_sums;             // [row_ctas][2 streams][D / 4][128 rows]: of long segments (rows_kernel's kSumTiles)
  float* row_refs;              // [row_ctas][2][128]: what they are relative to
  int32_t item_rows, row_ctas, row_least;
  int32_t row_whole;            // items are not split over CTAs
  int32_t expire;               // test hook: a wait is made to run out
  float group_inverse;          // 1 / group
};

// The flat range of chunks, as every kernel of the call computes it from the lengths.  Sequences: the requests;
// kShared: the prefixes (kMaxReq places), then the requests.
template <int SRC>
struct Plan {
  static constexpr int SEQS = SRC == kShared ? 2 * kMaxReq : kMaxReq;
  int32_t first[SEQS + 1];  // first chunk of each sequence's items; their number (below 2^31: checked on the host)
  int32_t warp_sum[kWarps];
  int32_t n[SEQS];          // chunks of one of a sequence's items
  int32_t len[SEQS];        // its length, within bounds
  int32_t req0[SRC == kShared ? kMaxReq + 1 : 1];  // the first request of each prefix, and one past the last one's
  int32_t row_tiles;        // (join_shared) rows_kernel's tiles
};

constexpr int kKeyTile = 128;  // keys of a tile of rows_kernel

// Sums x over the first kMaxReq threads of the block up to this one, and all of theirs into `total`.
__device__ __forceinline__ int block_scan(int x, int32_t* warp_sum, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31 && warp < kWarps) warp_sum[warp] = x;
  __syncthreads();
  int base = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int v = warp_sum[w];
    if (w < warp) base += v;
    total += v;
  }
  return base + x;
}

// The requests of each prefix: first[p] within bounds, and no lower than those before it.
__device__ __forceinline__ void prefix_requests(const int32_t* first, int n_prefix, int n_req, int32_t* req0, int32_t* warp_top,
                                                int* status) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int raw = t < n_prefix ? first[t] : 0, last = t == 0 ? first[n_prefix] : 0;
  int x = min(max(raw, 0), n_req);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x = max(x, y);
  }
  if (lane == 31 && warp < kWarps) warp_top[warp] = x;
  __syncthreads();
  int top = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int v = warp_top[w];
    if (w < warp) x = max(x, v);
    top = max(top, v);  // (threads behind the prefixes have 0)
  }
  if (t < kMaxReq) req0[t] = t < n_prefix ? x : top;  // (a prefix's end is the next one's begin)
  if (status && t < n_prefix && x != raw) atomicOr(status, kErrInput);
  __syncthreads();
  if (t == 0) {
    const int end = max(min(max(last, 0), n_req), top);
    req0[n_prefix] = end;
    if (status && end != last) atomicOr(status, kErrInput);
  }
  __syncthreads();
}

// `tiles`: the prefixes are rows_kernel's work, and `first` and `n` of theirs count its tiles, from 0 (the join's view).
template <int SRC, int CT>
__device__ __forceinline__ int build_plan(const AttendParams& P, Plan<SRC>& s, bool report, bool tiles = false) {
  // one request per thread (kMaxReq = threads of a block), prefix sum over the block
  static_assert(kMaxReq == kWarps * 32, "one thread per request");
  const int t = threadIdx.x;
  int before = 0;
  if constexpr (SRC == kShared) {
    prefix_requests(P.first, P.n_prefix, P.pages.n_req, s.req0, s.warp_sum, report ? P.pages.status : nullptr);
    int n = 0, rows = 0;
    if (t < P.n_prefix) {
      const int raw = P.prefix_len[t];
      n = min(max(raw, 0), P.max_prefix);
      if (report && n != raw) atomicOr(P.pages.status, kErrInput);
      rows = (s.req0[t + 1] - s.req0[t]) * P.group;
    }
    const int per = tiles ? kKeyTile : CT, block = tiles ? P.item_rows : kRowsMax;
    const int chunks = (P.prefix_apart && !tiles) || rows == 0 ? 0 : static_cast<int>((static_cast<uint32_t>(n) + (per - 1)) / per);
    s.n[t] = chunks;
    s.len[t] = n;
    const int mine = P.pages.n_kv_heads * ((rows + block - 1) / block) * chunks;
    s.first[t] = block_scan(mine, s.warp_sum, before) - mine;
    if (tiles) {
      if (t == 0) s.row_tiles = before;
      before = 0;
    }
    __syncthreads();
  }
  constexpr int at = SRC == kShared ? kMaxReq : 0;
  int n = 0;
  if (t < P.pages.n_req) {
    const int raw = SRC == kDense && !P.len ? P.max_len : P.len[t];
    n = min(max(raw, 0), P.max_len);
    if (report && n != raw && P.pages.status) atomicOr(P.pages.status, kErrInput);
  }
  const int chunks = static_cast<int>((static_cast<uint32_t>(n) + (CT - 1)) / CT);
  s.n[at + t] = chunks;
  s.len[at + t] = n;
  const int mine = P.pages.n_kv_heads * P.blocks * chunks;
  int total;
  s.first[at + t] = before + block_scan(mine, s.warp_sum, total) - mine;
  total += before;
  if (t == 0) s.first[Plan<SRC>::SEQS] = total;
  __syncthreads();
  return total;
}

// The T chunks over the CTAs: the first `used` ones share them, CTA c has [begin(c), begin(c + 1)) = [floor(c T / used), ..),
// in 32 bits with T = q used + r.
struct Split {
  uint32_t used, q, r, total;
  float per_used;
  __device__ __forceinline__ Split(const AttendParams& P, int T) {
    total = T;
    used = min((total + kMinChunks - 1) / kMinChunks, static_cast<uint32_t>(P.ctas));
    q = used ? total / used : 0;
    r = total - q * used;
    per_used = __frcp_rn(static_cast<float>(used));
  }
  // c r <= 2^16, and its quotient by used <= 256 is whole or at least 1/256 off: the float product is within 2^-14 of it
  __device__ __forceinline__ int begin(uint32_t c) const {
    return static_cast<int>(c * q) + __float2int_rd(fmaf(static_cast<float>(c * r), per_used, 0.001f));
  }
  // the CTA that holds chunk x
  __device__ __forceinline__ int of(int x) const {
    int c = min(static_cast<int>(static_cast<float>(x) * (static_cast<float>(used) / static_cast<float>(total))),
                static_cast<int>(used) - 1);
    while (c + 1 < static_cast<int>(used) && begin(c + 1) <= x) ++c;
    while (c > 0 && begin(c) > x) --c;
    return c;
  }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes),
               "l"(policy)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
struct Mma;
template <>
struct Mma<__nv_bfloat16> {
  static constexpr float kLift = 0.f;
  static __device__ __forceinline__ void go(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
  // two values rounded, and what the rounding left
  static __device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
    __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    hi = *reinterpret_cast<uint32_t*>(&h);
    __nv_bfloat162 l = __floats2bfloat162_rn(x - __low2float(h), y - __high2float(h));
    lo = *reinterpret_cast<uint32_t*>(&l);
  }
  static __device__ __forceinline__ uint32_t down2(float x, float y) {
    __nv_bfloat162 a = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<uint32_t*>(&a);
  }
  static __device__ __forceinline__ uint2 down4(float4 v) {
    __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    return make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
  }
};
template <>
struct Mma<__half> {
  // fp16 loses what lies below 2^-25: p is held 2^7 times as large (below 2^15), so that slots of little weight,
  // of which a long cache has many, keep theirs
  static constexpr float kLift = 7.f;
  static __device__ __forceinline__ void go(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
    __half2 h = __floats2half2_rn(x, y);
    hi = *reinterpret_cast<uint32_t*>(&h);
    __half2 l = __floats2half2_rn(x - __low2float(h), y - __high2float(h));
    lo = *reinterpret_cast<uint32_t*>(&l);
  }
  static __device__ __forceinline__ uint32_t down2(float x, float y) {
    __half2 a = __floats2half2_rn(x, y);
    return *reinterpret_cast<uint32_t*>(&a);
  }
  static __device__ __forceinline__ uint2 down4(float4 v) {
    __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
    return make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
  }
};

// A piece of an item that a warp does not finish itself.
struct Piece {
  int32_t first, end;  // the item's chunks; first < 0: there is no such piece
  int32_t b, h, blk;
};

template <int D>
struct Smem {
  static constexpr int RING = kStages * 2 * kChunkBytes;  // a warp's stages; at the end its tail [16 rows][D], then (m, l)
  static constexpr int OFF_PIECE = kWarps * RING;         // [leads, tails][8 warps]
  static constexpr int BYTES = OFF_PIECE + kWarps * 2 * static_cast<int>(sizeof(Piece));
  static_assert(kRowsMax * D * 4 + kRowsMax * 8 <= RING, "a tail fits the stages");
  // a row's float4 columns are permuted by the row, so that the fragments' stores spread over the banks
  static __device__ __forceinline__ int at(int r, int d) { return r * D + ((d >> 2 ^ (r & 7)) << 2) + (d & 3); }
};

// A place in the flat range: the item it lies in.
struct Cursor {
  int first, end;  // the item's chunks
  int b, h, blk;       // sequence, KV head, block of its rows
  int len;
};

// The rows of an item: query heads of a KV head for the request's token, or (kDense) for each of its tokens, or (kShared, a
// prefix) of each of its requests.
template <int SRC>
__device__ __forceinline__ int seq_rows(const AttendParams& P, const Plan<SRC>& s, int b) {
  if constexpr (SRC == kDense) return P.rows;
  if constexpr (SRC == kShared) return b < kMaxReq ? (s.req0[b + 1] - s.req0[b]) * P.group : P.group;
  return P.group;
}
template <int SRC>
__device__ __forceinline__ int item_rows(const AttendParams& P, const Plan<SRC>& s, int b, int blk) {
  return min(seq_rows(P, s, b) - blk * kRowsMax, kRowsMax);
}
// Row r of an item as a row of a dense [n_req][n_q] (kPaged, kShared), or its request, head and token.
template <int SRC>
__device__ __forceinline__ int64_t out_row(const AttendParams& P, const Plan<SRC>& s, int b, int h, int blk, int r) {
  r += blk * kRowsMax;
  if constexpr (SRC == kShared) {
    if (b < kMaxReq) {
      const int j = r / P.group;
      return static_cast<int64_t>(s.req0[b] + j) * P.n_q + h * P.group + (r - j * P.group);
    }
    b -= kMaxReq;
  }
  return static_cast<int64_t>(b) * P.n_q + h * P.group + r;
}
struct Token {
  int head, tok;
};
__device__ __forceinline__ Token dense_row(const AttendParams& P, int h, int blk, int r) {
  r += blk * kRowsMax;
  const int tok = P.n_tok == 1 ? 0 : r / P.group;
  return Token{h * P.group + (r - tok * P.group), tok};
}
template <int SRC, int D>
__device__ __forceinline__ int64_t q_at(const AttendParams& P, const Plan<SRC>& s, int b, int h, int blk, int r) {
  if constexpr (SRC == kDense) {
    const Token t = dense_row(P, h, blk, r);
    return b * P.q_b + t.head * P.q_h + t.tok * P.q_n;
  }
  return out_row<SRC>(P, s, b, h, blk, r) * D;
}
// Places of a finished row: O, and LSE (an index).
struct RowOut {
  int64_t o, lse;
};
template <int SRC, int D>
__device__ __forceinline__ RowOut place(const AttendParams& P, const Plan<SRC>& s, int b, int h, int blk, int r) {
  if constexpr (SRC == kDense) {
    const Token t = dense_row(P, h, blk, r);
    return RowOut{b * P.o_b + t.head * P.o_h + t.tok * P.o_n, (static_cast<int64_t>(b) * P.n_q + t.head) * P.n_tok + t.tok};
  }
  const int64_t row = out_row<SRC>(P, s, b, h, blk, r);
  return RowOut{row * D, row};
}

// Moves on to the item that holds x (all lanes of a warp alike).
template <int SRC>
__device__ __forceinline__ void seek(Cursor& c, const AttendParams& P, const Plan<SRC>& s, int x) {
  if (x >= s.first[c.b + 1]) {  // another sequence: as many lie before it as end at x or before
    const int seqs = (SRC == kShared ? kMaxReq : 0) + P.pages.n_req;
    c.b = 0;
    for (int i = 0; i < seqs; i += 32) {
      const int r = i + (threadIdx.x & 31);
      c.b += __popc(__ballot_sync(0xffffffffu, r < seqs && s.first[r + 1] <= x));
    }
  }
  const int n = s.n[c.b];
  const int i = static_cast<int>(static_cast<uint32_t>(x - s.first[c.b]) / static_cast<uint32_t>(n));
  c.len = s.len[c.b];
  c.first = s.first[c.b] + i * n;
  c.end = c.first + n;
  const int blocks = SRC == kShared && c.b < kMaxReq ? (seq_rows(P, s, c.b) + kRowsMax - 1) / kRowsMax : P.blocks;
  c.h = blocks == 1 ? i : i / blocks;
  c.blk = i - c.h * blocks;
}

// The first chunk at x or behind it that begins an item.
template <int SRC>
__device__ __forceinline__ int item_start(const AttendParams& P, const Plan<SRC>& s, int x, int total) {
  if (x >= total) return total;
  Cursor c{0, 0, 0, 0, 0, 0};
  seek(c, P, s, x);
  return c.first == x ? x : c.end;
}

// O and LSE of a row from its merged state.
template <typename T>
__device__ __forceinline__ void write_row(const AttendParams& P, const RowOut& at, int d4, float M, float L, float4 o) {
  const float inv = L == 0.f ? 0.f : 1.f / L;
  o = L == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(static_cast<T*>(P.o) + at.o + d4) = Mma<T>::down4(o);
  if (d4 == 0 && P.lse) P.lse[at.lse] = L == 0.f ? kNegInf : (M + log2f(L)) * kLn2;
}

// Requests without slots: O = 0, LSE = -inf.
template <typename T, int SRC, int D>
__device__ __forceinline__ void write_empty(const AttendParams& P, const Plan<SRC>& plan) {
  for (int b = blockIdx.x; b < P.pages.n_req; b += gridDim.x) {
    if (plan.first[b + 1] > plan.first[b]) continue;
    if constexpr (SRC == kDense) {
      const int rows = P.rows * P.pages.n_kv_heads;
      for (int i = threadIdx.x; i < rows * (D / 4); i += blockDim.x) {
        const int row = i / (D / 4), h = row / P.rows;
        write_row<T>(P, place<SRC, D>(P, plan, b, h, 0, row - h * P.rows), (i - row * (D / 4)) * 4, 0.f, 0.f, make_float4(0.f, 0.f, 0.f, 0.f));
      }
      continue;
    }
    uint32_t* ob = reinterpret_cast<uint32_t*>(static_cast<T*>(P.o) + static_cast<int64_t>(b) * P.n_q * D);
    for (int i = threadIdx.x; i < P.n_q * D / 2; i += blockDim.x) ob[i] = 0u;
    for (int i = threadIdx.x; i < P.n_q; i += blockDim.x) P.lse[static_cast<int64_t>(b) * P.n_q + i] = kNegInf;
  }
}

template <typename T, int SRC, int D, bool WIDE, bool SCORES>
__global__ void __launch_bounds__(kWarps * 32, 1) attend_kernel(const __grid_constant__ AttendParams P) {
  constexpr int CT = kChunkBytes / (2 * D);  // slots of a chunk: 16 (d = 128) or 32 (d = 64)
  constexpr int NT = CT / 8;                 // score tiles
  constexpr int KS = D / 16;
  constexpr int NO = D / 8;                  // output tiles
  constexpr int PIECES = D / 8;              // 16-byte pieces of a row
  constexpr int RPI = 32 / PIECES;           // rows that a warp's 32 lanes copy at a time
  using S = Smem<D>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Plan<SRC> plan;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  grid_dependency_wait();
  allow_dependents();
  const int T_all = build_plan<SRC, CT>(P, plan, blockIdx.x == 0);

  const Split split(P, T_all);
  if (blockIdx.x >= split.used) {
    if constexpr (SRC != kShared) write_empty<T, SRC, D>(P, plan);  // (kShared: the join's work)
    return;
  }
  int x0 = split.begin(blockIdx.x), x1 = split.begin(blockIdx.x + 1);
  if (P.whole) {  // the items that begin in the range, whole
    x0 = item_start(P, plan, x0, T_all);
    x1 = item_start(P, plan, x1, T_all);
  }
  const int w0 = x0 + static_cast<int>(static_cast<int64_t>(x1 - x0) * warp / kWarps);
  const int w1 = x0 + static_cast<int>(static_cast<int64_t>(x1 - x0) * (warp + 1) / kWarps);

  const uint32_t stage0 = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * S::RING;
  Piece* pieces = reinterpret_cast<Piece*>(smem + S::OFF_PIECE);
  if (lane < 2) pieces[lane * kWarps + warp].first = -1;
  __syncwarp();

  // K and V are read once: they leave L2 before the scores and pieces, which the join reads back (131072 slots with
  // weights 93 us, with the usual policy 98; 16 ragged requests 48 and 51; the largest batch 159 and 157)
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  // ---- this warp's loads.  look() fetches the page of each row of the next chunk, load() copies the rows
  const int my_row = lane % CT;  // the row of a chunk whose place this lane works out
  Cursor lc{0, 0, 0, 0, 0, 0};
  int lx = w0;
  struct Look {
    int64_t head;  // element offset of the KV head
    int32_t page, in_page;
    bool chunk, row;  // there is a chunk (the same in all lanes), and this lane's row of it
    uint8_t seen;     // kDense: the row's entry of the mask (looked at when the row is copied, an iteration later)
  };
  auto look = [&]() {
    Look k{0, -1, 0, lx < w1, false, 1};
    if (k.chunk) {
      if (lx >= lc.end) seek(lc, P, plan, lx);
      const int t = (lx - lc.first) * CT + my_row;
      k.row = t < lc.len;
      if (k.row) {
        if constexpr (SRC == kDense) {
          k.page = lc.b;
          k.in_page = t;
          if (P.mask) k.seen = __ldg(P.mask + lc.b * P.mask_stride + t);
        } else {
          const uint32_t pg = page_of(P.pages, static_cast<uint32_t>(t));
          k.in_page = t - pg * P.pages.page_size;
          if (SRC == kShared && lc.b < kMaxReq)
            k.page = __ldg(P.prefix_table + static_cast<int64_t>(lc.b) * P.prefix_max_pages + pg);
          else
            k.page = __ldg(P.pages.table + static_cast<int64_t>(lc.b - (SRC == kShared ? kMaxReq : 0)) * P.pages.max_pages + pg);
        }
      }
      k.head = static_cast<int64_t>(lc.h) * P.pages.head_stride;
      ++lx;
    }
    return k;
  };
  // (kDense) which rows of a chunk count: of the next chunk to be used, and the one behind it
  uint32_t seen0 = 0, seen1 = 0;
  auto load = [&](int stage, const Look& k) {
    if constexpr (SRC == kDense) {
      seen0 = seen1;
      seen1 = __ballot_sync(0xffffffffu, k.row && k.seen);
    }
    if (k.chunk) {
      int64_t off = -1;
      if (k.row && (SRC != kDense || k.seen)) {
        off = slot_offset(P.pages, k.page, k.in_page);
        if (off < 0) atomicOr(P.pages.status, kErrInput);
        else off += k.head;
        if (off >= 0 && !in_bounds(static_cast<const T*>(P.pages.k) + off, D, static_cast<const T*>(P.pages.k),
                                   P.pages.extent, P.pages.status, kSitePool))
          off = -1;
      }
      const uint32_t dst = stage0 + stage * (2 * kChunkBytes);
      const int piece = lane % PIECES;
#pragma unroll
      for (int i = 0; i < CT / RPI; ++i) {
        const int r = i * RPI + lane / PIECES;
        const int64_t ro = __shfl_sync(0xffffffffu, off, r);
        const int bytes = ro >= 0 ? 16 : 0;  // 0: the 16 bytes become zero
        const int64_t e = (ro >= 0 ? ro : 0) + piece * 8;
        const uint32_t at = dst + r * (2 * D) + ((piece ^ (r & 7)) << 4);
        cp16(at, static_cast<const T*>(P.pages.k) + e, bytes, policy);
        cp16(at + kChunkBytes, static_cast<const T*>(P.pages.v) + e, bytes, policy);
      }
    }
    cp_commit();
  };
  const int g = lane >> 2, c2 = (lane & 3) * 2;
  Cursor cc{0, 0, 0, 0, 0, 0};
  // q fragments of an item: rows g and (WIDE) g + 8
  uint32_t qa[KS][WIDE ? 4 : 2];
  auto load_q = [&]() {
    const int rows = item_rows(P, plan, cc.b, cc.blk);
    const T* q0 = static_cast<const T*>(P.q) + q_at<SRC, D>(P, plan, cc.b, cc.h, cc.blk, g) + c2;
    const T* q8 = q0 + 8 * D;
    if constexpr (SRC != kPaged && WIDE) q8 = static_cast<const T*>(P.q) + q_at<SRC, D>(P, plan, cc.b, cc.h, cc.blk, g + 8) + c2;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      qa[k][0] = g < rows ? __ldg(reinterpret_cast<const uint32_t*>(q0 + k * 16)) : 0u;
      qa[k][1] = g < rows ? __ldg(reinterpret_cast<const uint32_t*>(q0 + k * 16 + 8)) : 0u;
      if constexpr (WIDE) {
        qa[k][2] = g + 8 < rows ? __ldg(reinterpret_cast<const uint32_t*>(q8 + k * 16)) : 0u;
        qa[k][3] = g + 8 < rows ? __ldg(reinterpret_cast<const uint32_t*>(q8 + k * 16 + 8)) : 0u;
      }
    }
  };
  // pages are looked up two chunks ahead; the first two chunks' and the first q are fetched together
  Look next = look(), after = look();
  if (w0 < w1) {
    seek(cc, P, plan, w0);
    load_q();
  }
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) {
    load(i, next);
    next = after;
    after = look();
  }

  // ---- the parts of items in this warp's range
  int stage = 0;
  int cx = w0;  // the next chunk
  while (cx < w1) {
    const Cursor it = cc;
    const int seg_end = min(it.end, w1);
    const bool whole = it.first == cx && it.end <= w1;
    const int rows = item_rows(P, plan, it.b, it.blk);
    const int64_t row0 = static_cast<int64_t>(it.b) * P.n_q + it.h * P.group + it.blk * kRowsMax;  // (with scores)
    constexpr int H = WIDE ? 2 : 1;
    float m[H], l[H], acc[NO][4];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      m[h] = kNegInf;
      l[h] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < NO; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;

    for (; cx < seg_end; ++cx) {
      cp_wait<kStages - 2>();
      __syncwarp();  // every lane's copies of this chunk are here, and every lane is done with the last one
      const uint32_t seen = seen0;
      load(stage == 0 ? kStages - 1 : stage - 1, next);
      next = after;
      after = look();
      const uint32_t kb = stage0 + stage * (2 * kChunkBytes), vb = kb + kChunkBytes;
      stage = stage == kStages - 1 ? 0 : stage + 1;

      float sc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          // matrices: slots n*8.. x dims lo, same x dims hi, slots n*8+8.. x dims lo, x dims hi
          const int r = n * 8 + (lane & 7) + ((lane >> 4) << 3);
          const int piece = 2 * k + ((lane >> 3) & 1);
          uint32_t kf[4];
          ldsm4(kf, kb + r * (2 * D) + ((piece ^ (r & 7)) << 4));
          if constexpr (WIDE) {
            Mma<T>::go(sc[n], qa[k][0], qa[k][2], qa[k][1], qa[k][3], kf[0], kf[1]);
            Mma<T>::go(sc[n + 1], qa[k][0], qa[k][2], qa[k][1], qa[k][3], kf[2], kf[3]);
          } else {
            Mma<T>::go(sc[n], qa[k][0], 0u, qa[k][1], 0u, kf[0], kf[1]);
            Mma<T>::go(sc[n + 1], qa[k][0], 0u, qa[k][1], 0u, kf[2], kf[3]);
          }
        }
      }
      const int t0 = (cx - it.first) * CT;
      const int left = it.len - t0;
      float top[H];
#pragma unroll
      for (int h = 0; h < H; ++h) top[h] = kNegInf;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& v = sc[n][2 * h + e];
            v = (SRC == kDense ? (seen >> (n * 8 + c2 + e) & 1u) != 0 : n * 8 + c2 + e < left) ? v * P.scale : kNegInf;
            top[h] = fmaxf(top[h], v);
          }
      if constexpr (SCORES) {
#pragma unroll
        for (int h = 0; h < H; ++h)
          if (g + 8 * h < rows) {
            float* dst = P.scores + (row0 + g + 8 * h) * P.score_stride + t0 + c2;
#pragma unroll
            for (int n = 0; n < NT; ++n)
              *reinterpret_cast<float2*>(dst + n * 8) = make_float2(sc[n][2 * h], sc[n][2 * h + 1]);
          }
      }
      bool up = top[0] > m[0] + (kTau + Mma<T>::kLift);
      if constexpr (WIDE) up = up || top[1] > m[1] + (kTau + Mma<T>::kLift);
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          float t = fmaxf(top[h] - Mma<T>::kLift, m[h]);
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
          const float al = t == kNegInf ? 1.f : ex2(m[h] - t);
          m[h] = t;
          l[h] *= al;
#pragma unroll
          for (int i = 0; i < NO; ++i) {
            acc[i][2 * h] *= al;
            acc[i][2 * h + 1] *= al;
            if constexpr (!WIDE) {  // the upper rows hold the remainders of the same heads
              acc[i][2] *= al;
              acc[i][3] *= al;
            }
          }
        }
      }
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const float base = m[h] == kNegInf ? 0.f : m[h];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            sc[n][2 * h + e] = ex2(sc[n][2 * h + e] - base);
            l[h] += sc[n][2 * h + e];
          }
      }
#pragma unroll
      for (int n = 0; n < NT; n += 2) {  // 16 slots at a time
        uint32_t hi[2][H], lo[2][H];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int h = 0; h < H; ++h) Mma<T>::split(sc[n + u][2 * h], sc[n + u][2 * h + 1], hi[u][h], lo[u][h]);
#pragma unroll
        for (int i = 0; i < NO; i += 2) {
          const int r = n * 8 + (lane & 15);
          const int piece = i + (lane >> 4);
          uint32_t vf[4];
          ldsm4t(vf, vb + r * (2 * D) + ((piece ^ (r & 7)) << 4));
          if constexpr (WIDE) {
            Mma<T>::go(acc[i], hi[0][0], hi[0][1], hi[1][0], hi[1][1], vf[0], vf[1]);
            Mma<T>::go(acc[i + 1], hi[0][0], hi[0][1], hi[1][0], hi[1][1], vf[2], vf[3]);
            Mma<T>::go(acc[i], lo[0][0], lo[0][1], lo[1][0], lo[1][1], vf[0], vf[1]);
            Mma<T>::go(acc[i + 1], lo[0][0], lo[0][1], lo[1][0], lo[1][1], vf[2], vf[3]);
          } else {
            Mma<T>::go(acc[i], hi[0][0], lo[0][0], hi[1][0], lo[1][0], vf[0], vf[1]);
            Mma<T>::go(acc[i + 1], hi[0][0], lo[0][0], hi[1][0], lo[1][0], vf[2], vf[3]);
          }
        }
      }
    }

    // ---- the end of the item, or of the warp's range
    if (seg_end < w1) {  // the next item's q is on its way meanwhile
      seek(cc, P, plan, seg_end);
      load_q();
    }
#pragma unroll
    for (int h = 0; h < H; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    if constexpr (!WIDE) {
#pragma unroll
      for (int i = 0; i < NO; ++i) {
        acc[i][0] += acc[i][2];
        acc[i][1] += acc[i][3];
      }
    }
    if (whole) {
#pragma unroll
      for (int h = 0; h < H; ++h) {
        if (g + 8 * h >= rows) continue;
        const RowOut at = place<SRC, D>(P, plan, it.b, it.h, it.blk, g + 8 * h);
        if constexpr (SRC == kShared) {
          const int64_t row = at.lse + (it.b < kMaxReq ? 0 : static_cast<int64_t>(P.pages.n_req) * P.n_q);
#pragma unroll
          for (int i = 0; i < NO; ++i)
            *reinterpret_cast<float2*>(P.state_o + row * D + i * 8 + c2) = make_float2(acc[i][2 * h], acc[i][2 * h + 1]);
          if ((lane & 3) == 0) P.state_ml[row] = make_float2(m[h], l[h]);
          continue;
        }
        const float inv = l[h] == 0.f ? 0.f : 1.f / l[h];
        uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(P.o) + at.o + c2);
#pragma unroll
        for (int i = 0; i < NO; ++i)
          dst[i * 4] = l[h] == 0.f ? 0u : Mma<T>::down2(acc[i][2 * h] * inv, acc[i][2 * h + 1] * inv);
        if ((lane & 3) == 0) {
          if (SRC != kDense || P.lse) P.lse[at.lse] = l[h] == 0.f ? kNegInf : (m[h] + log2f(l[h])) * kLn2;
          if constexpr (SCORES) P.row_ml[at.lse] = make_float2(m[h], l[h]);
        }
      }
      continue;
    }
    const bool tail = seg_end == w1;
    float* po;
    float2* pml;
    if (tail) {  // every chunk has been read: the stages are free
      cp_wait<0>();
      __syncwarp();
      po = reinterpret_cast<float*>(smem + warp * S::RING);
      pml = reinterpret_cast<float2*>(po + kRowsMax * D);
    } else {
      po = P.lead + (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kRowsMax * D;
      pml = P.lead_ml + (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kRowsMax;
    }
#pragma unroll
    for (int h = 0; h < H; ++h) {
      if (g + 8 * h >= rows) continue;
      if ((lane & 3) == 0) pml[g + 8 * h] = make_float2(m[h], l[h]);
#pragma unroll
      for (int i = 0; i < NO; ++i)
        *reinterpret_cast<float2*>(po + S::at(g + 8 * h, i * 8 + c2)) = make_float2(acc[i][2 * h], acc[i][2 * h + 1]);
    }
    if (lane == 0) pieces[tail ? kWarps + warp : warp] = Piece{it.first, it.end, it.b, it.h, it.blk};
  }
  cp_wait<0>();
  __syncthreads();

  // ---- the items that have pieces here: lane p < 16 looks at piece p (leads, then tails) and names its item, if no
  // lower one has.  An item has tails in any number of warps and a lead in one at most.
  uint32_t named;
  {
    const int f = lane < 2 * kWarps ? pieces[lane].first : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, f);  // by all lanes
    named = __ballot_sync(0xffffffffu, f >= 0 && (same & ((1u << lane) - 1u)) == 0);
  }
  const int per_item = (SRC == kShared ? kRowsMax : min(SRC == kDense ? P.rows : P.group, kRowsMax)) * (D / 4);
  for (int i = tid; i < __popc(named) * per_item; i += kWarps * 32) {
    const int nth = i / per_item, e = i - nth * per_item;
    const int r = e / (D / 4), d4 = (e - r * (D / 4)) * 4;
    uint32_t which = named;
    for (int k = 0; k < nth; ++k) which &= which - 1u;
    const Piece it = pieces[__ffs(which) - 1];
    if (r >= item_rows(P, plan, it.b, it.blk)) continue;
    int lead = -1;
    float2 ml[kWarps + 1];
    float M = kNegInf;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (pieces[w].first == it.first) lead = w;
      ml[w] = make_float2(kNegInf, 0.f);
      if (pieces[kWarps + w].first == it.first)
        ml[w] = reinterpret_cast<const float2*>(smem + w * S::RING + kRowsMax * D * 4)[r];
      M = fmaxf(M, ml[w].x);
    }
    const int64_t at_lead = (static_cast<int64_t>(blockIdx.x) * kWarps + lead) * kRowsMax;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    ml[kWarps] = make_float2(kNegInf, 0.f);
    if (lead >= 0) {
      ml[kWarps] = P.lead_ml[at_lead + r];
      o = *reinterpret_cast<const float4*>(P.lead + at_lead * D + S::at(r, d4));
    }
    M = fmaxf(M, ml[kWarps].x);
    const float base = M == kNegInf ? 0.f : M;
    float f = ex2(ml[kWarps].x - base);
    float L = ml[kWarps].y * f;
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (pieces[kWarps + w].first != it.first) continue;
      const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + w * S::RING) + S::at(r, d4));
      f = ex2(ml[w].x - base);
      L = fmaf(ml[w].y, f, L);
      o.x = fmaf(v.x, f, o.x);
      o.y = fmaf(v.y, f, o.y);
      o.z = fmaf(v.z, f, o.z);
      o.w = fmaf(v.w, f, o.w);
    }
    if (it.first >= x0 && it.end <= x1) {
      const RowOut at = place<SRC, D>(P, plan, it.b, it.h, it.blk, r);
      if constexpr (SRC == kShared) {
        const int64_t row = at.lse + (it.b < kMaxReq ? 0 : static_cast<int64_t>(P.pages.n_req) * P.n_q);
        *reinterpret_cast<float4*>(P.state_o + row * D + d4) = o;
        if (d4 == 0) P.state_ml[row] = make_float2(M, L);
        continue;
      }
      write_row<T>(P, at, d4, M, L, o);
      if (SCORES && d4 == 0) P.row_ml[at.lse] = make_float2(M, L);
    } else {
      const int64_t slot = (static_cast<int64_t>(blockIdx.x) * 2 + (it.first >= x0 ? 1 : 0)) * kRowsMax + r;
      *reinterpret_cast<float4*>(P.part_o + slot * D + d4) = o;
      if (d4 == 0) P.part_ml[slot] = make_float2(M, L);
    }
  }
  if constexpr (SRC != kShared) write_empty<T, SRC, D>(P, plan);
}

// Merges the pieces of the items that more than one CTA worked on, and adds the weights.  CTA (x, y): KV head x of all
// requests' heads; block of query heads y, and slots [2048 y, 2048 (y + 1)):
// acc_out[t] = acc_in[t] + sum over the KV head's query heads of 2^(s_t - m) / l, from the stored scores.
constexpr int kMaxCtas = 256;
constexpr int kWeightSlots = 2048;
constexpr int kQuads = kWeightSlots / (4 * kWarps * 32);  // of slots, to a thread

template <typename T, int SRC, int D, bool SCORES>
__global__ void __launch_bounds__(kWarps * 32) join_kernel(const __grid_constant__ AttendParams P) {
  constexpr int CT = kChunkBytes / (2 * D);
  __shared__ Plan<SRC> plan;
  __shared__ float s_f[kMaxCtas * kRowsMax];  // a piece's factor for each row
  __shared__ float2 s_ml[kRowsMax];
  __shared__ float4 s_o[kWarps * 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // The lengths are not the attention kernel's work, and that kernel has waited for whoever wrote them before it let this
  // one start: the plan, and where the pieces lie, need not wait for it.
  const int T_all = build_plan<SRC, CT>(P, plan, false);
  const int b = blockIdx.x / P.pages.n_kv_heads, h = blockIdx.x - b * P.pages.n_kv_heads;
  const int n = plan.n[b], len = plan.len[b];
  const int t_first = blockIdx.y * kWeightSlots + tid * 4;  // this thread's slots: 4 here and 4 behind each 1024 more
  const bool weigh = SCORES && static_cast<int>(blockIdx.y) * kWeightSlots < len;
  const bool idle = n == 0 || (!weigh && static_cast<int>(blockIdx.y) >= P.blocks);
  const Split split(P, T_all);
  float4 w[kQuads], before[kQuads];  // the weights, and acc_in
#pragma unroll
  for (int u = 0; u < kQuads; ++u) w[u] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int64_t at_acc = static_cast<int64_t>(blockIdx.x) * P.pages.cap + t_first;
  bool waited = false;
  for (int blk = weigh ? 0 : blockIdx.y; !idle && blk < (weigh ? P.blocks : static_cast<int>(blockIdx.y) + 1); ++blk) {
    const bool merge = static_cast<int>(blockIdx.y) == blk;
    const int first = plan.first[b] + (h * P.blocks + blk) * n;
    const int c0 = split.of(first), c1 = split.of(first + n - 1);
    const int pieces = c1 - c0 + 1;
    if (pieces == 1 && !weigh) continue;
    const int rows = item_rows(P, plan, b, blk);
    const int64_t row0 = static_cast<int64_t>(b) * P.n_q + h * P.group + blk * kRowsMax;  // (kPaged)
    // piece c lies in slot 0 of its CTA, but the first in slot 1 if the item begins in that CTA's range
    const int64_t slot0 = static_cast<int64_t>(c0 * 2 + (split.begin(c0) <= first ? 1 : 0)) * kRowsMax;
    auto slot = [&](int c) { return c == 0 ? slot0 : static_cast<int64_t>(c0 + c) * 2 * kRowsMax; };
    // the outputs over the threads: several share one where there are more of them than outputs
    const int outs = rows * (D / 4), share = max(kWarps * 32 / outs, 1);
    const int part = share > 1 ? tid / outs : 0;
    int i = share > 1 ? tid - part * outs : tid;
    auto piece_o = [&](int c) {
      return __ldcg(reinterpret_cast<const float4*>(P.part_o + (slot(c) + i / (D / 4)) * D + (i % (D / 4)) * 4));
    };
    if (!waited) {
      grid_dependency_wait();
      allow_dependents();
      waited = true;
      if (weigh) {
#pragma unroll
        for (int u = 0; u < kQuads; ++u) {
          const int left = len - t_first - u * 1024;
          const float* a = P.acc_in + at_acc + u * 1024;
          before[u] = make_float4(left > 0 ? a[0] : 0.f, left > 1 ? a[1] : 0.f, left > 2 ? a[2] : 0.f, left > 3 ? a[3] : 0.f);
        }
      }
    }
    // this thread's first pieces are fetched along with the states
    constexpr int kAhead = 4;
    float4 v[kAhead];
    const bool mine = merge && pieces > 1 && i < outs && part < share;
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (mine && part + u * share < pieces) v[u] = piece_o(part + u * share);
    for (int r = warp; r < rows; r += kWarps) {
      if (pieces == 1) {
        if (lane == 0) s_ml[r] = P.row_ml[row0 + r];
        continue;
      }
      float2 ml = lane < pieces ? __ldcg(&P.part_ml[slot(lane) + r]) : make_float2(kNegInf, 0.f);
      float M = ml.x;
      for (int c = lane + 32; c < pieces; c += 32) M = fmaxf(M, __ldcg(&P.part_ml[slot(c) + r]).x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float base = M == kNegInf ? 0.f : M;
      float L = 0.f;
      for (int c = lane; c < pieces; c += 32) {
        if (c != lane) ml = __ldcg(&P.part_ml[slot(c) + r]);
        const float f = ex2(ml.x - base);
        s_f[c * kRowsMax + r] = f;
        L = fmaf(ml.y, f, L);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
      if (lane == 0) s_ml[r] = make_float2(M, L);
    }
    __syncthreads();
    if (merge && pieces > 1) {
      for (bool again = false;; again = true) {  // (once, unless there are more outputs than threads)
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < outs && part < share) {
          const int r = i / (D / 4);
          auto add = [&](const float4& x, int c) {
            const float f = s_f[c * kRowsMax + r];
            o.x = fmaf(x.x, f, o.x);
            o.y = fmaf(x.y, f, o.y);
            o.z = fmaf(x.z, f, o.z);
            o.w = fmaf(x.w, f, o.w);
          };
          int c = part;
          if (!again) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u, c += share)
              if (c < pieces) add(v[u], c);
          }
#pragma unroll 4
          for (; c < pieces; c += share) add(piece_o(c), c);
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
        if (i < outs && part == 0) {
          const int r = i / (D / 4);
          // (worked out anew from b, h and blk here: 5 requests of 28 / 4 heads 11.7 us, of 48 / 4 16.5; from row0 11.1 and 14.9)
          const RowOut at = SRC == kPaged ? RowOut{(row0 + r) * D, row0 + r} : place<SRC, D>(P, plan, b, h, blk, r);
          write_row<T>(P, at, (i - r * (D / 4)) * 4, s_ml[r].x, s_ml[r].y, o);
        }
        if (share > 1 || i + kWarps * 32 - tid >= outs) break;  // the same for all threads
        i += kWarps * 32;
      }
    }
    if (weigh) {
      constexpr int kRowsAtOnce = 4;
      for (int r0 = 0; r0 < rows; r0 += kRowsAtOnce) {
        float4 sc[kRowsAtOnce][kQuads];
#pragma unroll
        for (int q = 0; q < kRowsAtOnce; ++q)
#pragma unroll
          for (int u = 0; u < kQuads; ++u) {
            sc[q][u] = make_float4(kNegInf, kNegInf, kNegInf, kNegInf);
            if (r0 + q < rows && t_first + u * 1024 < len)
              sc[q][u] = __ldcg(reinterpret_cast<const float4*>(P.scores + (row0 + r0 + q) * P.score_stride + t_first + u * 1024));
          }
#pragma unroll
        for (int q = 0; q < kRowsAtOnce; ++q) {
          const float2 ml = r0 + q < rows ? s_ml[r0 + q] : make_float2(0.f, 0.f);
          if (ml.y == 0.f) continue;  // only scores of -inf: no weight
          const float inv = 1.f / ml.y;
#pragma unroll
          for (int u = 0; u < kQuads; ++u) {
            w[u].x = fmaf(ex2(sc[q][u].x - ml.x), inv, w[u].x);
            w[u].y = fmaf(ex2(sc[q][u].y - ml.x), inv, w[u].y);
            w[u].z = fmaf(ex2(sc[q][u].z - ml.x), inv, w[u].z);
            w[u].w = fmaf(ex2(sc[q][u].w - ml.x), inv, w[u].w);
          }
        }
      }
    }
    __syncthreads();
  }
  if (!waited) {  // every CTA waits: the next kernel relies on this one's end for all that came before
    grid_dependency_wait();
    allow_dependents();
  }
  if (idle || !weigh) return;
#pragma unroll
  for (int u = 0; u < kQuads; ++u) {
    const float v[4] = {before[u].x + w[u].x, before[u].y + w[u].y, before[u].z + w[u].z, before[u].w + w[u].w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (t_first + u * 1024 + e < len) P.acc_out[at_acc + u * 1024 + e] = v[e];
  }
}


// ------------------------------------------------------------------ host

constexpr int64_t kWholeItem = 32;  // chunks

struct Sizes {
  int32_t max_len, blocks, ctas;
  bool whole;  // no item is split over CTAs, whatever the lengths
  int64_t score_stride;
  size_t part_o, part_ml, lead, lead_ml, row_ml, scores, state_o, state_ml, total;
};

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// CTAs for `chunks` chunks, and where their pieces lie in a workspace; z->total: the bytes.
inline void size_pieces(Sizes* z, int64_t chunks, int head_dim, int sms) {
  z->ctas = static_cast<int32_t>(std::min<int64_t>(std::min(sms, kMaxCtas), std::max<int64_t>((chunks + kMinChunks - 1) / kMinChunks, 1)));
  z->part_o = 0;
  z->part_ml = z->part_o + up256(static_cast<size_t>(z->ctas) * 2 * kRowsMax * head_dim * 4);
  z->lead = z->part_ml + up256(static_cast<size_t>(z->ctas) * 2 * kRowsMax * 8);
  z->lead_ml = z->lead + up256(static_cast<size_t>(z->ctas) * kWarps * kRowsMax * head_dim * 4);
  z->total = z->lead_ml + up256(static_cast<size_t>(z->ctas) * kWarps * kRowsMax * 8);
}

inline void place_pieces(AttendParams& p, const Sizes& z, char* ws) {
  p.part_o = reinterpret_cast<float*>(ws + z.part_o);
  p.part_ml = reinterpret_cast<float2*>(ws + z.part_ml);
  p.lead = reinterpret_cast<float*>(ws + z.lead);
  p.lead_ml = reinterpret_cast<float2*>(ws + z.lead_ml);
  p.max_len = z.max_len;
  p.blocks = z.blocks;
  p.whole = z.whole;
  p.ctas = z.ctas;
}

// The softmax scale in log2 units; 0 given: 1 / sqrt(head_dim).  False: not positive, or not finite in those units.
inline bool log2_scale(float scale, int head_dim, float* out) {
  const double sc = scale > 0.f ? static_cast<double>(scale) : 1.0 / sqrt(static_cast<double>(head_dim));
  const double x = sc * 1.4426950408889634074;
  *out = static_cast<float>(x);
  return scale >= 0.f && x <= FLT_MAX;
}

template <typename T, int SRC, int D, bool WIDE, bool SCORES>
cudaError_t launch_attend(const AttendParams& p, int device, cudaStream_t s) {
  constexpr int bytes = Smem<D>::BYTES;
  // set on each device's first use; setting it twice is harmless
  static std::atomic<bool> done[64];
  if (device >= 64 || !done[device].load(std::memory_order_acquire)) {
    const cudaError_t e =
        cudaFuncSetAttribute(attend_kernel<T, SRC, D, WIDE, SCORES>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (device < 64) done[device].store(true, std::memory_order_release);
  }
  return launch_pdl(attend_kernel<T, SRC, D, WIDE, SCORES>, dim3(p.ctas), dim3(kWarps * 32), bytes, s, p);
}

}  // namespace
}  // namespace svx
