// Attention of many rows to the same keys on the 5th-generation tensor cores: the rows of a prefix (the query heads of all its
// requests, svx_paged_decode_shared) or of an encoder's states (query heads times tokens, svx_cross_attn).
//
//   S = Q K^T,  P = 2^(S scale - m) by row,  O += P V,  l += sum P,   O and (m, l) of a row merged or finished at the end
//
// Work.  An item is up to 256 rows of one sequence and KV head; its keys are cut into tiles of 128.  All items' tiles form one flat range,
// cut evenly over the CTAs (one an SM); the part of an item in a CTA's range is a segment.  An item that lies in one CTA is
// finished there; of the others each CTA leaves (m, l, O) in its slot 0 (the item began before the CTA's range) or 1.
//
// A CTA.  Two streams of products alternate, so that the tensor cores work on one while the softmax works on the other:
// with more than 128 rows, stream s has rows 128 s .. and both take every tile; else both have the same rows, stream s takes the
// tiles of its parity, and their states are merged at the end.
//   S = Q K^T       M = 128 rows, N = 128 keys, both operands in shared memory (K-major); fp32 in tensor memory
//   P               128 threads, one a row: read from tensor memory, exponentials, rounded, written over S in tensor memory
//   O += P V        M = 128 rows, N = D, K = 128 keys: P from tensor memory, V from shared memory as it lies (MN-major)
//   warps 0-3, 4-7  softmax of stream 0 and 1, and the segment's end
//   warp 8          issues the products (one thread)
//   warps 9, 10     bring K and V tiles in (16-byte cp.async, rows found through the page table or by stride)
//   warp 11         brings Q in
// Up to 128 rows the tensor cores have time to spare (the bytes of K and V bound the time), and P enters the product in two 16-bit pieces:
// O is then as exact as with fp32 weights.  With more rows the products bound the time, and P is rounded once.
//
// Every wait is bounded (2 s of global time): one that gives up raises the status word and makes all roles stop, drain and leave.
#pragma once

#include "svx_attend.cuh"

#include <type_traits>

namespace svx {
namespace {

constexpr int kRowTile = 128;
constexpr int kTile = 128;                   // keys
constexpr uint32_t kHalf = kTile * 128;      // bytes of 64 dimensions of 128 rows (an operand's swizzle atoms: 8 rows of 128 bytes)
constexpr uint64_t kWaitLimit = 2000000000ull;
constexpr int kRowThreads = 384;

// QT: row tiles of an item, 1 or 2.
template <int D, int QT>
struct RowsCfg {
  static constexpr uint32_t TILE = kTile * D * 2;  // K or V
  // with one row tile the bytes in flight decide: 5 tiles of 32 KiB (d = 128), 9 of 16 KiB (d = 64)
  static constexpr int KST = D == 128 ? 2 : 4;
  static constexpr int VST = D == 128 ? 4 - QT : 5;
  static constexpr uint32_t Q_TILE = kRowTile * D * 2;
  static constexpr uint32_t OFF_K = 0;
  static constexpr uint32_t OFF_V = OFF_K + KST * TILE;
  static constexpr uint32_t OFF_Q = OFF_V + VST * TILE;
  static constexpr uint32_t OFF_ML = OFF_Q + QT * Q_TILE;  // float2 [2][128]: the streams' states at a segment's end
  static constexpr int N_BAR = 2 * KST + 2 * VST + 2 + 2 + 2 + 2 + 1 + 1;
  static constexpr uint32_t OFF_BAR = OFF_ML + 2 * kRowTile * 8;
  static constexpr uint32_t OFF_MISC = OFF_BAR + N_BAR * 8;  // [0] TMEM base, [1] abort flag
  static constexpr uint32_t BYTES = OFF_MISC + 16;
  static constexpr uint32_t SMEM = BYTES + 1024;  // slack to align the base to 1024 bytes
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t O_COL = 256;  // S (and P over it): 128 columns a stream; O: D a stream
  static_assert(SMEM + 5 * 1024 <= 232448, "shared memory per CTA, with the plan");
};

// ------------------------------------------------------------------ PTX

__device__ __forceinline__ uint32_t smem_at(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// this thread's copies so far, once they are in, arrive on the barrier
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Named barrier 1 of the softmax threads, which also ANDs their flags: a wait that gave up in one stops all of them.
__device__ __forceinline__ bool softmax_sync(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(ok))
      : "memory");
  return r != 0;
}
// D = A B (+ D), operands as the low words of shared-memory descriptors (the high word is the same for all).
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}
// The same with A in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// 32 columns of this warp's 32 lanes (a thread: its lane); the wait is in the same statement, so that no value is used early.
template <int OFF, int N>
__device__ __forceinline__ void tmem_read32(uint32_t at, float (&v)[N]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[OFF + i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_write32(uint32_t at, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]),
      "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]),
      "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_write16(uint32_t at, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_written() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Instruction descriptor of tcgen05.mma kind::f16: 16-bit A and B of one type, fp32 D, M = 128.
template <typename T>
constexpr uint32_t rows_idesc(int N, bool b_mn_major) {
  constexpr uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return (1u << 4) | (type << 7) | (type << 10) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(kRowTile >> 4) << 24);
}
// Shared-memory descriptor, 128-byte swizzle: high word (stride between groups of 8 rows 1024 bytes, version, swizzle mode), low word
// (address, leading-dimension offset).
constexpr uint32_t kRowsDescHi = (1024u >> 4) | (1u << (46 - 32)) | (2u << (61 - 32));
__device__ __forceinline__ uint32_t desc_of(uint32_t addr, uint32_t lead) {
  return ((addr >> 4) & 0x3FFFu) | (((lead >> 4) & 0x3FFFu) << 16);
}

// ------------------------------------------------------------------ the flat range

// As Plan, of items of up to P.item_rows rows and tiles of kTile keys.  Sequences: the requests, or (kShared) the prefixes.
struct RowPlan {
  int32_t first[kMaxReq + 1];
  int32_t warp_sum[kWarps];
  int32_t n[kMaxReq];
  int32_t len[kMaxReq];
  int32_t req0[kMaxReq + 1];
};

template <int SRC>
__device__ __forceinline__ int row_rows(const AttendParams& P, const RowPlan& s, int b) {
  return SRC == kShared ? (s.req0[b + 1] - s.req0[b]) * P.group : P.rows;
}

template <int SRC>
__device__ __forceinline__ int build_row_plan(const AttendParams& P, RowPlan& s, bool report) {
  const int t = threadIdx.x;
  int* const status = report ? P.pages.status : nullptr;
  if constexpr (SRC == kShared) prefix_requests(P.first, P.n_prefix, P.pages.n_req, s.req0, s.warp_sum, status);
  int n = 0, rows = 0;
  if (t < (SRC == kShared ? P.n_prefix : P.pages.n_req)) {
    const int most = SRC == kShared ? P.max_prefix : P.max_len;
    const int raw = SRC == kShared ? P.prefix_len[t] : P.len ? P.len[t] : most;
    n = min(max(raw, 0), most);
    if (status && n != raw) atomicOr(status, kErrInput);
    rows = row_rows<SRC>(P, s, t);
  }
  const int tiles = rows ? static_cast<int>((static_cast<uint32_t>(n) + (kTile - 1)) / kTile) : 0;
  const int mine = P.pages.n_kv_heads * ((rows + P.item_rows - 1) / P.item_rows) * tiles;
  int total;
  const int upto = block_scan(mine, s.warp_sum, total);
  if (t < kMaxReq) {
    s.n[t] = tiles;
    s.len[t] = n;
    s.first[t] = upto - mine;
  }
  if (t == 0) s.first[kMaxReq] = total;
  __syncthreads();
  return total;
}

// The T tiles over the CTAs, as Split, but a CTA takes at least P.min_tiles.
struct RowSplit {
  uint32_t used, q, r, total;
  __device__ __forceinline__ RowSplit(const AttendParams& P, int T) {
    total = T;
    used = min((total + P.min_tiles - 1) / P.min_tiles, static_cast<uint32_t>(P.row_ctas));
    q = used ? total / used : 0;
    r = total - q * used;
  }
  __device__ __forceinline__ int begin(uint32_t c) const { return used ? static_cast<int>(c * q + c * r / used) : 0; }
  __device__ __forceinline__ int of(int x) const {
    int c = min(static_cast<int>(static_cast<float>(x) * (static_cast<float>(used) / static_cast<float>(total))),
                static_cast<int>(used) - 1);
    while (c + 1 < static_cast<int>(used) && begin(c + 1) <= x) ++c;
    while (c > 0 && begin(c) > x) --c;
    return c;
  }
};

// The segment of a CTA that begins at x: its item, and the tiles [tile0, tile0 + n) of it.
struct RowSeg {
  int b, h, rt;         // sequence, KV head, block of item_rows rows
  int rows;             // of the block
  int len;              // keys of the sequence
  int tile0, n;
  int first, end;       // the item's tiles in the flat range
};

// (all lanes of a warp alike)
template <int SRC>
__device__ __forceinline__ RowSeg row_seg(const AttendParams& P, const RowPlan& s, int x, int x1) {
  const int seqs = SRC == kShared ? P.n_prefix : P.pages.n_req;
  RowSeg g;
  g.b = 0;
  for (int i = 0; i < seqs; i += 32) {
    const int r = i + (threadIdx.x & 31);
    g.b += __popc(__ballot_sync(0xffffffffu, r < seqs && s.first[r + 1] <= x));
  }
  const int n = s.n[g.b], rows = row_rows<SRC>(P, s, g.b), blocks = (rows + P.item_rows - 1) / P.item_rows;
  const int i = (x - s.first[g.b]) / n;
  g.h = i / blocks;
  g.rt = i - g.h * blocks;
  g.rows = min(rows - g.rt * P.item_rows, P.item_rows);
  g.len = s.len[g.b];
  g.first = s.first[g.b] + i * n;
  g.end = g.first + n;
  g.tile0 = x - g.first;
  g.n = min(g.end, x1) - x;
  return g;
}

// Element offset of row r of a segment's block in q, and the places of its outputs.
template <int SRC, int D>
__device__ __forceinline__ int64_t row_q(const AttendParams& P, const RowPlan& s, const RowSeg& g, int r) {
  r += g.rt * P.item_rows;
  const int j = r / P.group, head = g.h * P.group + (r - j * P.group);
  if constexpr (SRC == kShared) return (static_cast<int64_t>(s.req0[g.b] + j) * P.n_q + head) * D;
  return g.b * P.q_b + head * P.q_h + j * P.q_n;
}
template <int SRC, int D>
__device__ __forceinline__ RowOut row_out(const AttendParams& P, const RowPlan& s, const RowSeg& g, int r) {
  r += g.rt * P.item_rows;
  const int j = r / P.group, head = g.h * P.group + (r - j * P.group);
  if constexpr (SRC == kShared) {
    const int64_t row = static_cast<int64_t>(s.req0[g.b] + j) * P.n_q + head;
    return RowOut{row * D, row};
  }
  return RowOut{g.b * P.o_b + head * P.o_h + j * P.o_n, (static_cast<int64_t>(g.b) * P.n_q + head) * P.n_tok + j};
}

struct RowWaiter {
  volatile uint32_t* abort;
  int* status;
  __device__ __forceinline__ void give_up() {
    *abort = 1u;
    if (status) atomicOr(status, kErrWait);
  }
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) {
    if (bar_try(bar, parity)) return true;
    const uint64_t t0 = now_ns();
    for (uint32_t it = 1;; ++it) {
      if (bar_try(bar, parity)) return true;
      if ((it & 63u) == 0) {
        if (*abort) return false;
        if (now_ns() - t0 > kWaitLimit) {
          give_up();
          return false;
        }
      }
    }
  }
  // ignores the abort flag: products in flight end by themselves
  __device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = now_ns();
    while (!bar_try(bar, parity))
      if (now_ns() - t0 > kWaitLimit) {
        give_up();
        return;
      }
  }
};

// Which keys of a tile count, bit r % 32 of word r / 32; a warp's lanes together.
struct Seen {
  uint32_t w[4];
  __device__ __forceinline__ bool at(int r) const { return w[r >> 5] >> (r & 31) & 1u; }
};
template <int SRC>
__device__ __forceinline__ Seen keys_seen(const AttendParams& P, const RowSeg& g, int t0) {
  const int lane = threadIdx.x & 31;
  Seen s;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + i * 32 + lane;
    bool in = t < g.len;
    if (SRC == kDense && P.mask && in) in = __ldg(P.mask + g.b * P.mask_stride + t) != 0;
    s.w[i] = __ballot_sync(0xffffffffu, in);
  }
  return s;
}

// ------------------------------------------------------------------ the kernel

template <typename T, int SRC, int D, int QT>
__global__ void __launch_bounds__(kRowThreads, 1) rows_kernel(const __grid_constant__ AttendParams P) {
  using C = RowsCfg<D, QT>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ RowPlan plan;
  const uint32_t raw = smem_at(smem_raw), base = (raw + 1023u) & ~1023u;
  unsigned char* const gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t KFULL = base + C::OFF_BAR, KEMPTY = KFULL + 8u * C::KST, VFULL = KEMPTY + 8u * C::KST,
                 VEMPTY = VFULL + 8u * C::VST, QFULL = VEMPTY + 8u * C::VST, QEMPTY = QFULL + 8u, SFULL = QEMPTY + 8u,
                 PFULL = SFULL + 16u, OFULL = PFULL + 16u, OEMPTY = OFULL + 16u, DRAIN = OEMPTY + 8u;
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(gbase + C::OFF_MISC);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::KST; ++i) {
      bar_init(KFULL + 8u * i, 32);
      bar_init(KEMPTY + 8u * i, 1);
    }
    for (int i = 0; i < C::VST; ++i) {
      bar_init(VFULL + 8u * i, 32);
      bar_init(VEMPTY + 8u * i, 1);
    }
    bar_init(QFULL, 32);
    bar_init(QEMPTY, 1);
    for (int i = 0; i < 2; ++i) {
      bar_init(SFULL + 8u * i, 1);
      bar_init(PFULL + 8u * i, 128);
      bar_init(OFULL + 8u * i, 1);
    }
    bar_init(OEMPTY, 256);
    bar_init(DRAIN, 1);
    misc[1] = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + C::OFF_MISC), "r"(C::TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  grid_dependency_wait();
  allow_dependents();
  const int T_all = build_row_plan<SRC>(P, plan, blockIdx.x == 0);  // (its barriers also show the lines above to all threads)
  tc_after();
  const uint32_t tmem = misc[0];
  const RowSplit split(P, T_all);
  const int x0 = blockIdx.x < split.used ? split.begin(blockIdx.x) : 0, x1 = blockIdx.x < split.used ? split.begin(blockIdx.x + 1) : 0;
  RowWaiter W{misc + 1, P.pages.status};

  // requests without keys
  if constexpr (SRC == kDense) {
    for (int b = blockIdx.x; b < P.pages.n_req; b += gridDim.x) {
      if (plan.first[b + 1] > plan.first[b]) continue;
      for (int64_t i = threadIdx.x; i < static_cast<int64_t>(P.n_q) * P.n_tok; i += kRowThreads) {
        const int j = static_cast<int>(i / P.n_q), head = static_cast<int>(i - static_cast<int64_t>(j) * P.n_q);
        uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(P.o) + b * P.o_b + head * P.o_h + j * P.o_n);
        for (int c = 0; c < D / 8; ++c) o[c] = make_uint4(0u, 0u, 0u, 0u);
        if (P.lse) P.lse[(static_cast<int64_t>(b) * P.n_q + head) * P.n_tok + j] = kNegInf;
      }
    }
  }
  // registers: the softmax holds a row of S (2 x 128 x 208 + 128 x 88 = 384 x 168)
  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  if (warp == 9 || warp == 10) {
    // ---- K and V tiles
    const bool is_v = warp == 10;
    const int stages = is_v ? C::VST : C::KST;
    const uint32_t ring = base + (is_v ? C::OFF_V : C::OFF_K), full = is_v ? VFULL : KFULL, empty = is_v ? VEMPTY : KEMPTY;
    const T* const pool = static_cast<const T*>(is_v ? P.pages.v : P.pages.k);
    constexpr int PIECES = D / 8, RPI = 32 / PIECES;  // a row's pieces of 16 bytes; rows that a warp copies at a time
    const int piece = lane % PIECES, r0 = lane / PIECES;
    int i = 0;
    bool ok = true;
    for (int x = x0; x < x1 && ok;) {
      const RowSeg g = row_seg<SRC>(P, plan, x, x1);
      for (int t = 0; t < g.n; ++t, ++i) {
        const int t0 = (g.tile0 + t) * kTile;
        const Seen seen = keys_seen<SRC>(P, g, t0);
        // the rows' places: lane l works out rows l, l + 32, ..
        int64_t off[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          off[u] = -1;
          const int key = t0 + u * 32 + lane;
          if (!(seen.w[u] >> lane & 1u)) continue;
          if constexpr (SRC == kShared) {
            const uint32_t pg = page_of(P.pages, static_cast<uint32_t>(key));
            off[u] = slot_offset(P.pages, __ldg(P.prefix_table + static_cast<int64_t>(g.b) * P.prefix_max_pages + pg),
                                 key - pg * P.pages.page_size);
            if (off[u] < 0) atomicOr(P.pages.status, kErrInput);
          } else {
            off[u] = g.b * P.pages.page_stride + key * P.pages.tok_stride;
          }
          if (off[u] >= 0) off[u] += g.h * P.pages.head_stride;
          if (off[u] >= 0 && !in_bounds(pool + off[u], D, pool, P.pages.extent, P.pages.status, kSitePool)) off[u] = -1;
        }
        const int stage = i % stages;
        if (i >= stages && !__all_sync(0xffffffffu, W.wait(empty + 8u * stage, (i / stages - 1) & 1u))) {
          ok = false;
          break;
        }
        const uint32_t dst = ring + stage * C::TILE + (piece >> 3) * kHalf;
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll 8
          for (int j = 0; j < 32 / RPI; ++j) {
            const int in32 = j * RPI + r0, r = u * 32 + in32;
            const int64_t ro = __shfl_sync(0xffffffffu, off[u], in32);
            copy16(dst + r * 128 + (((piece & 7) ^ (r & 7)) << 4), pool + (ro >= 0 ? ro : 0) + piece * 8, ro >= 0 ? 16 : 0);
          }
        copies_arrive(full + 8u * stage);
      }
      x += g.n;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 11) {
    // ---- Q: the segment's rows, once the products of the last one's are done
    const T* const q = static_cast<const T*>(P.q);
    int seg = 0;
    for (int x = x0; x < x1; ++seg) {
      const RowSeg g = row_seg<SRC>(P, plan, x, x1);
      if (seg > 0 && !__all_sync(0xffffffffu, W.wait(QEMPTY, (seg - 1) & 1u))) break;
      constexpr int PIECES = D / 8, RPI = 32 / PIECES;
      const int piece = lane % PIECES, rows = g.rows > kRowTile ? 2 * kRowTile : kRowTile;
#pragma unroll 4
      for (int r = lane / PIECES; r < rows; r += RPI) {
        const bool in = r < g.rows;
        copy16(base + C::OFF_Q + (r / kRowTile) * C::Q_TILE + (piece >> 3) * kHalf + (r % kRowTile) * 128 + (((piece & 7) ^ (r & 7)) << 4),
               q + (in ? row_q<SRC, D>(P, plan, g, r) + piece * 8 : 0), in ? 16 : 0);
      }
      copies_arrive(QFULL);
      x += g.n;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ---- the products.  Step u of a segment: stream u & 1; S(u + 2) follows P V(u), whose P lies over it
    constexpr uint32_t idesc_s = rows_idesc<T>(kTile, false), idesc_o = rows_idesc<T>(D, true);
    int seg = 0, kt = 0, vt = 0;  // segments, and tiles of K and V used, so far
    uint32_t np[2] = {0, 0};      // P's of each stream so far
    bool ok = true;
    for (int x = x0; x < x1 && ok; ++seg) {
      const RowSeg g = row_seg<SRC>(P, plan, x, x1);
      if (lane == 0) {
        const bool two = QT == 2 && g.rows > kRowTile;
        const int steps = two ? 2 * g.n : g.n;
        auto issue_s = [&](int u) {
          const int s = u & 1;
          const bool opens = !two || s == 0, closes = !two || s == 1;  // the first and last use of the tile
          const int stage = kt % C::KST;
          if (opens && !W.wait(KFULL + 8u * stage, (kt / C::KST) & 1u)) return false;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // copies (generic proxy) before the tensor cores' reads
          tc_after();
          const uint32_t a = desc_of(base + C::OFF_Q + (two ? s : 0) * C::Q_TILE, 16), b = desc_of(base + C::OFF_K + stage * C::TILE, 16);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t adv = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
            mma_ss(tmem + s * 128, a + adv, b + adv, kRowsDescHi, idesc_s, k > 0);
          }
          commit(SFULL + 8u * s);
          if (closes) {
            commit(KEMPTY + 8u * stage);
            ++kt;
          }
          if (u == steps - 1) commit(QEMPTY);
          return true;
        };
        ok = W.wait(QFULL, seg & 1u) && issue_s(0) && (steps == 1 || issue_s(1));
        for (int u = 0; u < steps && ok; ++u) {
          const int s = u & 1;
          const bool opens = !two || s == 0, closes = !two || s == 1;
          const int stage = vt % C::VST;
          ok = (!opens || W.wait(VFULL + 8u * stage, (vt / C::VST) & 1u)) && (u > 0 || seg == 0 || W.wait(OEMPTY, (seg - 1) & 1u)) &&
               W.wait(PFULL + 8u * s, np[s] & 1u);
          if (!ok) break;
          ++np[s];
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          tc_after();
          const uint32_t a = tmem + s * 128, d = tmem + C::O_COL + s * D;
          const uint32_t b = desc_of(base + C::OFF_V + stage * C::TILE, kHalf);
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k) mma_ts(d, a + k * 8, b + ((k * 2048) >> 4), kRowsDescHi, idesc_o, u > 1 || k > 0);
          if (!two) {
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k) mma_ts(d, a + 64 + k * 8, b + ((k * 2048) >> 4), kRowsDescHi, idesc_o, true);
          }
          if (closes) {
            commit(VEMPTY + 8u * stage);
            ++vt;
          }
          if (u + 2 >= steps) commit(OFULL + 8u * s);  // the stream's last
          else ok = issue_s(u + 2);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      x += g.n;
    }
    if (lane == 0) {  // every product issued here has ended before the tensor memory is given back
      commit(DRAIN);
      W.drain(DRAIN, 0u);
    }
    __syncwarp();
  }
  } else {
    // ---- softmax.  Thread: row `row` of its stream
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int s = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // 32 lanes a warp, in an address's upper half
    const uint32_t at_s = tmem + lanes + s * 128;
    float2* const s_ml = reinterpret_cast<float2*>(gbase + C::OFF_ML);
    uint32_t ns = 0, no[2] = {0, 0};  // S's of this stream, and ends of both, so far
    bool ok = true;
    for (int x = x0; x < x1;) {
      if (!softmax_sync(ok)) break;  // (and the last segment's states have been read)
      const RowSeg g = row_seg<SRC>(P, plan, x, x1);
      const bool two = QT == 2 && g.rows > kRowTile;
      const int steps = two ? 2 * g.n : g.n, mine = (steps + 1 - s) / 2;  // steps of this stream
      const int my_rows = two ? g.rows - s * kRowTile : g.rows;
      const bool busy = (warp & 3) * 32 < my_rows;  // this warp has rows
      float m = kNegInf, l = 0.f;
      for (int i = 0; i < mine; ++i, ++ns) {
        const int t0 = (g.tile0 + (two ? i : 2 * i + s)) * kTile;
        const bool all = (SRC != kDense || !P.mask) && t0 + kTile <= g.len;
        Seen seen;
        if (!all) seen = keys_seen<SRC>(P, g, t0);
        if (!__all_sync(0xffffffffu, W.wait(SFULL + 8u * s, ns & 1u))) {
          ok = false;
          break;
        }
        if (busy) {
          tc_after();
          float v[kTile];
          tmem_read32<0>(at_s, v);
          tmem_read32<32>(at_s + 32, v);
          tmem_read32<64>(at_s + 64, v);
          tmem_read32<96>(at_s + 96, v);
          if (!all) {
#pragma unroll
            for (int k = 0; k < kTile; ++k) v[k] = seen.at(k) ? v[k] : kNegInf;
          }
          float top = v[0];
#pragma unroll
          for (int k = 1; k < kTile; ++k) top = fmaxf(top, v[k]);
          top = top * P.scale;
          if (__any_sync(0xffffffffu, top > m + (kTau + Mma<T>::kLift))) {
            const float now = fmaxf(m, top - Mma<T>::kLift);
            const float f = now == kNegInf ? 1.f : ex2(m - now);
            m = now;
            l *= f;
            if (i > 0) {  // S(i) was issued behind P V(i - 1), so O holds all up to it
#pragma unroll
              for (int c = 0; c < D; c += 32) {
                float o[32];
                tmem_read32<0>(tmem + lanes + C::O_COL + s * D + c, o);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] *= f;
                tmem_write32(tmem + lanes + C::O_COL + s * D + c, o);
              }
            }
          }
          const float less = m == kNegInf ? 0.f : -m;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < kTile; c += 32) {
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float a = ex2(fmaf(v[c + 2 * k], P.scale, less)), b = ex2(fmaf(v[c + 2 * k + 1], P.scale, less));
              sum[(2 * k) & 3] += a;
              sum[(2 * k + 1) & 3] += b;
              if (two) hi[k] = Mma<T>::down2(a, b);
              else Mma<T>::split(a, b, hi[k], lo[k]);
            }
            tmem_write16(at_s + c / 2, hi);
            if (!two) tmem_write16(at_s + 64 + c / 2, lo);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_written();
          tc_before();
        }
        bar_arrive(PFULL + 8u * s);
      }
      // ---- the segment's end
      const bool whole = g.tile0 == 0 && g.first + g.n == g.end;
      const int slot = blockIdx.x * 2 + (g.tile0 == 0 ? 1 : 0);
      const bool other = !two && steps > 1;  // the same rows' other half
      if (!two) {
        if (mine > 0) s_ml[s * kRowTile + row] = make_float2(m, l);
        ok = softmax_sync(ok);
      }
      if (ok) {
        if (two || s == 0 || mine > 0) ok = W.wait(OFULL + 8u * s, no[s] & 1u);
        if (!two && ok) ok = (s == 1 || other) ? W.wait(OFULL + 8u * (1 - s), no[1 - s] & 1u) : true;
        ok = __all_sync(0xffffffffu, ok);
      }
      ++no[0];
      if (two || other) ++no[1];
      if (ok && busy) {
        tc_after();
        // two row blocks: all of this stream's columns; one: half of the columns, of both streams
        float f0 = 1.f, f1 = 0.f;
        if (!two) {
          const float2 a = s_ml[row], b = other ? s_ml[kRowTile + row] : make_float2(kNegInf, 0.f);
          m = fmaxf(a.x, b.x);
          const float less = m == kNegInf ? 0.f : -m;
          f0 = ex2(a.x + less);
          f1 = ex2(b.x + less);
          l = a.y * f0 + b.y * f1;
        }
        const bool mine_too = row < my_rows;
        const int r = two ? s * kRowTile + row : row;
        const int c0 = two ? 0 : s * (D / 2), c1 = two ? D : c0 + D / 2;
        RowOut at{0, 0};
        if (mine_too) at = row_out<SRC, D>(P, plan, g, r);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        for (int c = c0; c < c1; c += 32) {
          float o[32];
          tmem_read32<0>(tmem + lanes + C::O_COL + (two ? s * D : 0) + c, o);
          if (!two) {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] *= f0;
            if (other) {
              float o1[32];
              tmem_read32<0>(tmem + lanes + C::O_COL + D + c, o1);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = fmaf(o1[k], f1, o[k]);
            }
          }
          if (!mine_too) continue;
          if (whole && SRC == kDense) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = l == 0.f ? 0u : Mma<T>::down2(o[k + 2 * e] * inv, o[k + 2 * e + 1] * inv);
              *reinterpret_cast<uint4*>(static_cast<T*>(P.o) + at.o + c + k) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else if (whole) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<float4*>(P.state_o + at.o + c + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          } else {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              P.rows_o[(static_cast<int64_t>(slot) * (D / 4) + (c + k) / 4) * P.item_rows + r] = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          }
        }
        if (mine_too && (two || s == 0)) {
          if (!whole) P.rows_ml[static_cast<int64_t>(slot) * P.item_rows + r] = make_float2(m, l);
          else if (SRC == kShared) P.state_ml[at.lse] = make_float2(m, l);
          else if (P.lse) P.lse[at.lse] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
        }
        tc_before();
      }
      bar_arrive(OEMPTY);
      x += g.n;
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS) : "memory");
}

// Merges the pieces of the items that more than one CTA worked on.  A job: an item, found at the first boundary between CTAs that it
// crosses, and 8 of its rows; a warp: 8 rows x 16 dimensions.
template <typename T, int SRC, int D>
__global__ void __launch_bounds__(kWarps * 32) join_rows(const __grid_constant__ AttendParams P) {
  constexpr int BLOCKS = D / 16, PER = kWarps / BLOCKS;  // blocks of dimensions; row groups at a time
  __shared__ RowPlan plan;
  const int T_all = build_row_plan<SRC>(P, plan, false);
  const RowSplit split(P, T_all);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r8 = lane & 7, d4 = (warp % BLOCKS) * 4 + (lane >> 3);
  grid_dependency_wait();
  allow_dependents();
  const int groups = P.item_rows / 8, jobs = max(static_cast<int>(split.used) - 1, 0) * groups;
  for (int j = blockIdx.x * PER + warp / BLOCKS; j < jobs; j += gridDim.x * PER) {
    const int c0 = j / groups, r = (j - c0 * groups) * 8 + r8;
    const int x = split.begin(c0 + 1);
    const RowSeg g = row_seg<SRC>(P, plan, x, x + 1);
    if (g.first >= x || g.first < split.begin(c0) || r - r8 >= g.rows) continue;
    const int pieces = split.of(g.end - 1) - c0 + 1;
    const float2* ml = P.rows_ml + static_cast<int64_t>(c0) * 2 * P.item_rows + r;
    const float4* po = P.rows_o + (static_cast<int64_t>(c0) * 2 * (D / 4) + d4) * P.item_rows + r;
    auto slot = [](int c) { return c == 0 ? 1 : 2 * c; };
    const bool in = r < g.rows;
    float M = kNegInf;
    for (int c = lane >> 3; c < pieces && in; c += 4) M = fmaxf(M, __ldcg(ml + static_cast<int64_t>(slot(c)) * P.item_rows).x);
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 8));
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
    if (!in) continue;
    const float less = M == kNegInf ? 0.f : -M;
    float L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int c = 0; c < pieces; ++c) {
      const float2 s = __ldcg(ml + static_cast<int64_t>(slot(c)) * P.item_rows);
      const float4 v = __ldcg(po + static_cast<int64_t>(slot(c)) * (D / 4) * P.item_rows);
      const float f = ex2(s.x + less);
      L = fmaf(s.y, f, L);
      o.x = fmaf(v.x, f, o.x);
      o.y = fmaf(v.y, f, o.y);
      o.z = fmaf(v.z, f, o.z);
      o.w = fmaf(v.w, f, o.w);
    }
    write_row<T>(P, row_out<SRC, D>(P, plan, g, r), d4 * 4, M, L, o);
  }
}

// ------------------------------------------------------------------ host

struct RowSizes {
  int32_t item_rows, ctas, min_tiles;
  size_t rows_o, rows_ml, total;
};

// CTAs for `tiles` tiles of items of at most `rows` rows, and where their pieces lie behind `at` bytes of a workspace.
inline void size_rows(RowSizes* z, int64_t tiles, int64_t rows, int head_dim, int sms, size_t at) {
  z->item_rows = rows > kRowTile ? 2 * kRowTile : kRowTile;
  z->min_tiles = 2;
  z->ctas = static_cast<int32_t>(std::min<int64_t>(std::min(sms, kMaxCtas), std::max<int64_t>((tiles + z->min_tiles - 1) / z->min_tiles, 1)));
  z->rows_o = up256(at);
  z->rows_ml = z->rows_o + static_cast<size_t>(z->ctas) * 2 * z->item_rows * head_dim * 4;
  z->total = z->rows_ml + up256(static_cast<size_t>(z->ctas) * 2 * z->item_rows * 8);
}
inline void place_rows(AttendParams& p, const RowSizes& z, char* ws) {
  p.rows_o = reinterpret_cast<float4*>(ws + z.rows_o);
  p.rows_ml = reinterpret_cast<float2*>(ws + z.rows_ml);
  p.item_rows = z.item_rows;
  p.row_ctas = z.ctas;
  p.min_tiles = z.min_tiles;
}

template <typename T, int SRC, int D, int QT>
cudaError_t launch_rows_of(const AttendParams& p, int device, cudaStream_t s) {
  constexpr int bytes = RowsCfg<D, QT>::SMEM;
  static std::atomic<bool> done[64];
  if (device >= 64 || !done[device].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(rows_kernel<T, SRC, D, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (device < 64) done[device].store(true, std::memory_order_release);
  }
  return launch_pdl(rows_kernel<T, SRC, D, QT>, dim3(p.row_ctas), dim3(kRowThreads), bytes, s, p);
}
template <typename T, int SRC, int D>
cudaError_t launch_rows(const AttendParams& p, int device, cudaStream_t s) {
  return p.item_rows > kRowTile ? launch_rows_of<T, SRC, D, 2>(p, device, s) : launch_rows_of<T, SRC, D, 1>(p, device, s);
}

}  // namespace
}  // namespace svx
