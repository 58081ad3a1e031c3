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
//   warp 8          issues the products (one lane, the warp converged)
//   warps 9, 10     bring K and V tiles in: by tensor map, in boxes of a page or a tile, where pages and strides allow and all of the
//                   tile's keys count (of K, an encoder's states: any of them), else in 16-byte cp.async, rows found through the
//                   page table or by stride
//   warp 11         brings Q in: by tensor map where 128 rows are a whole number of tokens or requests
// Up to 128 rows the tensor cores have time to spare (the bytes of K and V bound the time), and P enters the product in two 16-bit pieces:
// O is then as exact as with fp32 weights.  Where there are more than 128 rows to the same keys (of prefixes: on average) the products
// bound the time, and P is rounded once: a weight is off by up to 2^-8 (bf16) or 2^-11 (fp16) of itself.
//
// Long sums.  The tensor cores drop from each product what lies some 26 bits below the sum that it joins: where V is positive, O lost 2^-27 of
// itself a key (0.08% of 131072 keys in one segment, 2.6% of 4 million, half of 2^27).  So every kSumTiles tiles a stream's O goes to memory,
// where it is added up in fp32, and begins anew: the loss is that of 32768 keys, 2^-12, half of what rounding O to fp16 may take.  (256
// rows to an SM x 131072 keys: d = 128 1369 us without, 1404; d = 64 1178, 1162.)
//
// What bounds it.  Two row tiles, d = 128: the products; 8192 x 16384 tokens of 32 heads 1204 us = 1827 TFLOP/s, 95% of the measured cuBLAS
// rate.  d = 64: half the products to the same softmax, whose own steps decide (2 x 2048 x 4096 tokens of 16 heads: the tensor
// pipe busy for 39%, the exponentials' for 39%, 43% of the issue slots).  One row tile: the bytes of K and V (16 samples behind 32768
// slots, 8 KV heads, 134 MB: 44 us with the start, the join and the samples' own slots).  Few tiles to an item: the way from Q through S, P
// and O to the output, which a stream takes while the other one computes, 6000 to 7000 cycles an item (8 x 4096 tokens x 77 states,
// 16 heads of d = 64: 68 us, of which the bytes are 20).  There leaving out the chunks of 32 keys behind a length gained 0 to 4%, and
// cost full tiles 3 to 5%; P beside S in tensor memory, so that S(i + 2) need not wait for P V(i), gained nothing at d = 64.
//
// Every wait is bounded (2 s of global time; that for a segment's last product with Q, which a segment of many keys takes longer to reach, 2 s
// without a new tile): one that gives up raises the status word and makes all roles stop, drain and leave; the rows that the CTA had to do become
// NaN, since there may be no status word.
#pragma once

#include "svx_attend.cuh"

#include <cuda.h>

#include <type_traits>

namespace svx {
namespace {

constexpr int kRowTile = 128;
constexpr uint32_t kHalf = kKeyTile * 128;      // bytes of 64 dimensions of 128 rows (an operand's swizzle atoms: 8 rows of 128 bytes)
constexpr uint64_t kWaitLimit = 2000000000ull;  // ns
constexpr int kRowThreads = 384;
constexpr int kSumTiles = 256;  // that a stream adds up in tensor memory (a power of two)

// QT: row tiles of an item, 1 or 2.
template <int D, int QT>
struct RowsCfg {
  static constexpr uint32_t TILE = kKeyTile * D * 2;  // K or V
  // with one row tile the bytes in flight decide: 5 tiles of 32 KiB (d = 128), 8 of 16 KiB (d = 64)
  static constexpr int KST = D == 128 ? 2 : 4;
  static constexpr int VST = D == 128 ? 4 - QT : 4;
  static constexpr int QST = D == 128 ? 1 : 2;  // segments' Q: where there is room, the next one's comes in meanwhile
  static constexpr uint32_t Q_TILE = kRowTile * D * 2;
  static constexpr uint32_t OFF_K = 0;
  static constexpr uint32_t OFF_V = OFF_K + KST * TILE;
  static constexpr uint32_t OFF_Q = OFF_V + VST * TILE;
  static constexpr uint32_t OFF_OUT = OFF_Q + QST * QT * Q_TILE;  // [8 warps][32 rows][32 dimensions]: outputs on their way
  static constexpr uint32_t OFF_ML = OFF_OUT + 8 * 2048;  // float2 [2][128]: the streams' states at a segment's end
  static constexpr int N_BAR = 2 * KST + 2 * VST + 2 * QST + 4 * 2 + 1;
  static constexpr uint32_t OFF_BAR = OFF_ML + 2 * kRowTile * 8;
  static constexpr uint32_t OFF_MISC = OFF_BAR + N_BAR * 8;  // [0] TMEM base, [1] abort flag, [2] K tiles begun
  static constexpr uint32_t BYTES = OFF_MISC + 16;
  static constexpr uint32_t SMEM = BYTES + 1024;  // slack to align the base to 1024 bytes
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t O_COL = 256;  // S (and P over it): 128 columns a stream; O: D a stream
  static_assert(SMEM + 5 * 1024 <= 232448, "shared memory per CTA, with the plan");
};

// The kernel's parameters: with tensor maps of K and V, of dimensions (d, KV head, slot, page) or (d, KV head, state, request), if their
// strides allow: a box is 64 dimensions of `box` slots of a head, a page's or a part of them, at most a tile's.  And one of Q, (d, query
// head, token, request) or (d, query head, request, 1), where a row tile is a whole number of tokens or requests.
struct RowsParams : AttendParams {
  CUtensorMap k_map, v_map, q_map;
  int32_t box;                 // 0: no maps of K and V
  int32_t q_box;               // tokens or requests of a row tile; 0: no map of Q
  int32_t head_step, page_step;  // 0 where all heads or requests are the same
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
__device__ __forceinline__ void arrive_expecting(uint32_t bar, uint32_t bytes) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes) : "memory");
}
// A box of a map, from (x, y, z, w), to shared memory; its bytes count on the barrier.
__device__ __forceinline__ void bring_box(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
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
// Shared-memory descriptor, 128-byte swizzle: high word (stride between groups of 8 rows 1024 bytes, version, swizzle mode); low word:
// desc_of (address, leading-dimension offset).
constexpr uint32_t kRowsDescHi = (1024u >> 4) | (1u << (46 - 32)) | (2u << (61 - 32));
// One lane of a converged warp.  The warp that issues the products stays converged and holds their operands alike in all lanes: then they
// are in uniform registers, where the instructions take them from (issued from a branch of one lane, a product took 60 to 70
// cycles to issue, as long as it takes to run, and a commit 100).
__device__ __forceinline__ uint32_t one_lane() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e) :: "memory");
  return e;
}
// D = A B (+ D), issued by the lane with `one`; operands as the low words of shared-memory descriptors (the high word is the same
// for all).
__device__ __forceinline__ void mma_ss(uint32_t one, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 e, %6, 0;\n\tmov.b64 da, {%1, %3};\n\t"
      "mov.b64 db, {%2, %3};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(kRowsDescHi), "r"(idesc), "r"(static_cast<uint32_t>(add)), "r"(one)
      : "memory");
}
// The same with A in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t one, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 e, %6, 0;\n\tmov.b64 db, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(kRowsDescHi), "r"(idesc), "r"(static_cast<uint32_t>(add)), "r"(one)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t one, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(one)
      : "memory");
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
// 64 columns.
__device__ __forceinline__ void tmem_read64(uint32_t at, float (&v)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]),
        "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]),
        "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]), "=f"(v[32]), "=f"(v[33]), "=f"(v[34]), "=f"(v[35]),
        "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]), "=f"(v[40]), "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]),
        "=f"(v[45]), "=f"(v[46]), "=f"(v[47]), "=f"(v[48]), "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]),
        "=f"(v[54]), "=f"(v[55]), "=f"(v[56]), "=f"(v[57]), "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]),
        "=f"(v[63])
      : "r"(at)
      : "memory");
}
// 128 columns.
__device__ __forceinline__ void tmem_read128(uint32_t at, float (&v)[128]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x128.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,"
      "%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,"
      "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95,"
      "%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,"
      "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%128];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]), "=f"(v[32]),
        "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]), "=f"(v[40]),
        "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]), "=f"(v[48]),
        "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]), "=f"(v[56]),
        "=f"(v[57]), "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63]), "=f"(v[64]),
        "=f"(v[65]), "=f"(v[66]), "=f"(v[67]), "=f"(v[68]), "=f"(v[69]), "=f"(v[70]), "=f"(v[71]), "=f"(v[72]),
        "=f"(v[73]), "=f"(v[74]), "=f"(v[75]), "=f"(v[76]), "=f"(v[77]), "=f"(v[78]), "=f"(v[79]), "=f"(v[80]),
        "=f"(v[81]), "=f"(v[82]), "=f"(v[83]), "=f"(v[84]), "=f"(v[85]), "=f"(v[86]), "=f"(v[87]), "=f"(v[88]),
        "=f"(v[89]), "=f"(v[90]), "=f"(v[91]), "=f"(v[92]), "=f"(v[93]), "=f"(v[94]), "=f"(v[95]), "=f"(v[96]),
        "=f"(v[97]), "=f"(v[98]), "=f"(v[99]), "=f"(v[100]), "=f"(v[101]), "=f"(v[102]), "=f"(v[103]), "=f"(v[104]),
        "=f"(v[105]), "=f"(v[106]), "=f"(v[107]), "=f"(v[108]), "=f"(v[109]), "=f"(v[110]), "=f"(v[111]),
        "=f"(v[112]), "=f"(v[113]), "=f"(v[114]), "=f"(v[115]), "=f"(v[116]), "=f"(v[117]), "=f"(v[118]),
        "=f"(v[119]), "=f"(v[120]), "=f"(v[121]), "=f"(v[122]), "=f"(v[123]), "=f"(v[124]), "=f"(v[125]),
        "=f"(v[126]), "=f"(v[127])
      : "r"(at)
      : "memory");
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
__device__ __forceinline__ uint32_t desc_of(uint32_t addr, uint32_t lead) {
  return ((addr >> 4) & 0x3FFFu) | (((lead >> 4) & 0x3FFFu) << 16);
}

// ------------------------------------------------------------------ the flat range

// As Plan, of items of up to P.item_rows rows and tiles of kKeyTile keys.  Sequences: the requests, or (kShared) the prefixes.
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
  const int tiles = rows ? static_cast<int>((static_cast<uint32_t>(n) + (kKeyTile - 1)) / kKeyTile) : 0;
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

// The T tiles over the CTAs, as Split.  Fewer CTAs have more to do, and leave the join fewer pieces: with up to 8 tiles each is a CTA's
// (5 tiles of an item: 9.4 us; two or four to a CTA 9.9 and 11.5), else at least two (8 items of 16: single 15.7 us, two 13.9, four 14.6;
// one of 32: 13.6, 12.6, 14.5), or four of long items (one of 128: 26.3, 19.6, 17.7; two of 79, d = 64: 28.0, 21.3, 17.0), until there
// are three to each of all CTAs (8 items of 63: at least four 23.8 us, all CTAs 21.6).
struct RowSplit {
  uint32_t used, q, r, total;
  float per_used;
  __device__ __forceinline__ RowSplit(const AttendParams& P, int T) {
    total = T;
    const uint32_t ctas = P.row_ctas, least = total <= 8 ? 1 : total <= 40 ? min(P.row_least, 2) : P.row_least;
    used = total >= 3 * ctas ? ctas : min((total + least - 1) / least, ctas);
    q = used ? total / used : 0;
    r = total - q * used;
    per_used = __frcp_rn(static_cast<float>(used));
  }
  __device__ __forceinline__ int begin(uint32_t c) const {  // (the float product: see Split)
    return used ? static_cast<int>(c * q) + __float2int_rd(fmaf(static_cast<float>(c * r), per_used, 0.001f)) : 0;
  }
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

// (of sequence b)
template <int SRC>
__device__ __forceinline__ RowSeg row_seg_of(const AttendParams& P, const RowPlan& s, int b, int x, int x1) {
  RowSeg g;
  g.b = b;
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
// (all lanes of a warp alike)
template <int SRC>
__device__ __forceinline__ RowSeg row_seg(const AttendParams& P, const RowPlan& s, int x, int x1) {
  const int seqs = SRC == kShared ? P.n_prefix : P.pages.n_req;
  int b = 0;  // as many sequences lie before x's as end at x or before
  for (int i = 0; i < seqs; i += 32) {
    const int r = i + (threadIdx.x & 31);
    b += __popc(__ballot_sync(0xffffffffu, r < seqs && s.first[r + 1] <= x));
  }
  return row_seg_of<SRC>(P, s, b, x, x1);
}
// (each thread its own)
template <int SRC>
__device__ __forceinline__ RowSeg row_seg_at(const AttendParams& P, const RowPlan& s, int x) {
  int b = 0;
  for (int step = kMaxReq / 2; step > 0; step >>= 1)
    if (s.first[b + step] <= x) b += step;
  return row_seg_of<SRC>(P, s, b, x, x + 1);
}

// The first tile at x or behind it that begins an item.
template <int SRC>
__device__ __forceinline__ int row_item_start(const AttendParams& P, const RowPlan& s, int x, int total) {
  if (x >= total) return total;
  const RowSeg g = row_seg<SRC>(P, s, x, total);
  return g.tile0 == 0 ? x : g.end;
}

// x / n for x < 2^24: the float product with the inverse is off by less than one
__device__ __forceinline__ int fast_div(int x, int n, float inverse) {
  int q = static_cast<int>(static_cast<float>(x) * inverse);
  const int left = x - q * n;
  if (left < 0) --q;
  else if (left >= n) ++q;
  return q;
}

// Element offset of row r of a segment's block in q, and the places of its outputs.
template <int SRC, int D>
__device__ __forceinline__ int64_t row_q(const AttendParams& P, const RowPlan& s, const RowSeg& g, int r) {
  r += g.rt * P.item_rows;
  const int j = fast_div(r, P.group, P.group_inverse), head = g.h * P.group + (r - j * P.group);
  if constexpr (SRC == kShared) return (static_cast<int64_t>(s.req0[g.b] + j) * P.n_q + head) * D;
  return g.b * P.q_b + head * P.q_h + j * P.q_n;
}
template <int SRC, int D>
__device__ __forceinline__ RowOut row_out(const AttendParams& P, const RowPlan& s, const RowSeg& g, int r) {
  r += g.rt * P.item_rows;
  const int j = fast_div(r, P.group, P.group_inverse), head = g.h * P.group + (r - j * P.group);
  if constexpr (SRC == kShared) {
    const int64_t row = static_cast<int64_t>(s.req0[g.b] + j) * P.n_q + head;
    return RowOut{row * D, row};
  }
  return RowOut{g.b * P.o_b + head * P.o_h + j * P.o_n, (static_cast<int64_t>(g.b) * P.n_q + head) * P.n_tok + j};
}

struct RowWaiter {
  volatile uint32_t* abort;  // [1]: K tiles begun
  int* status;
  __device__ __forceinline__ void give_up() {
    *abort = 1u;
    if (status) atomicOr(status, kErrWait);
  }
  // (a converged warp stays so: all lanes' results are the same)
  __device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); }
  // For Q's place, which is free once all of a segment's tiles have met it: the limit runs from the last tile begun.
  __device__ __forceinline__ bool warp_wait_q(uint32_t bar, uint32_t parity) {
    bool ok = bar_try(bar, parity);
    uint64_t t0 = ok ? 0 : now_ns();
    uint32_t tiles = abort[1];
    for (uint32_t it = 1; !ok; ++it) {
      ok = bar_try(bar, parity);
      if (ok || (it & 63u) != 0) continue;
      if (*abort) break;
      if (abort[1] != tiles) {
        tiles = abort[1];
        t0 = now_ns();
      } else if (now_ns() - t0 > kWaitLimit) {
        give_up();
        break;
      }
    }
    return __all_sync(0xffffffffu, ok);
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

// The test hook: a wait on a barrier on which nothing arrives before the products have ended, for a millisecond.
__device__ __noinline__ bool run_out(RowWaiter w, uint32_t bar) {
  const uint64_t t0 = now_ns();
  while (now_ns() - t0 < 1000000ull)
    if (bar_try(bar, 0u)) return true;  // (a CTA without work)
  w.give_up();
  return false;
}

// Which keys of a tile count, bit r % 32 of word r / 32; a warp's lanes together.
struct Seen {
  uint32_t w[4];
};
// Scores of keys that do not count become -inf (out of line, so that the loop's usual path stays short).
__device__ __noinline__ void hide_keys(uint32_t at, Seen seen) {
#pragma unroll 1
  for (int c = 0; c < kKeyTile; c += 64) {
    const uint32_t w0 = c ? seen.w[2] : seen.w[0], w1 = c ? seen.w[3] : seen.w[1];
    if ((w0 & w1) == ~0u) continue;
    float v[64];
    tmem_read64(at + c, v);
#pragma unroll
    for (int h = 0; h < 64; h += 32) {
      float x[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) x[k] = (h ? w1 : w0) >> k & 1u ? v[h + k] : kNegInf;
      tmem_write32(at + c + h, x);
    }
  }
  tmem_written();
}
__device__ __noinline__ void scale_columns(uint32_t at, int n, float f) {
#pragma unroll 1
  for (int c = 0; c < n; c += 32) {
    float v[32];
    tmem_read32<0>(at + c, v);
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] *= f;
    tmem_write32(at + c, v);
  }
}
// A stream's O of this thread's row, in tensor memory, and what it had before that is in memory: a column's quad every kRowTile, relative to
// 2^ref.  Moves O there (first: there was nothing), or brings it back on top of O.  (Out of line, addresses and all.)
template <int D>
__device__ __noinline__ void put_sums(uint32_t at, float4* sums, float* ref, float m, bool first) {
  const int stream = blockIdx.x * 2 + threadIdx.x / kRowTile, row = threadIdx.x % kRowTile;
  sums += static_cast<int64_t>(stream) * (D / 4) * kRowTile + row;
  ref += stream * kRowTile + row;
  const float f = first || m == kNegInf ? 0.f : ex2(*ref - m);  // (no key so far: zeros)
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    float o[32];
    tmem_read32<0>(at + c, o);
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      float4* const to = sums + (c + k) / 4 * kRowTile;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!first) x = *to;
      *to = make_float4(fmaf(x.x, f, o[k]), fmaf(x.y, f, o[k + 1]), fmaf(x.z, f, o[k + 2]), fmaf(x.w, f, o[k + 3]));
    }
  }
  *ref = m;
}
template <int D>
__device__ __noinline__ void take_sums(uint32_t at, const float4* sums, const float* ref, float m) {
  const int stream = blockIdx.x * 2 + threadIdx.x / kRowTile, row = threadIdx.x % kRowTile;
  sums += static_cast<int64_t>(stream) * (D / 4) * kRowTile + row;
  ref += stream * kRowTile + row;
  const float f = m == kNegInf ? 0.f : ex2(*ref - m);
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    float o[32];
    tmem_read32<0>(at + c, o);
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      const float4 x = sums[(c + k) / 4 * kRowTile];
      o[k] = fmaf(x.x, f, o[k]), o[k + 1] = fmaf(x.y, f, o[k + 1]), o[k + 2] = fmaf(x.z, f, o[k + 2]), o[k + 3] = fmaf(x.w, f, o[k + 3]);
    }
    tmem_write32(at + c, o);
  }
  tmem_written();
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <int N>
__device__ __forceinline__ float max_of(const float (&v)[N]) {
  float m[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
  for (int k = 4; k < N - 4; k += 8)
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = max3(m[e], v[k + 2 * e], v[k + 2 * e + 1]);
#pragma unroll
  for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], v[N - 4 + e]);
  return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}
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
__global__ void __launch_bounds__(kRowThreads, 1) rows_kernel(const __grid_constant__ RowsParams P) {
  using C = RowsCfg<D, QT>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ RowPlan plan;
  const uint32_t raw = smem_at(smem_raw), base = (raw + 1023u) & ~1023u;
  unsigned char* const gbase = smem_raw + (base - raw);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t KFULL = base + C::OFF_BAR, KEMPTY = KFULL + 8u * C::KST, VFULL = KEMPTY + 8u * C::KST,
                 VEMPTY = VFULL + 8u * C::VST, QFULL = VEMPTY + 8u * C::VST, QEMPTY = QFULL + 8u * C::QST, SFULL = QEMPTY + 8u * C::QST,
                 PFULL = SFULL + 16u, OFULL = PFULL + 16u, OEMPTY = OFULL + 16u, DRAIN = OEMPTY + 16u;
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
    for (int i = 0; i < C::QST; ++i) {
      bar_init(QFULL + 8u * i, 32);
      bar_init(QEMPTY + 8u * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(SFULL + 8u * i, 1);
      bar_init(PFULL + 8u * i, 128);
      bar_init(OFULL + 8u * i, 1);
      bar_init(OEMPTY + 8u * i, 128);
    }
    bar_init(DRAIN, 1);
    misc[1] = misc[2] = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  // (before the tensor memory is asked for: a kernel that still runs may hold it)
  if (SRC != kShared) grid_dependency_wait();
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + C::OFF_MISC), "r"(C::TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  // Behind attend_kernel, which takes the requests' own slots: neither reads what the other writes, and that one had waited for all
  // that came before when it let this one start.  The wait is for the join, which relies on this kernel's end.
  allow_dependents();
  const int T_all = build_row_plan<SRC>(P, plan, blockIdx.x == 0);  // (its barriers also show the lines above to all threads)
  tc_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, misc[0], 0);
  const RowSplit split(P, T_all);
  int x0 = blockIdx.x < split.used ? split.begin(blockIdx.x) : 0, x1 = blockIdx.x < split.used ? split.begin(blockIdx.x + 1) : 0;
  if (P.row_whole) {  // the items that begin in the range, whole
    x0 = row_item_start<SRC>(P, plan, x0, T_all);
    x1 = x1 ? row_item_start<SRC>(P, plan, x1, T_all) : x0;
  }
  RowWaiter W{misc + 1, P.pages.status};

  // requests without keys: their rows over all threads
  if constexpr (SRC == kDense) {
    for (int b0 = 0; b0 < P.pages.n_req; b0 += 32) {
      const int mine = b0 + lane;
      uint32_t none = __ballot_sync(0xffffffffu, mine < P.pages.n_req && plan.first[mine + 1] <= plan.first[mine]);
      for (; none; none &= none - 1) {
        const int b = b0 + __ffs(none) - 1;
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x; i < static_cast<int64_t>(P.n_q) * P.n_tok;
             i += static_cast<int64_t>(gridDim.x) * kRowThreads) {
          const int j = static_cast<int>(i / P.n_q), head = static_cast<int>(i - static_cast<int64_t>(j) * P.n_q);
          uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(P.o) + b * P.o_b + head * P.o_h + j * P.o_n);
          for (int c = 0; c < D / 8; ++c) o[c] = make_uint4(0u, 0u, 0u, 0u);
          if (P.lse) P.lse[(static_cast<int64_t>(b) * P.n_q + head) * P.n_tok + j] = kNegInf;
        }
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
    const CUtensorMap* const map = is_v ? &P.v_map : &P.k_map;
    const bool maps = P.box > 0;
    const int box = maps ? P.box : kKeyTile;
    if (maps && lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
    int i = 0;
    bool ok = true;
    for (int x = x0; x < x1 && ok;) {
      const RowSeg g = row_seg<SRC>(P, plan, x, x1);
      const int32_t* const table = SRC == kShared ? P.prefix_table + static_cast<int64_t>(g.b) * P.prefix_max_pages : nullptr;
      // lane l works out the places of keys l, l + 32, ..; their pages are looked up a tile ahead
      int32_t page[4];
      auto look = [&](int t) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t key = static_cast<uint32_t>(g.tile0 + t) * kKeyTile + u * 32 + lane;  // (behind the last tile: up to 2^31 + 127)
          page[u] = t < g.n && key < static_cast<uint32_t>(g.len) ? __ldg(table + page_of(P.pages, key)) : 0;
        }
      };
      if constexpr (SRC == kShared) look(0);
      for (int t = 0; t < g.n; ++t, ++i) {
        const int t0 = (g.tile0 + t) * kKeyTile;
        const int stage = i % stages;
        if (!is_v && lane == 0) misc[2] = i;
        const uint32_t dst = ring + stage * C::TILE;
        const Seen seen = keys_seen<SRC>(P, g, t0);
        const bool all = (seen.w[0] & seen.w[1] & seen.w[2] & seen.w[3]) == 0xffffffffu;
        // (keys that do not count: their scores are put out, whatever K holds; but V has to be zero there)
        const bool any = (seen.w[0] | seen.w[1] | seen.w[2] | seen.w[3]) != 0u;
        bool boxes = maps && (all || (SRC == kDense && !is_v && any && t0 + kKeyTile <= P.max_len));
        if constexpr (SRC == kShared) {
          const uint32_t n = P.pages.n_pages;
          boxes = boxes && __all_sync(0xffffffffu, static_cast<uint32_t>(page[0]) < n && static_cast<uint32_t>(page[1]) < n &&
                                                       static_cast<uint32_t>(page[2]) < n && static_cast<uint32_t>(page[3]) < n);
        }
        // in boxes, one or more a lane.  Lane l: half l / runs of the dimensions, run l % runs
        const int runs = kKeyTile / box, half = lane / runs, key = lane % runs * box;
        int w = g.b * P.page_step, z = t0;
        if (boxes) {
          if constexpr (SRC == kShared) {
            const int32_t p01 = __shfl_sync(0xffffffffu, page[0], key & 31), p1 = __shfl_sync(0xffffffffu, page[1], key & 31),
                          p2 = __shfl_sync(0xffffffffu, page[2], key & 31), p3 = __shfl_sync(0xffffffffu, page[3], key & 31);
            w = key < 64 ? (key < 32 ? p01 : p1) : key < 96 ? p2 : p3;
            z = t0 + key - page_of(P.pages, static_cast<uint32_t>(t0 + key)) * P.pages.page_size;
          }
          if constexpr (kBoundsChecked) {  // (its first and last row: where one is outside, row by row, which finds it again and reports it)
            const T* const from = pool + w * P.pages.page_stride + g.h * P.pages.head_stride + z * P.pages.tok_stride;
            const bool in = in_bounds(from, D, pool, P.pages.extent, nullptr, kSitePool) &&
                            in_bounds(from + (box - 1) * P.pages.tok_stride, D, pool, P.pages.extent, nullptr, kSitePool);
            boxes = __all_sync(0xffffffffu, in || half >= D / 64);
          }
        }
        if (boxes) {
          if constexpr (SRC == kShared) look(t + 1);
          if (i >= stages && !W.warp_wait(empty + 8u * stage, (i / stages - 1) & 1u)) {
            ok = false;
            break;
          }
          if (lane == 0) arrive_expecting(full + 8u * stage, C::TILE);
          __syncwarp();
          if (half < D / 64) bring_box(dst + half * kHalf + key * 128, map, half * 64, g.h * P.head_step, z, w, full + 8u * stage);
          if (lane != 0) bar_arrive(full + 8u * stage);
          continue;
        }
        if constexpr (SRC == kDense) {  // rows a stride apart
          const T* from = pool + g.b * P.pages.page_stride + g.h * P.pages.head_stride + (t0 + r0) * P.pages.tok_stride + piece * 8;
          if (i >= stages && !W.warp_wait(empty + 8u * stage, (i / stages - 1) & 1u)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll 8
            for (int j = 0; j < 32 / RPI; ++j, from += RPI * P.pages.tok_stride) {
              const int in32 = j * RPI + r0, r = u * 32 + in32;
              const bool is = (seen.w[u] >> in32 & 1u) != 0 && in_bounds(from, 8, pool, P.pages.extent, P.pages.status, kSitePool);
              copy16(dst + (piece >> 3) * kHalf + r * 128 + (((piece & 7) ^ (r & 7)) << 4), is ? from : pool, is ? 16 : 0);
            }
        } else {
          int64_t off[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            off[u] = -1;
            const int key = t0 + u * 32 + lane;
            if (!(seen.w[u] >> lane & 1u)) continue;
            off[u] = slot_offset(P.pages, page[u], key - page_of(P.pages, static_cast<uint32_t>(key)) * P.pages.page_size);
            if (off[u] < 0) atomicOr(P.pages.status, kErrInput);
            if (off[u] >= 0) off[u] += g.h * P.pages.head_stride;
            if (off[u] >= 0 && !in_bounds(pool + off[u], D, pool, P.pages.extent, P.pages.status, kSitePool)) off[u] = -1;
          }
          look(t + 1);
          if (i >= stages && !W.warp_wait(empty + 8u * stage, (i / stages - 1) & 1u)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll 8
            for (int j = 0; j < 32 / RPI; ++j) {
              const int in32 = j * RPI + r0, r = u * 32 + in32;
              const int64_t ro = __shfl_sync(0xffffffffu, off[u], in32);
              copy16(dst + (piece >> 3) * kHalf + r * 128 + (((piece & 7) ^ (r & 7)) << 4), pool + (ro >= 0 ? ro : 0) + piece * 8, ro >= 0 ? 16 : 0);
            }
        }
        copies_arrive(full + 8u * stage);
      }
      x += g.n;
    }
    // nothing is on its way to this CTA's memory any more (of interest where the others have given up)
    for (int j = max(i - stages, 0); j < i; ++j) W.drain(full + 8u * (j % stages), (j / stages) & 1u);
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 11) {
    // ---- Q: a segment's rows, once the products of the one before it in the same place are done
    constexpr int PIECES = D / 8, RPI = 32 / PIECES;
    const int piece = lane % PIECES, r0 = lane / PIECES;
    const T* const q = static_cast<const T*>(P.q) + piece * 8;
    int seg = 0;
    for (int x = x0; x < x1; ++seg) {
      const RowSeg g = row_seg<SRC>(P, plan, x, x1);
      const int buf = seg % C::QST;
      const uint32_t full = QFULL + 8u * buf;
      uint32_t dst = base + C::OFF_Q + buf * (QT * C::Q_TILE);
      if (P.q_box) {
        if (seg >= C::QST && !W.warp_wait_q(QEMPTY + 8u * buf, (seg / C::QST - 1) & 1u)) break;
        const int boxes = (QT == 2 && g.rows > kRowTile ? 2 : 1) * (D / 64);
        if (lane == 0) arrive_expecting(full, boxes * kHalf);
        __syncwarp();
        if (lane < boxes) {  // lane: a row tile and 64 of its dimensions
          const int tile = lane / (D / 64), half = lane % (D / 64);
          const int tok = (SRC == kShared ? plan.req0[g.b] : 0) + (g.rt * (P.item_rows / kRowTile) + tile) * P.q_box;
          bring_box(dst + tile * C::Q_TILE + half * kHalf, &P.q_map, half * 64, g.h * P.group, tok, SRC == kShared ? 0 : g.b, full);
        }
        if (lane != 0) bar_arrive(full);
        x += g.n;
        continue;
      }
      dst += (piece >> 3) * kHalf;
      // lane l works out the places of rows l, l + 32, ..
      int64_t off[QT * 4];
#pragma unroll
      for (int u = 0; u < QT * 4; ++u) off[u] = u * 32 + lane < g.rows ? row_q<SRC, D>(P, plan, g, u * 32 + lane) : -1;
      if (seg >= C::QST && !W.warp_wait_q(QEMPTY + 8u * buf, (seg / C::QST - 1) & 1u)) break;
#pragma unroll
      for (int u = 0; u < QT * 4; ++u) {
        if (QT == 2 && u >= 4 && g.rows <= kRowTile) break;
#pragma unroll 8
        for (int j = 0; j < 32 / RPI; ++j) {
          const int in32 = j * RPI + r0, r = (u & 3) * 32 + in32;
          const int64_t ro = __shfl_sync(0xffffffffu, off[u], in32);
          copy16(dst + (u >> 2) * C::Q_TILE + r * 128 + (((piece & 7) ^ (r & 7)) << 4), q + (ro >= 0 ? ro : 0), ro >= 0 ? 16 : 0);
        }
      }
      copies_arrive(full);
      x += g.n;
    }
    for (int j = max(seg - C::QST, 0); j < seg; ++j) W.drain(QFULL + 8u * (j % C::QST), (j / C::QST) & 1u);
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ---- the products.  Step u of a segment: stream u & 1; S(u + 2) follows P V(u), whose P lies over it
    constexpr uint32_t idesc_s = rows_idesc<T>(kKeyTile, false), idesc_o = rows_idesc<T>(D, true);
    const uint32_t one = one_lane();
    int seg = 0, kt = 0, vt = 0, qb = 0;     // segments so far, and the places of the next K, V and Q
    uint32_t kp = 0, vp = 0, qp = 0, np = 0; // parities: of the rings' rounds, and of each stream's P's (bit s)
    uint32_t ends = 0, used = 0;  // of each stream's O: parity of its ends, and whether there were any
    bool ok = true;
    for (int x = x0; x < x1 && ok; ++seg) {
      const RowSeg g = row_seg<SRC>(P, plan, x, x1);
      const bool two = QT == 2 && __shfl_sync(0xffffffffu, g.rows, 0) > kRowTile;
      const int steps = __shfl_sync(0xffffffffu, g.n, 0) << (two ? 1 : 0);
      auto issue_s = [&](int u) {
        const int s = u & 1;
        const bool opens = !two || s == 0, closes = !two || s == 1;  // the first and last use of the tile
        if (opens && !W.warp_wait(KFULL + 8u * kt, kp)) return false;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // copies (generic proxy) before the tensor cores' reads
        tc_after();
        const uint32_t a = desc_of(base + C::OFF_Q, 16) + (qb * QT * C::Q_TILE >> 4) + (two && s ? C::Q_TILE >> 4 : 0), b = desc_of(base + C::OFF_K, 16) + kt * (C::TILE >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t adv = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
          mma_ss(one, tmem + s * 128, a + adv, b + adv, idesc_s, k > 0);
        }
        commit(one, SFULL + 8u * s);
        if (closes) {
          commit(one, KEMPTY + 8u * kt);
          if (++kt == C::KST) kt = 0, kp ^= 1u;
        }
        if (u == steps - 1) commit(one, QEMPTY + 8u * qb);
        return true;
      };
      ok = W.warp_wait(QFULL + 8u * qb, qp) && issue_s(0) && (steps == 1 || issue_s(1));
      for (int u = 0; u < steps && ok; ++u) {
        const int s = u & 1;
        const bool opens = !two || s == 0, closes = !two || s == 1;
        ok = (!opens || W.warp_wait(VFULL + 8u * vt, vp)) && (u > 1 || !(used >> s & 1u) || W.warp_wait(OEMPTY + 8u * s, (ends >> s & 1u) ^ 1u)) &&
             W.warp_wait(PFULL + 8u * s, np >> s & 1u);
        if (!ok) break;
        np ^= 1u << s;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_after();
        const uint32_t a = tmem + s * 128, d = tmem + C::O_COL + s * D;
        const uint32_t b = desc_of(base + C::OFF_V, kHalf) + vt * (C::TILE >> 4);
#pragma unroll
        for (int k = 0; k < kKeyTile / 16; ++k)
          mma_ts(one, d, a + (k >> 1) * 32 + (k & 1) * 8, b + ((k * 2048) >> 4), idesc_o, (u >> 1) % kSumTiles != 0 || k > 0);
        if constexpr (QT == 1) {
#pragma unroll
          for (int k = 0; k < kKeyTile / 16; ++k) mma_ts(one, d, a + (k >> 1) * 32 + 16 + (k & 1) * 8, b + ((k * 2048) >> 4), idesc_o, true);
        }
        if (closes) {
          commit(one, VEMPTY + 8u * vt);
          if (++vt == C::VST) vt = 0, vp ^= 1u;
        }
        if (u + 2 >= steps) {  // the stream's last
          commit(one, OFULL + 8u * s);
          ends ^= 1u << s;
          used |= 1u << s;
        } else {
          ok = issue_s(u + 2);
        }
      }
      if (++qb == C::QST) qb = 0, qp ^= 1u;
      x += g.n;
    }
    // every product issued here has ended before the tensor memory is given back
    commit(one, DRAIN);
    W.drain(DRAIN, 0u);
    __syncwarp();
  }
  } else {
    // ---- softmax.  Thread: row `row` of its stream
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int s = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // 32 lanes a warp, in an address's upper half
    const uint32_t at_s = tmem + lanes + s * 128;
    float2* const s_ml = reinterpret_cast<float2*>(gbase + C::OFF_ML);
    uint4* const out = reinterpret_cast<uint4*>(gbase + C::OFF_OUT) + warp * 128;
    uint32_t ns = 0, no[2] = {0, 0};  // S's of this stream, and ends of both, so far
    bool ok = !P.expire || run_out(W, DRAIN);  // (once a wait has given up, all that follows is left out, but for the barriers of all softmax threads)
    for (int x = x0; x < x1;) {
      const RowSeg g = row_seg<SRC>(P, plan, x, x1);
      const bool two = QT == 2 && g.rows > kRowTile;
      const int steps = two ? 2 * g.n : g.n, mine = (steps + 1 - s) / 2;  // steps of this stream
      const int my_rows = two ? g.rows - s * kRowTile : g.rows;
      const bool busy = (warp & 3) * 32 < my_rows;  // this warp has rows
      float m = kNegInf, l = 0.f;
      for (int i = 0; i < mine && ok; ++i, ++ns) {
        const int t0 = (g.tile0 + (two ? i : 2 * i + s)) * kKeyTile;
        const bool all = (SRC != kDense || !P.mask) && t0 <= g.len - kKeyTile;  // (t0 + kKeyTile can be 2^31)
        Seen seen = {};
        if (!all) seen = keys_seen<SRC>(P, g, t0);
        if (!W.warp_wait(SFULL + 8u * s, ns & 1u)) {
          ok = false;
          break;
        }
        if (busy) {
          tc_after();
          if (i % kSumTiles == 0 && i > 0) put_sums<D>(tmem + lanes + C::O_COL + s * D, P.row_sums, P.row_refs, m, i == kSumTiles);  // (O holds all up to i - 1)
          const bool some = !all && (seen.w[0] & seen.w[1] & seen.w[2] & seen.w[3]) != ~0u;
          if (QT == 1 && some) hide_keys(at_s, seen);
          const uint64_t scale2 = pair(P.scale, P.scale);
          uint64_t sum[2] = {0, 0}, less2;
          auto move_reference = [&](float top) {  // where the row's largest score has passed it
            if (__any_sync(0xffffffffu, top > m + (kTau + Mma<T>::kLift))) {
              const float now = fmaxf(m, top - Mma<T>::kLift);
              const float f = now == kNegInf ? 1.f : ex2(m - now);
              m = now;
              l *= f;
              if (i > 0) scale_columns(tmem + lanes + C::O_COL + s * D, D, f);  // S(i) was issued behind P V(i - 1): O holds all up to it
            }
            const float less = m == kNegInf ? 0.f : -m;
            less2 = pair(less, less);
          };
          auto weights = [&](float& x, float& y, int k) {
            unpair(fma2(pair(x, y), scale2, less2), x, y);
            x = ex2(x);
            y = ex2(y);
            sum[k & 1] = add2(sum[k & 1], pair(x, y));
          };
          if constexpr (QT == 1) {
            // 32 columns at a time, and S read twice: the bytes of K and V leave the time for it, and there are a quarter of the
            // instructions, which what came before has often put out of the caches (the first tile of a launch 5 us, with all 128 unrolled 8)
            float top = kNegInf;
#pragma unroll 1
            for (int c = 0; c < kKeyTile; c += 32) {
              float v[32];
              tmem_read32<0>(at_s + c, v);
              top = fmaxf(top, max_of(v));
            }
            move_reference(top * P.scale);
#pragma unroll 1
            for (int c = 0; c < kKeyTile; c += 32) {
              float v[32];
              tmem_read32<0>(at_s + c, v);
              uint32_t hi[16], lo[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                weights(v[2 * k], v[2 * k + 1], k);
                Mma<T>::split(v[2 * k], v[2 * k + 1], hi[k], lo[k]);
              }
              // P of 32 keys, and what its rounding left, over the 32 columns of their S
              tmem_write16(at_s + c, hi);
              tmem_write16(at_s + c + 16, lo);
            }
          } else {
            float v[kKeyTile];
            tmem_read128(at_s, v);
            if (some) {  // (by hide_keys, 20% of the keys hidden: 4096 x 8192 tokens of 32 heads 480 us, so 440; none hidden: 320)
#pragma unroll
              for (int k = 0; k < kKeyTile; ++k) v[k] = seen.w[k / 32] >> (k % 32) & 1u ? v[k] : kNegInf;
            }
            move_reference(max_of(v) * P.scale);
#pragma unroll
            for (int c = 0; c < kKeyTile; c += 32) {
              uint32_t hi[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                weights(v[c + 2 * k], v[c + 2 * k + 1], k);
                hi[k] = Mma<T>::down2(v[c + 2 * k], v[c + 2 * k + 1]);
              }
              tmem_write16(at_s + c, hi);
            }
          }
          float a, b;
          unpair(add2(sum[0], sum[1]), a, b);
          l += a + b;
          tmem_written();
          tc_before();
        }
        bar_arrive(PFULL + 8u * s);
      }
      // ---- the segment's end
      const bool whole = g.tile0 == 0 && g.first + g.n == g.end;
      const int slot = blockIdx.x * 2 + (g.tile0 == 0 ? 1 : 0);
      const bool other = !two && steps > 1;  // the same rows' other half
      if (mine > kSumTiles && ok) {
        ok = W.warp_wait(OFULL + 8u * s, no[s] & 1u);
        if (ok && busy) {
          tc_after();
          take_sums<D>(tmem + lanes + C::O_COL + s * D, P.row_sums, P.row_refs, m);
          tc_before();
        }
      }
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
      if (busy) {
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
        if (!ok) l = f0 = __int_as_float(0x7fffffff);  // a wait gave up: whatever is in O, the row becomes NaN, here or where it is joined
        const bool mine_too = row < my_rows;
        const int r = two ? s * kRowTile + row : row;
        const int c0 = two ? 0 : s * (D / 2), c1 = two ? D : c0 + D / 2;
        RowOut at{0, 0};
        if (mine_too) at = row_out<SRC, D>(P, plan, g, r);
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
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
          if (whole && SRC == kDense) {
            // through shared memory, so that four lanes write 64 bytes of a row (a row a lane: 32 rows a store, and four
            // times as long).  16-byte pieces are permuted by the row: no two of a store's or a load's 8 lanes share a bank
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = l == 0.f ? 0u : Mma<T>::down2(o[k * 8 + 2 * e] * inv, o[k * 8 + 2 * e + 1] * inv);
              out[lane * 4 + (k ^ (lane >> 1 & 3))] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int from = k * 8 + (lane >> 2);
              const int64_t to = __shfl_sync(0xffffffffu, mine_too ? at.o : -1, from);
              const uint4 w = out[from * 4 + ((lane & 3) ^ (from >> 1 & 3))];
              if (to >= 0) *reinterpret_cast<uint4*>(static_cast<T*>(P.o) + to + c + (lane & 3) * 8) = w;
            }
            __syncwarp();
          } else if (!mine_too) {
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
      if (!two) ok = softmax_sync(ok);  // (both have read O and the states)
      if (mine > 0) bar_arrive(OEMPTY + 8u * s);
      x += g.n;
    }
  }
  if (SRC == kShared) grid_dependency_wait();
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS) : "memory");
}

// Merges the pieces of the items that more than one CTA worked on, each of which crosses a boundary between CTAs first.  A job: such an
// item, 32 of its rows and 32 dimensions; a CTA takes every nth.  A thread: a row (its lane) and four dimensions (its warp);
// eight pieces are fetched at a time with their states, and merged as they come (20 rows x 65536 keys of one item, 152 pieces: four at a
// time and four CTAs an SM 52 us, 45; 8 items of 20 pieces 36.0 and 35.4).
template <typename T, int SRC, int D>
__global__ void __launch_bounds__(kWarps * 32, 3) join_rows(const __grid_constant__ AttendParams P) {
  constexpr int AT_ONCE = 8, PARTS = D / 32;
  static_assert(kMaxCtas <= kWarps * 32, "a boundary for each thread");
  struct Item {
    int16_t b, pieces;
    int32_t h, rt, rows, c0;  // c0: the first CTA
  };
  __shared__ RowPlan plan;
  __shared__ Item items[kMaxCtas];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int T_all = build_row_plan<SRC>(P, plan, false);
  const RowSplit split(P, T_all);
  allow_dependents();
  int n_items;
  {
    const int c0 = threadIdx.x, x = c0 + 1 < static_cast<int>(split.used) ? split.begin(c0 + 1) : -1;
    RowSeg g{};
    if (x >= 0) g = row_seg_at<SRC>(P, plan, x);
    const bool is = x >= 0 && g.first < x && g.first >= split.begin(c0);
    const int at = block_scan(is, plan.warp_sum, n_items) - 1;
    if (is) items[at] = Item{static_cast<int16_t>(g.b), static_cast<int16_t>(split.of(g.end - 1) - c0 + 1), g.h, g.rt, g.rows, c0};
  }
  __syncthreads();
  grid_dependency_wait();
  const int per = P.item_rows / 32 * PARTS;
  for (int j = blockIdx.x; j < n_items * per; j += gridDim.x) {
    const Item& it = items[j / per];
    const int k = j % per, r = k / PARTS * 32 + lane, d4 = k % PARTS * 8 + warp;
    if (r >= it.rows) continue;  // (no lane is waited for below)
    const int pieces = it.pieces;
    // (slot 1 of the first CTA, slot 0 of the others)
    const float2* const ml = P.rows_ml + static_cast<int64_t>(it.c0) * 2 * P.item_rows + r;
    const float4* const po = P.rows_o + (static_cast<int64_t>(it.c0) * 2 * (D / 4) + d4) * P.item_rows + r;
    float M = kNegInf, L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int c = 0; c < pieces; c += AT_ONCE) {
      float2 s[AT_ONCE];
      float4 v[AT_ONCE];
#pragma unroll
      for (int u = 0; u < AT_ONCE; ++u) {
        const int slot = c + u == 0 ? 1 : 2 * (c + u);
        const bool is = c + u < pieces;
        s[u] = is ? __ldcg(ml + slot * P.item_rows) : make_float2(kNegInf, 0.f);
        v[u] = is ? __ldcg(po + static_cast<int64_t>(slot) * (D / 4) * P.item_rows) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float top = M;
#pragma unroll
      for (int u = 0; u < AT_ONCE; ++u) top = fmaxf(top, s[u].x);
      const float less = top == kNegInf ? 0.f : -top, back = ex2(M + less);
      M = top;
      L *= back;
      o = make_float4(o.x * back, o.y * back, o.z * back, o.w * back);
#pragma unroll
      for (int u = 0; u < AT_ONCE; ++u) {
        const float f = ex2(s[u].x + less);
        L = fmaf(s[u].y, f, L);
        o.x = fmaf(v[u].x, f, o.x);
        o.y = fmaf(v[u].y, f, o.y);
        o.z = fmaf(v[u].z, f, o.z);
        o.w = fmaf(v[u].w, f, o.w);
      }
    }
    RowSeg g{};
    g.b = it.b;
    g.h = it.h;
    g.rt = it.rt;
    write_row<T>(P, row_out<SRC, D>(P, plan, g, r), d4 * 4, M, L, o);
  }
}

// ------------------------------------------------------------------ host

// What splitting items over CTAs costs, their pieces written, read and joined, in tiles of a CTA: more where its pieces are 256 KiB
// each.  (128 items of 16 tiles, two row tiles, d = 128: whole 31 us, split 46; 256 of 32: 95 and 103; d = 64, 256 of 12: 40 and 47;
// 64 of 12: 21.8 and 21.4; 32 of 64 tiles: 89 and 39; one row tile, d = 128: 40 of 8: 16.6 and 17.8, 32 of 8: 16.5 and 15.1.)  By the most
// tiles of an item that the host knows of: of 152 items of up to 128 tiles, 8 of 128 and the others of one tile take 173 us, all of 128 204.
constexpr int kJoinTiles = 8, kJoinTilesLarge = 14, kJoinTilesOne = 6;

struct RowSizes {
  int32_t item_rows, ctas;
  int32_t least;  // tiles of a CTA (RowSplit)
  bool whole;     // no item is split over CTAs
  size_t rows_o, rows_ml, sums, refs, total;
};

// Rows of an item where the rows with the same keys are at most `rows`.
inline int item_rows_for(int64_t rows) { return rows > kRowTile ? 2 * kRowTile : kRowTile; }

// At most `most` CTAs for `items` items of up to `per` tiles, and where their pieces lie behind `at` bytes of a workspace.
// may_whole: items may stay whole, and their join go, where the CTA with the most work has little more of it than the
// others.
inline void size_rows(RowSizes* z, int64_t items, int64_t per, int item_rows, int head_dim, int most, size_t at, bool may_whole) {
  const int64_t tiles = items * per;
  z->item_rows = item_rows;
  most = std::min(most, kMaxCtas);
  const int join = item_rows == kRowTile ? kJoinTilesOne : head_dim == 128 ? kJoinTilesLarge : kJoinTiles;
  z->whole = may_whole && (items + most - 1) / most * per <= tiles / most + join;
  z->least = z->whole ? 1 : per >= 64 ? 4 : 2;
  z->ctas = static_cast<int32_t>(tiles ? std::min<int64_t>(most, tiles) : most);  // (without tiles: for the rows that have no keys)
  const size_t rows = static_cast<size_t>(z->ctas) * 2 * z->item_rows, sums = per > kSumTiles ? static_cast<size_t>(z->ctas) * 2 * kRowTile : 0;
  z->rows_o = up256(at);
  z->rows_ml = z->rows_o + (z->whole ? 0 : rows * head_dim * 4);  // (whole items leave no pieces)
  z->sums = z->rows_ml + (z->whole ? 0 : up256(rows * 8));
  z->refs = z->sums + sums * head_dim * 4;
  z->total = std::max(z->refs + sums * 4, z->rows_o + 256);
}
inline void place_rows(AttendParams& p, const RowSizes& z, char* ws) {
  p.rows_o = reinterpret_cast<float4*>(ws + z.rows_o);
  p.rows_ml = reinterpret_cast<float2*>(ws + z.rows_ml);
  p.row_sums = reinterpret_cast<float4*>(ws + z.sums);
  p.row_refs = reinterpret_cast<float*>(ws + z.refs);
  p.item_rows = z.item_rows;
  p.row_ctas = z.ctas;
  p.row_least = z.least;
  p.row_whole = z.whole;
  p.expire = expire_waits();
  p.group_inverse = 1.f / static_cast<float>(p.group);
}

// Tensor maps, where sizes and strides allow; what has none is copied row by row.
inline void make_maps(RowsParams& p, int src, int D, bool bf16) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static std::atomic<void*> known{nullptr};
  void* fn = known.load(std::memory_order_acquire);
  if (!fn) {
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess || !fn) {
      cudaGetLastError();
      return;
    }
    known.store(fn, std::memory_order_release);
  }
  // Dimensions (D, n[0], n[1], n[2]) with strides of s elements and boxes of (64, box[0], box[1], 1).  A dimension of one entry has any
  // stride; a stride of 0 over more has no map.
  auto encode = [&](CUtensorMap* map, const void* at, const int64_t (&n)[3], const int64_t (&s)[3], int b0, int b1) {
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(D)}, strides[3];
    for (int i = 0; i < 3; ++i) {
      if (n[i] < 1 || (n[i] > 1 && (s[i] <= 0 || s[i] >= int64_t{1} << 39))) return false;
      dims[i + 1] = static_cast<cuuint64_t>(n[i]);
      strides[i] = static_cast<cuuint64_t>(n[i] > 1 ? s[i] : D) * 2;
    }
    const cuuint32_t boxes[4] = {64, static_cast<cuuint32_t>(b0), static_cast<cuuint32_t>(b1), 1}, ones[4] = {1, 1, 1, 1};
    return reinterpret_cast<Encode>(fn)(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(at),
                                        dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  int box = kKeyTile;
  if (src == kShared)
    while (p.pages.page_size % box) box /= 2;
  // (a lane a box: 8 slots at least.  256 requests behind 16384 slots in pages of 24: in boxes 91 us, row by row 120)
  if (box >= 8 && p.pages.k) {
    p.head_step = p.pages.n_kv_heads > 1 && p.pages.head_stride != 0;
    p.page_step = p.pages.n_pages > 1 && p.pages.page_stride != 0;
    const int64_t n[3] = {p.head_step ? p.pages.n_kv_heads : 1, p.pages.page_size, p.page_step ? p.pages.n_pages : 1};
    const int64_t s[3] = {p.pages.head_stride, p.pages.tok_stride, p.pages.page_stride};
    if (encode(&p.k_map, p.pages.k, n, s, 1, box) && encode(&p.v_map, p.pages.v, n, s, 1, box)) p.box = box;
  }
  if (kRowTile % p.group == 0) {
    const int64_t one = static_cast<int64_t>(p.n_q) * D;
    const int64_t n[3] = {p.n_q, src == kShared ? p.pages.n_req : p.n_tok, src == kShared ? 1 : p.pages.n_req};
    const int64_t s[3] = {src == kShared ? D : p.q_h, src == kShared ? one : p.q_n, src == kShared ? one : p.q_b};
    if (encode(&p.q_map, p.q, n, s, p.group, kRowTile / p.group)) p.q_box = kRowTile / p.group;
  }
}

template <typename T, int SRC, int D, int QT>
cudaError_t launch_rows_of(const AttendParams& params, int device, cudaStream_t s) {
  RowsParams p = {};
  static_cast<AttendParams&>(p) = params;
  make_maps(p, SRC, D, std::is_same<T, __nv_bfloat16>::value);
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
