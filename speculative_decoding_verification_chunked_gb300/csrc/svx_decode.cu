// Attention of one new token per request over a paged cache.
//
//   s_t = scale q.k_t,  m = max s,  p_t = e^(s_t - m),  l = sum p,  O = sum p v / l,  LSE = m + ln l
//
// Every K and V row is used by the G query heads of its KV head and never again: 4 G flops an element read, so
// the bytes of K and V are the floor, and the kernel's task is to keep enough of them in flight.
//
// Work.  The slots of every (request, KV head, block of 16 query heads) - an item - are cut into chunks of
// 4 KiB of K; all items' chunks form one flat range, which is cut evenly over the CTAs ("stream-K"), so a
// ragged batch loads every SM alike, and one long request uses all of them.  The lengths are read on the device.
// An item that lies in one CTA is finished there; a piece of an item leaves (m, l, O) in the CTA's slot 0 (the item
// began before the CTA's range) or 1 (it goes on behind it), and join_kernel merges the pieces.
//
// A warp is its own pipeline: chunk i of a CTA's range belongs to warp i mod 8, which brings its chunks in with 16-byte
// cp.async (rows found through the page table, the next entry fetched a chunk ahead), kStages deep, with no
// barrier shared with the other warps.  8 warps x 2 chunks in flight are 128 KiB an SM.  The warps' states meet in
// shared memory at the end of an item's part only, while their next chunks are already on the way.
//
// Products: mma.sync m16n8k16, query heads on M.  They cost a few percent of the time (32 a chunk), so the
// tensor memory path, which wants 64 rows or more on M and a second trip through it, gains nothing here.  With up to 8
// query heads per KV head the upper 8 rows would be idle: they carry what is left of p after its rounding to 16 bits,
// so P.V has p to 16 bits or more at no extra product.  With 9 to 16 the remainder is a second product.
// Softmax state, scores and sums are fp32.  m is not the maximum but a reference that moves only when a score passes it
// by more than kTau, so most chunks need no exchange between lanes; every merge takes (m, l, O) with any reference.
#include "svx_paged.h"

#include <algorithm>
#include <atomic>

namespace svx {
namespace {

constexpr int kWarps = 8;
constexpr int kStages = 3;
constexpr int kChunkBytes = 4096;  // of K (and as much of V)
constexpr int kRowsMax = 16;       // query heads of an item
constexpr float kTau = 8.0f;       // p stays below 2^8
constexpr float kLn2 = 0.69314718055994530942f;
#define kNegInf (-INFINITY)

struct DecodeParams {
  PageView pages;
  const void* q;
  const int32_t* len;
  void* o;
  float* lse;
  const float* acc_in;
  float* acc_out;
  float* part_o;    // [ctas][2][16][D]
  float2* part_ml;  // [ctas][2][16]
  float2* row_ml;   // [n_req * n_q]: final (m, l), for the weights
  float* scores;    // [n_req * n_q][score_stride], log2 units
  int64_t score_stride;
  float scale;      // softmax scale * log2(e)
  int32_t max_len;
  int32_t n_q, group, blocks;  // blocks of 16 query heads per KV head
  int32_t min_chunks;          // a CTA takes at least this many (if there are)
  int32_t ctas;                // of the attention kernel
};

// The flat range of chunks, as every kernel of the call computes it from the lengths: first[b] is the first
// chunk of request b's items (KV head, block of query heads), first[kMaxReq] their number.
struct Plan {
  int64_t first[kMaxReq + 1];
  int64_t warp_sum[kWarps];
  uint8_t pad[kMaxReq];  // slots by which a request's length falls short of whole chunks
  // chunks of one of request b's items, and its length
  __device__ __forceinline__ int chunks(int b, int items) const {
    return static_cast<int>((first[b + 1] - first[b]) / items);
  }
};

template <int CT>
__device__ __forceinline__ int64_t build_plan(const DecodeParams& P, Plan& s, bool report) {
  // one request per thread (kMaxReq = threads of a block), prefix sum over the block
  static_assert(kMaxReq == kWarps * 32, "one thread per request");
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  int n = 0;
  if (t < P.pages.n_req) {
    const int raw = P.len[t];
    n = min(max(raw, 0), P.max_len);
    if (report && n != raw) atomicOr(P.pages.status, kErrInput);
  }
  const int chunks = (n + CT - 1) / CT;
  s.pad[t] = static_cast<uint8_t>(chunks * CT - n);
  const int64_t mine = static_cast<int64_t>(P.pages.n_kv_heads) * P.blocks * chunks;
  int64_t x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s.warp_sum[warp] = x;
  __syncthreads();
  int64_t base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int64_t v = s.warp_sum[w];
    if (w < warp) base += v;
    total += v;
  }
  s.first[t] = base + x - mine;
  if (t == 0) s.first[kMaxReq] = total;
  __syncthreads();
  return total;
}

// CTAs that share T chunks, and their ranges [c T / n, (c + 1) T / n).
__device__ __forceinline__ int64_t used_ctas(const DecodeParams& P, int64_t T) {
  const int64_t n = (T + P.min_chunks - 1) / P.min_chunks;
  return n < P.ctas ? n : P.ctas;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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
  static __device__ __forceinline__ uint2 down4(float4 v) {
    __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
    return make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
  }
};

template <int D>
struct Smem {
  static constexpr int OFF_O = kWarps * kStages * 2 * kChunkBytes;  // [8 warps][8 rows][D] partial outputs
  static constexpr int OFF_ML = OFF_O + kWarps * 8 * D * 4;         // [8 warps][8 rows] (m, l)
  static constexpr int BYTES = OFF_ML + kWarps * 8 * 8;
  // a row's float4 columns are permuted by the row, so that the fragments' stores spread over the banks
  static __device__ __forceinline__ int at(int w, int r, int d) { return (w * 8 + r) * D + ((d >> 2 ^ r) << 2) + (d & 3); }
};

// A place in the flat range: the item it lies in.
struct Cursor {
  int64_t first, end;  // the item's chunks
  int b, h, blk;       // request, KV head, block of query heads
  int len;
};

template <int CT>
__device__ __forceinline__ void seek(Cursor& c, const DecodeParams& P, const Plan& s, int64_t x) {
  // moves on to the item that holds x (x >= c.first); requests without chunks are passed over
  while (x >= s.first[c.b + 1]) ++c.b;
  const int n = s.chunks(c.b, P.pages.n_kv_heads * P.blocks);
  c.len = n * CT - s.pad[c.b];
  const int i = static_cast<int>((x - s.first[c.b]) / n);
  c.first = s.first[c.b] + static_cast<int64_t>(i) * n;
  c.end = c.first + n;
  c.h = i / P.blocks;
  c.blk = i - c.h * P.blocks;
}

template <typename T, int D, bool WIDE, bool SCORES>
__global__ void __launch_bounds__(kWarps * 32, 1) attend_kernel(const __grid_constant__ DecodeParams P) {
  constexpr int CT = kChunkBytes / (2 * D);  // slots of a chunk: 16 (d = 128) or 32 (d = 64)
  constexpr int NT = CT / 8;                 // score tiles
  constexpr int KS = D / 16;
  constexpr int NO = D / 8;                  // output tiles
  constexpr int PIECES = D / 8;              // 16-byte pieces of a row
  constexpr int RPI = 32 / PIECES;           // rows that a warp's 32 lanes copy at a time
  using S = Smem<D>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Plan plan;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  grid_dependency_wait();
  allow_dependents();
  const int64_t T_all = build_plan<CT>(P, plan, blockIdx.x == 0);

  // requests without slots: O = 0, LSE = -inf
  for (int b = blockIdx.x; b < P.pages.n_req; b += gridDim.x) {
    if (plan.first[b + 1] > plan.first[b]) continue;
    uint32_t* ob = reinterpret_cast<uint32_t*>(static_cast<T*>(P.o) + static_cast<int64_t>(b) * P.n_q * D);
    for (int i = tid; i < P.n_q * D / 2; i += blockDim.x) ob[i] = 0u;
    for (int i = tid; i < P.n_q; i += blockDim.x) P.lse[static_cast<int64_t>(b) * P.n_q + i] = kNegInf;
  }
  const int64_t used = used_ctas(P, T_all);
  if (static_cast<int64_t>(blockIdx.x) >= used) return;
  const int64_t x0 = cta_tile_begin(blockIdx.x, used, T_all), x1 = cta_tile_begin(blockIdx.x + 1, used, T_all);

  const uint32_t stage0 = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * (kStages * 2 * kChunkBytes);
  float* s_o = reinterpret_cast<float*>(smem + S::OFF_O);
  float2* s_ml = reinterpret_cast<float2*>(smem + S::OFF_ML);

  // ---- this warp's loads: chunk lx next; its rows' pages are looked up one chunk ahead
  const int my_row = lane % CT;  // the row of a chunk whose place this lane works out
  Cursor lc{0, 0, 0, 0, 0, 0};
  int64_t lx = x0 + warp;
  int look_page = -1, look_in = 0;
  bool look_live = false;
  auto look = [&]() {
    look_live = false;
    if (lx < x1) {
      if (lx >= lc.end) seek<CT>(lc, P, plan, lx);
      const int t = static_cast<int>(lx - lc.first) * CT + my_row;
      if (t < lc.len) {
        const uint32_t pg = static_cast<uint32_t>(t) / static_cast<uint32_t>(P.pages.page_size);
        look_in = t - pg * P.pages.page_size;
        look_page = __ldg(P.pages.table + static_cast<int64_t>(lc.b) * P.pages.max_pages + pg);
        look_live = true;
      }
    }
  };
  auto load = [&](int stage) {
    if (lx < x1) {
      int64_t off = -1;
      if (look_live) {
        off = slot_offset(P.pages, look_page, look_in);
        if (off < 0) atomicOr(P.pages.status, kErrInput);
        else off += static_cast<int64_t>(lc.h) * P.pages.head_stride;
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
        cp16(at, static_cast<const T*>(P.pages.k) + e, bytes);
        cp16(at + kChunkBytes, static_cast<const T*>(P.pages.v) + e, bytes);
      }
      lx += kWarps;
    }
    cp_commit();
  };
  look();
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    load(i);
    look();
  }

  // ---- the parts of items in this CTA's range
  const int g = lane >> 2, c2 = (lane & 3) * 2;
  int stage = 0;
  int64_t cx = x0 + warp;  // this warp's next chunk
  Cursor cc{0, 0, 0, 0, 0, 0};
  for (int64_t seg = x0; seg < x1; seg = cc.end) {
    seek<CT>(cc, P, plan, seg);
    const int64_t seg_end = cc.end < x1 ? cc.end : x1;
    const int rows = min(P.group - cc.blk * kRowsMax, kRowsMax);
    const int64_t row0 = static_cast<int64_t>(cc.b) * P.n_q + cc.h * P.group + cc.blk * kRowsMax;
    // q fragments: rows g and (WIDE) g + 8
    uint32_t qa[KS][WIDE ? 4 : 2];
    {
      const T* q0 = static_cast<const T*>(P.q) + (row0 + g) * D + c2;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qa[k][0] = g < rows ? __ldg(reinterpret_cast<const uint32_t*>(q0 + k * 16)) : 0u;
        qa[k][1] = g < rows ? __ldg(reinterpret_cast<const uint32_t*>(q0 + k * 16 + 8)) : 0u;
        if constexpr (WIDE) {
          qa[k][2] = g + 8 < rows ? __ldg(reinterpret_cast<const uint32_t*>(q0 + 8 * D + k * 16)) : 0u;
          qa[k][3] = g + 8 < rows ? __ldg(reinterpret_cast<const uint32_t*>(q0 + 8 * D + k * 16 + 8)) : 0u;
        }
      }
    }
    constexpr int H = WIDE ? 2 : 1;
    float m[H], l[H], acc[NO][4];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      m[h] = kNegInf;
      l[h] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < NO; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;

    for (; cx < seg_end; cx += kWarps) {
      cp_wait<kStages - 2>();
      __syncwarp();  // every lane's copies of this chunk are here, and every lane is done with the last one
      load(stage == 0 ? kStages - 1 : stage - 1);
      look();
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
      const int t0 = static_cast<int>(cx - cc.first) * CT;
      const int left = cc.len - t0;
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
            v = n * 8 + c2 + e < left ? v * P.scale : kNegInf;
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

    // ---- the warps' states meet, 8 query heads at a time
#pragma unroll
    for (int h = 0; h < H; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    const bool whole = cc.first >= x0 && cc.end <= x1;
    const int64_t slot = (static_cast<int64_t>(blockIdx.x) * 2 + (cc.first >= x0 ? 1 : 0)) * kRowsMax;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      if (h * 8 >= rows) break;  // the same for all threads
      if ((lane & 3) == 0) s_ml[warp * 8 + g] = make_float2(m[h], l[h]);
#pragma unroll
      for (int i = 0; i < NO; ++i) {
        float2 v = make_float2(acc[i][2 * h], acc[i][2 * h + 1]);
        if constexpr (!WIDE) {
          v.x += acc[i][2];
          v.y += acc[i][3];
        }
        *reinterpret_cast<float2*>(s_o + S::at(warp, g, i * 8 + c2)) = v;
      }
      __syncthreads();
      const int n_here = min(rows - h * 8, 8);
      for (int i = tid; i < n_here * (D / 4); i += kWarps * 32) {
        const int r = i / (D / 4), d4 = (i - r * (D / 4)) * 4;
        float M = kNegInf;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_ml[w * 8 + r].x);
        const float base = M == kNegInf ? 0.f : M;
        float L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 ml = s_ml[w * 8 + r];
          const float f = ex2(ml.x - base);
          const float4 v = *reinterpret_cast<const float4*>(s_o + S::at(w, r, d4));
          L = fmaf(ml.y, f, L);
          o.x = fmaf(v.x, f, o.x);
          o.y = fmaf(v.y, f, o.y);
          o.z = fmaf(v.z, f, o.z);
          o.w = fmaf(v.w, f, o.w);
        }
        const int64_t row = row0 + h * 8 + r;
        if (whole) {
          const float inv = L == 0.f ? 0.f : 1.f / L;
          o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
          if (L == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
          *reinterpret_cast<uint2*>(static_cast<T*>(P.o) + row * D + d4) = Mma<T>::down4(o);
          if (d4 == 0) {
            P.lse[row] = L == 0.f ? kNegInf : (M + log2f(L)) * kLn2;
            if constexpr (SCORES) P.row_ml[row] = make_float2(M, L);
          }
        } else {
          *reinterpret_cast<float4*>(P.part_o + (slot + h * 8 + r) * D + d4) = o;
          if (d4 == 0) P.part_ml[slot + h * 8 + r] = make_float2(M, L);
        }
      }
      __syncthreads();
    }
  }
  cp_wait<0>();
}

// Merges the pieces of the items that more than one CTA worked on: one CTA per item.
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) join_kernel(const __grid_constant__ DecodeParams P) {
  constexpr int CT = kChunkBytes / (2 * D);
  __shared__ Plan plan;
  grid_dependency_wait();
  allow_dependents();
  const int per = P.pages.n_kv_heads * P.blocks;
  const int b = blockIdx.x / per, i = blockIdx.x - b * per;
  const int64_t T_all = build_plan<CT>(P, plan, false);
  const int n = plan.chunks(b, per);
  if (n == 0) return;
  const int64_t used = used_ctas(P, T_all);
  const int64_t first = plan.first[b] + static_cast<int64_t>(i) * n;
  const int64_t c0 = cta_of_tile(first, used, T_all), c1 = cta_of_tile(first + n - 1, used, T_all);
  if (c0 == c1) return;
  const int h = i / P.blocks, blk = i - h * P.blocks;
  const int rows = min(P.group - blk * kRowsMax, kRowsMax);
  const int64_t row0 = static_cast<int64_t>(b) * P.n_q + h * P.group + blk * kRowsMax;
  const bool at_start = cta_tile_begin(c0, used, T_all) <= first;  // the item begins inside c0's range
  for (int x = threadIdx.x; x < rows * (D / 4); x += kWarps * 32) {
    const int r = x / (D / 4), d4 = (x - r * (D / 4)) * 4;
    float M = kNegInf, L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int64_t c = c0; c <= c1; ++c) {
      const int64_t s = (c * 2 + (c == c0 && at_start ? 1 : 0)) * kRowsMax + r;
      const float2 ml = P.part_ml[s];
      const float4 v = *reinterpret_cast<const float4*>(P.part_o + s * D + d4);
      const float t = fmaxf(M, ml.x);
      const float base = t == kNegInf ? 0.f : t;
      const float fa = ex2(M - base), fb = ex2(ml.x - base);
      L = L * fa + ml.y * fb;
      o.x = o.x * fa + v.x * fb;
      o.y = o.y * fa + v.y * fb;
      o.z = o.z * fa + v.z * fb;
      o.w = o.w * fa + v.w * fb;
      M = t;
    }
    const int64_t row = row0 + r;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    o = L == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(static_cast<T*>(P.o) + row * D + d4) = Mma<T>::down4(o);
    if (d4 == 0) {
      P.lse[row] = L == 0.f ? kNegInf : (M + log2f(L)) * kLn2;
      if (P.row_ml) P.row_ml[row] = make_float2(M, L);
    }
  }
}

// acc_out[t] = acc_in[t] + sum over a KV head's query heads of 2^(s_t - m) / l, from the stored scores.
__global__ void __launch_bounds__(256) weights_kernel(const __grid_constant__ DecodeParams P) {
  grid_dependency_wait();
  allow_dependents();
  const int bh = blockIdx.y, b = bh / P.pages.n_kv_heads, h = bh - b * P.pages.n_kv_heads;
  const int len = min(max(P.len[b], 0), P.max_len);
  const int t0 = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (t0 >= len) return;
  const int64_t row0 = static_cast<int64_t>(b) * P.n_q + static_cast<int64_t>(h) * P.group;
  float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int g = 0; g < P.group; ++g) {
    const float2 ml = P.row_ml[row0 + g];
    if (ml.y == 0.f) continue;  // only scores of -inf: no weight
    const float inv = 1.f / ml.y;
    const float4 s = *reinterpret_cast<const float4*>(P.scores + (row0 + g) * P.score_stride + t0);
    w.x = fmaf(ex2(s.x - ml.x), inv, w.x);
    w.y = fmaf(ex2(s.y - ml.x), inv, w.y);
    w.z = fmaf(ex2(s.z - ml.x), inv, w.z);
    w.w = fmaf(ex2(s.w - ml.x), inv, w.w);
  }
  const int64_t a = static_cast<int64_t>(bh) * P.pages.cap + t0;
  const float v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (t0 + e < len) P.acc_out[a + e] = P.acc_in[a + e] + v[e];
}

// ------------------------------------------------------------------ host

struct Sizes {
  int32_t max_len, blocks, ctas;
  int64_t score_stride;
  size_t part_o, part_ml, row_ml, scores, total;
};

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
  z->ctas = static_cast<int32_t>(std::min<int64_t>(sms, std::max<int64_t>(chunks, 1)));
  z->score_stride = (max_len + ct - 1) / ct * ct;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  z->part_o = 0;
  z->part_ml = z->part_o + up(static_cast<size_t>(z->ctas) * 2 * kRowsMax * c->head_dim * 4);
  z->row_ml = z->part_ml + up(static_cast<size_t>(z->ctas) * 2 * kRowsMax * 8);
  z->scores = z->row_ml + (weights ? up(static_cast<size_t>(n_req) * n_q * 8) : 0);
  z->total = z->scores + (weights ? up(static_cast<size_t>(n_req) * n_q * z->score_stride * 4) : 0);
  return SVX_OK;
}

constexpr int kMinChunks = 2 * kWarps;

template <typename T, int D, bool WIDE, bool SCORES>
cudaError_t launch_attend(const DecodeParams& p, int device, cudaStream_t s) {
  constexpr int bytes = Smem<D>::BYTES;
  // set on each device's first use; setting it twice is harmless
  static std::atomic<bool> done[64];
  if (device >= 64 || !done[device].load(std::memory_order_acquire)) {
    const cudaError_t e =
        cudaFuncSetAttribute(attend_kernel<T, D, WIDE, SCORES>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (device < 64) done[device].store(true, std::memory_order_release);
  }
  return launch_pdl(attend_kernel<T, D, WIDE, SCORES>, dim3(p.ctas), dim3(kWarps * 32), bytes, s, p);
}

template <typename T, int D>
cudaError_t launch_all(const DecodeParams& p, int device, cudaStream_t s) {
  const bool wide = p.group > 8, scores = p.scores != nullptr;
  cudaError_t e = wide ? (scores ? launch_attend<T, D, true, true>(p, device, s) : launch_attend<T, D, true, false>(p, device, s))
                       : (scores ? launch_attend<T, D, false, true>(p, device, s) : launch_attend<T, D, false, false>(p, device, s));
  if (e != cudaSuccess) return e;
  const int64_t items = static_cast<int64_t>(p.pages.n_req) * p.pages.n_kv_heads * p.blocks;
  e = launch_pdl(join_kernel<T, D>, dim3(static_cast<unsigned>(items)), dim3(kWarps * 32), 0, s, p);
  if (e != cudaSuccess || !scores) return e;
  return launch_pdl(weights_kernel, dim3((p.max_len + 1023) / 1024, p.pages.n_req * p.pages.n_kv_heads), dim3(256), 0, s, p);
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
  svx::DecodeParams p = {};
  svx_status st = svx::paged_view(cache, n_req, &p.pages);
  if (st != SVX_OK) return st;
  if ((acc_in == nullptr) != (acc_out == nullptr))
    return paged_fail(SVX_ERR_INVALID_ARG, "give both acc_in and acc_out, or neither");
  if (!q || !o || !lse || !len || !svx::is_aligned(q, 16) || !svx::is_aligned(o, 16) || !svx::is_aligned(lse, 4))
    return paged_fail(SVX_ERR_INVALID_ARG, "q, len, o and lse must be device pointers, q and o 16-byte aligned");
  if (!(scale >= 0.f) || scale > 3.0e38f) return paged_fail(SVX_ERR_INVALID_ARG, "scale must be positive and finite, or 0");
  svx::Sizes z = {};
  st = svx::sizes(cache, n_req, n_q_heads, max_len, acc_in != nullptr, &z);
  if (st != SVX_OK) return st;
  if (!workspace || !svx::is_aligned(workspace, 256) || workspace_bytes < static_cast<int64_t>(z.total))
    return paged_fail(SVX_ERR_INVALID_ARG, "workspace must be 256-byte aligned, of at least %zu bytes", z.total);
  svx::PagedDevice dev(cache->device);
  if (!dev.ok) return paged_fail(SVX_ERR_CUDA, "cannot use device %d", cache->device);
  const void* ptrs[] = {cache->k, cache->v, cache->table, cache->status, q, len, o, lse, acc_in, acc_out, workspace};
  for (const void* x : ptrs)
    if (x && !(cache->flags & SVX_POINTERS_CHECKED) && !svx::on_device(x, cache->device))
      return paged_fail(SVX_ERR_INVALID_ARG, "a pointer is not memory of device %d", cache->device);

  char* ws = static_cast<char*>(workspace);
  p.q = q;
  p.len = len;
  p.o = o;
  p.lse = lse;
  p.acc_in = acc_in;
  p.acc_out = acc_out;
  p.part_o = reinterpret_cast<float*>(ws + z.part_o);
  p.part_ml = reinterpret_cast<float2*>(ws + z.part_ml);
  p.row_ml = acc_in ? reinterpret_cast<float2*>(ws + z.row_ml) : nullptr;
  p.scores = acc_in ? reinterpret_cast<float*>(ws + z.scores) : nullptr;
  p.score_stride = z.score_stride;
  const double sc = scale > 0.f ? static_cast<double>(scale) : 1.0 / sqrt(static_cast<double>(cache->head_dim));
  p.scale = static_cast<float>(sc * 1.4426950408889634074);
  p.max_len = z.max_len;
  p.n_q = n_q_heads;
  p.group = n_q_heads / cache->n_kv_heads;
  p.blocks = z.blocks;
  p.min_chunks = svx::kMinChunks;
  p.ctas = z.ctas;
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
