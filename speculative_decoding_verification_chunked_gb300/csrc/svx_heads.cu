// Norms of query and key heads with the position rotation, in one pass from a projection's output to a
// round's tensors or a paged cache.
//
//   y_i = x_i w_i / sqrt(mean(x^2) + eps)
//   (z_a, z_b) = s (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = pos * inv_freq   for each pair (a, b)
//
// All in fp32, rounded once at the end (a rounding between norm and rotation would be a second one).
//
// Phase.  t is needed mod 2 pi, and an fp32 product pos * inv_freq has lost it for far positions (2^17 * 2^-24 is
// 8e-3 rad).  The host keeps inv_freq / 2 pi as a 64-bit fraction of a turn, so pos * turns mod 2^64 is
// the fraction of a turn exactly, in three integer multiply-adds instead of FP64.  Its top bits name the nearest quarter
// turn, and what is left of all 64 goes to fp32 without cancelling, so that the smallest angle keeps its relative precision:
// a pair with y_a = 0 puts out y_b sin t alone, and is owed that to one rounding.  (The hardware's fast sine is within
// 2^-21 of any sine, however small: outputs of small angles were up to 9% off.)
//
// Layout.  A head is d / 16 lanes; a lane holds 16 elements as two 16-byte vectors, chosen so that both members
// of each rotated pair sit in one lane: vectors l and l + rot/16 of the rotated part, or two neighbouring vectors of the
// rest.  So a rotation needs no shuffle, a norm three (d = 128).  A warp takes 4 (d = 128) or 8 tokens and walks up to
// kMaxWalk heads of one kind (q, k or v) of them; a lane's eight angles and its weights become 32 factors once for the
// whole walk, which leaves three operations an element besides the sum of squares.  The walk's heads are all brought in at
// once, into shared memory, so the loads need no registers and do not wait for the sines.
// What bounds it: the copy rate.  32768 tokens of 32 + 8 + 8 heads, d = 128 (806 MB moved): 120 us = 6740 GB/s, 99% of the
// measured copy rate (138 us with four heads held ahead in registers, 210 us with angles and weights applied head by head).
// With few heads to a token the angles and a warp's start show: 106272 tokens of 4 + 2 + 2 heads, d = 64 (218 MB) 44 us
// (41 with the fast sine).  One token: 3.3 us, the latency of a launch and three trips to memory.
#include "svx_paged.h"

namespace svx {
namespace {

constexpr int kThreads = 64;
constexpr int kCtas = 12;  // per SM: 24 warps with 8 KiB each on the way
constexpr int kMaxWalk = 8;
constexpr int kGroup = 4;  // heads whose copies are waited for together

struct HeadsParams {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const void *q_norm, *k_norm;
  const int32_t* pos;
  const int32_t* n_new;
  int* status;
  void *q_out, *k_out, *v_out;  // k_out, v_out: dense; or NULL with a cache
  const int32_t* start;         // cache: first slot of each request's tokens
  float* acc;
  int32_t* slot_pos;
  PageView pages;
  uint64_t turns[64];
  int64_t tokens;               // n_req * n_tok
  int64_t q_ext, k_ext, v_ext;    // elements of the inputs (checked build)
  int64_t q_out_ext, kv_out_ext;  // and of the dense outputs
  float eps, scale;
  int32_t n_tok, n_q, n_kv;
  int32_t walk;                 // heads that a warp walks
  int32_t q_parts, kv_parts;    // warps per block of tokens for the heads of q, of k (and of v)
  uint32_t parts;               // all of them
  int32_t rot_dim, neighbours, norm, paged;
};

template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ float2 up(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t down(float a, float b) {
    __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&p);
  }
};
template <>
struct Pair<__half> {
  static __device__ __forceinline__ float2 up(uint32_t u) { return __half22float2(*reinterpret_cast<__half2*>(&u)); }
  static __device__ __forceinline__ uint32_t down(float a, float b) {
    __half2 p = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&p);
  }
};

template <typename T>
__device__ __forceinline__ void unpack(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = Pair<T>::up(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float* f) {
  return make_uint4(Pair<T>::down(f[0], f[1]), Pair<T>::down(f[2], f[3]), Pair<T>::down(f[4], f[5]),
                    Pair<T>::down(f[6], f[7]));
}

// Sine and cosine of 2 pi phase / 2^64, within 4 2^-24 of their own size: a quarter turn and a rest of at most pi/4, on which
// the Taylor series are summed to x^9 and x^8 (the next terms are 2^-28 of the sine and 2^-25 of the cosine).
__device__ __forceinline__ void turn_by(uint64_t phase, float& sn, float& cs) {
  const uint32_t hi = static_cast<uint32_t>(phase >> 32), lo = static_cast<uint32_t>(phase);
  const uint32_t quarter = (hi + 0x20000000u) >> 30;
  // the rest as a 32-bit high part, rounded, and a signed low part: no bits cancel where they are added
  const int32_t top = static_cast<int32_t>(hi - (quarter << 30)) + static_cast<int32_t>(lo >> 31);
  const float x = fmaf(static_cast<float>(top), 4294967296.f, static_cast<float>(static_cast<int32_t>(lo))) *
                  3.4061215800865545e-19f;  // 2 pi / 2^64
  const float u = x * x;
  const float s = fmaf(x * u, fmaf(u, fmaf(u, fmaf(u, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
  const float c = fmaf(u, fmaf(u, fmaf(u, fmaf(u, 1.f / 40320.f, -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
  sn = quarter & 1u ? c : s;
  cs = quarter & 1u ? s : c;
  if (quarter & 2u) sn = -sn;
  if ((quarter + 1u) & 2u) cs = -cs;
}

// RING: a walk of up to kMaxWalk heads, all of them on their way at once in shared memory; else one head, in registers.
template <typename T, int D, bool RING>
__global__ void __launch_bounds__(kThreads, kCtas) heads_kernel(const __grid_constant__ HeadsParams P) {
  constexpr int LANES = D / 16;       // lanes per head
  constexpr int TOKENS = 32 / LANES;  // tokens of a warp
  grid_dependency_wait();
  allow_dependents();
  const uint32_t gw = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const uint32_t block = gw / P.parts;
  const int part = static_cast<int>(gw - block * P.parts);  // which heads: the same for the whole warp
  const int lane = threadIdx.x % LANES;
  uint32_t token32 = block * TOKENS + (threadIdx.x & 31) / LANES;
  bool live = token32 < static_cast<uint32_t>(P.tokens);
  if (!live) token32 = 0;
  const int b = static_cast<int>(token32 / static_cast<uint32_t>(P.n_tok));
  const int j = static_cast<int>(token32) - b * P.n_tok;
  const int64_t token = token32;
  if (live && P.n_new) {
    const int n = P.n_new[b];
    if (P.status && (n < 0 || n > P.n_tok) && j == 0 && part == 0 && lane == 0) atomicOr(P.status, kErrInput);
    live = j < n;
  }
  // the part's heads: of q, of k or of v
  const bool is_q = part < P.q_parts, is_v = part >= P.q_parts + P.kv_parts;
  const int h0 = (is_q ? part : part - P.q_parts - (is_v ? P.kv_parts : 0)) * P.walk;
  const int count = min(P.walk, (is_q ? P.n_q : P.n_kv) - h0);
  const T* in = static_cast<const T*>(is_q ? P.q : is_v ? P.v : P.k);
  const int64_t in_ext = is_q ? P.q_ext : is_v ? P.v_ext : P.k_ext;
  const T* src = in + token * (is_q ? P.q_stride : is_v ? P.v_stride : P.k_stride) + static_cast<int64_t>(h0) * D;

  // this lane's vectors
  const int nvec = P.rot_dim / 16;  // vectors in one half of the rotated part
  const bool turn = lane < nvec;
  const int v0 = turn ? lane : 2 * nvec + 2 * (lane - nvec);
  const int v1 = turn ? lane + nvec : v0 + 1;
  // Every lane copies what it reads itself, so no lane waits for another.
  extern __shared__ uint4 ring[];
  const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) +
                        (threadIdx.x / 32 * (kMaxWalk * 64) + (threadIdx.x & 31)) * 16u;
  uint4 only[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  if constexpr (RING) {
#pragma unroll
    for (int i = 0; i < kMaxWalk; ++i) {
      if (live && i < count && in_bounds(src + i * D, D, in, in_ext, P.status, kSiteHeadsIn)) {
        const uint4* from = reinterpret_cast<const uint4*>(src + i * D);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(mine + i * 1024u), "l"(from + v0) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(mine + i * 1024u + 512u), "l"(from + v1) : "memory");
      }
      if (i % kGroup == kGroup - 1) asm volatile("cp.async.commit_group;" ::: "memory");
    }
  } else if (live && in_bounds(src, D, in, in_ext, P.status, kSiteHeadsIn)) {
    only[0] = __ldg(reinterpret_cast<const uint4*>(src) + v0);
    only[1] = __ldg(reinterpret_cast<const uint4*>(src) + v1);
  }
  // the walk's i-th head of this lane, once its group of copies has come in
  auto fetch = [&](int i, uint4 (&raw)[2]) {
    if constexpr (RING) {
      const uint4* at = ring + (threadIdx.x / 32 * (kMaxWalk * 64) + (threadIdx.x & 31)) + i * 64;
      raw[0] = at[0];
      raw[1] = at[32];
    } else {
      raw[0] = only[0];
      raw[1] = only[1];
    }
  };
  auto arrive = [&](int group) {  // group by group
    if constexpr (RING) {
      if (group == 0) asm volatile("cp.async.wait_group %0;" ::"n"(kMaxWalk / kGroup - 1) : "memory");
      else if (group == 1) asm volatile("cp.async.wait_group %0;" ::"n"(kMaxWalk / kGroup > 1 ? kMaxWalk / kGroup - 2 : 0) : "memory");
      else asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
  };

  // where the heads go: dst + i * step
  T* out = nullptr;
  int64_t at = -1, step = D, out_ext = 0;
  int32_t slot = 0;
  const int32_t pos = P.pos[token];
  if (is_q) {
    out = static_cast<T*>(P.q_out);
    step = static_cast<int64_t>(P.n_tok) * D;
    at = ((static_cast<int64_t>(b) * P.n_q + h0) * P.n_tok + j) * D;
    out_ext = P.q_out_ext;
  } else if (!P.paged) {
    out = static_cast<T*>(is_v ? P.v_out : P.k_out);
    at = (token * P.n_kv + h0) * D;
    out_ext = P.kv_out_ext;
  } else if (live) {
    out = static_cast<T*>(is_v ? P.pages.v : P.pages.k);
    step = P.pages.head_stride;
    out_ext = P.pages.extent;
    const int64_t s = static_cast<int64_t>(P.start[b]) + j;
    if (s >= 0 && s < P.pages.cap) {
      slot = static_cast<int32_t>(s);
      const uint32_t pg = page_of(P.pages, static_cast<uint32_t>(slot));
      at = slot_offset(P.pages, P.pages.table[static_cast<int64_t>(b) * P.pages.max_pages + pg],
                       static_cast<uint32_t>(slot) - pg * P.pages.page_size);
    }
    if (at < 0) {
      if (lane == 0) atomicOr(P.pages.status, kErrInput);
    } else {
      at += h0 * step;
    }
  }
  if (at < 0) live = false;
  const int out_site = P.paged && !is_q ? kSitePool : kSiteHeadsOut;

  const int walk = RING ? count : 1;
  if (is_v) {
    for (int i = 0; i < walk; ++i) {
      if (i % kGroup == 0) arrive(i / kGroup);
      uint4 raw[2];
      fetch(i, raw);
      T* dst = out + at + i * step;
      if (live && in_bounds(dst, D, out, out_ext, P.status, out_site)) {
        reinterpret_cast<uint4*>(dst)[v0] = raw[0];
        reinterpret_cast<uint4*>(dst)[v1] = raw[1];
      }
    }
    return;
  }

  // a lane's factors, weights included: z_a = r (x_a fa - x_b fb), z_b = r (x_b ga + x_a gb)
  // pairs 8 lane .. 8 lane + 7 (halves), or 4 v0 .. and 4 v1 .. (neighbours)
  float fa[8], fb[8], ga[8], gb[8];
  {
    float w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = 1.f;
    if (const T* wp = static_cast<const T*>(is_q ? P.q_norm : P.k_norm)) {
      unpack<T>(__ldg(reinterpret_cast<const uint4*>(wp) + v0), w);
      unpack<T>(__ldg(reinterpret_cast<const uint4*>(wp) + v1), w + 8);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float wa = P.neighbours && turn ? w[2 * i] : w[i], wb = P.neighbours && turn ? w[2 * i + 1] : w[8 + i];
      fa[i] = wa;
      ga[i] = wb;
      fb[i] = gb[i] = 0.f;
      if (turn) {
        const int f = P.neighbours ? (i < 4 ? 4 * v0 + i : 4 * v1 + i - 4) : 8 * lane + i;
        const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * P.turns[f];
        float sn, cs;
        turn_by(phase, sn, cs);
        sn *= P.scale;
        cs *= P.scale;
        fa[i] = wa * cs;
        fb[i] = wb * sn;
        ga[i] = wb * cs;
        gb[i] = wa * sn;
      }
    }
  }

  for (int i = 0; i < walk; ++i) {  // the same number of turns for all lanes
    if (i % kGroup == 0) arrive(i / kGroup);
    uint4 raw[2];
    fetch(i, raw);
    float x[16];
    unpack<T>(raw[0], x);
    unpack<T>(raw[1], x + 8);
    float r = 1.f;
    if (P.norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      r = rsqrtf(fmaf(ss, 1.f / D, P.eps));
    }
    if (!turn) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = x[e] * r * fa[e];
        x[8 + e] = x[8 + e] * r * ga[e];
      }
    } else if (P.neighbours) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = x[2 * e], c = x[2 * e + 1];
        x[2 * e] = (a * fa[e] - c * fb[e]) * r;
        x[2 * e + 1] = (c * ga[e] + a * gb[e]) * r;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = x[e], c = x[8 + e];
        x[e] = (a * fa[e] - c * fb[e]) * r;
        x[8 + e] = (c * ga[e] + a * gb[e]) * r;
      }
    }
    T* dst = out + at + i * step;
    if (!live || !in_bounds(dst, D, out, out_ext, P.status, out_site)) continue;
    reinterpret_cast<uint4*>(dst)[v0] = pack<T>(x);
    reinterpret_cast<uint4*>(dst)[v1] = pack<T>(x + 8);
    if (P.paged && !is_q && lane == 0) {
      const int64_t m = (static_cast<int64_t>(b) * P.n_kv + h0 + i) * P.pages.cap + slot;
      if (P.acc) P.acc[m] = 0.f;
      if (P.slot_pos) P.slot_pos[m] = pos;
    }
  }
}

template <typename T, int D>
cudaError_t launch(HeadsParams& p, cudaStream_t stream, int sms) {
  // Heads that a warp walks (its tokens' heads of one kind): one where tokens are few (latency: every head its own
  // warp), more once the grid half fills the card anyway, so that a lane's eight sines and cosines serve several heads.
  // Walks of 1, 2, 4 and 8, in us: 20436 tokens of 4 + 1 + 1 heads (d = 64) 13.3, 11.4, 10.3, 10.3 and 1024 tokens of
  // 32 + 8 + 8 (d = 128) 10.7, 8.3, 6.9, 6.2, eight taken in both.  Around one filling of the card it depends on where the last
  // warps fall, which the rule does not see: 2331 tokens of 12 + 3 + 3 (d = 64) 5.6, 5.4, 4.1, 5.2, two taken; 5 x 777 places,
  // 2331 of them live, 7.8, 6.8, 7.6, 7.2, four taken (dead places count: how many live is known on the device only).
  const int64_t blocks_of_tokens = (p.tokens * (D / 16) + 31) / 32;
  const int64_t room = static_cast<int64_t>(sms) * 32;  // warps
  const int64_t warps = blocks_of_tokens * (p.n_q + p.n_kv);
  p.walk = 1;
  while (p.walk < kMaxWalk && 2 * warps >= room * p.walk) p.walk *= 2;
  p.q_parts = (p.n_q + p.walk - 1) / p.walk;
  p.kv_parts = (p.n_kv + p.walk - 1) / p.walk;
  p.parts = p.q_parts + (p.v ? 2 : 1) * p.kv_parts;
  const int64_t blocks = (blocks_of_tokens * p.parts + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks));
  return p.walk > 1 ? launch_pdl(heads_kernel<T, D, true>, grid, dim3(kThreads), kThreads / 32 * kMaxWalk * 1024, stream, p)
                    : launch_pdl(heads_kernel<T, D, false>, grid, dim3(kThreads), 0, stream, p);
}

svx_status run_heads(const svx_heads* in, const svx_rope* rope, const svx_pages* cache, const int32_t* start, void* q_out,
                     void* k_out, void* v_out, float* acc, int32_t* slot_pos, void* stream) {
  if (!in || !rope) return paged_fail(SVX_ERR_INVALID_ARG, "heads or rope is NULL");
  if (in->n_req < 1 || in->n_req > kMaxReq) return paged_fail(SVX_ERR_INVALID_ARG, "n_req must be in [1, %d]", kMaxReq);
  if (in->n_tok < 1) return paged_fail(SVX_ERR_INVALID_ARG, "n_tok must be >= 1");
  if (in->head_dim != 64 && in->head_dim != 128) return paged_fail(SVX_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (in->dtype != SVX_BF16 && in->dtype != SVX_FP16)
    return paged_fail(SVX_ERR_UNSUPPORTED, "dtype must be SVX_BF16 or SVX_FP16");
  if (in->n_kv_heads < 1 || in->n_q_heads < in->n_kv_heads || in->n_q_heads % in->n_kv_heads || in->n_q_heads > 4096)
    return paged_fail(SVX_ERR_INVALID_ARG, "n_q_heads must be a positive multiple of n_kv_heads, at most 4096");
  if (rope->rot_dim < 0 || rope->rot_dim % 16 || rope->rot_dim > in->head_dim)
    return paged_fail(SVX_ERR_INVALID_ARG, "rope: rot_dim must be a multiple of 16, at most head_dim");
  const bool has_v = in->v != nullptr;
  const int d = in->head_dim;
  const int64_t q_row = static_cast<int64_t>(in->n_q_heads) * d, kv_row = static_cast<int64_t>(in->n_kv_heads) * d;
  const int64_t tokens = static_cast<int64_t>(in->n_req) * in->n_tok;
  if (tokens > 0x7fffffff) return paged_fail(SVX_ERR_UNSUPPORTED, "n_req * n_tok must be below 2^31");
  const int64_t most = (int64_t{1} << 46) / tokens;
  const int64_t str[3] = {in->q_stride, in->k_stride, in->v_stride}, row[3] = {q_row, kv_row, kv_row};
  for (int i = 0; i < (has_v ? 3 : 2); ++i)
    if (str[i] < row[i] || str[i] % 8 || str[i] > most)
      return paged_fail(SVX_ERR_INVALID_ARG, "token strides must be multiples of 8 elements that hold all heads");
  if (!in->q || !in->k || !q_out || !is_aligned(in->q, 16) || !is_aligned(in->k, 16) || !is_aligned(q_out, 16) ||
      (has_v && !is_aligned(in->v, 16)))
    return paged_fail(SVX_ERR_INVALID_ARG, "q, k, v and q_out must be 16-byte aligned device pointers");
  if (!in->pos) return paged_fail(SVX_ERR_INVALID_ARG, "pos must be a device pointer");
  if (!words_aligned({in->pos, in->n_new, in->status, start, acc, slot_pos}))
    return paged_fail(SVX_ERR_INVALID_ARG, "pos, n_new, status, start, acc and slot_pos must be 4-byte aligned");
  if (!(in->eps >= 0.f) && !(in->eps < 0.f)) return paged_fail(SVX_ERR_INVALID_ARG, "eps is not a number");
  if (in->eps < 0.f && (in->q_norm || in->k_norm))
    return paged_fail(SVX_ERR_INVALID_ARG, "norm weights given with eps < 0 (no norms)");
  if ((in->q_norm && !is_aligned(in->q_norm, 16)) || (in->k_norm && !is_aligned(in->k_norm, 16)))
    return paged_fail(SVX_ERR_INVALID_ARG, "norm weights must be 16-byte aligned");

  HeadsParams p = {};
  if (cache) {
    const svx_status st = paged_view(cache, in->n_req, &p.pages);
    if (st != SVX_OK) return st;
    if (cache->n_kv_heads != in->n_kv_heads || cache->head_dim != d || cache->dtype != in->dtype ||
        cache->device != in->device)
      return paged_fail(SVX_ERR_INVALID_ARG, "heads and cache differ in KV heads, head_dim, dtype or device");
    if (!start || !has_v) return paged_fail(SVX_ERR_INVALID_ARG, "start and v are required");
    if (pools_collide(cache, true)) return paged_fail(SVX_ERR_INVALID_ARG, "rows of the K and V pages share memory");
    p.paged = 1;
    p.status = cache->status;
  } else {
    if (!k_out || !is_aligned(k_out, 16) || has_v != (v_out != nullptr) || (v_out && !is_aligned(v_out, 16)))
      return paged_fail(SVX_ERR_INVALID_ARG, "k_out (and v_out with v) must be 16-byte aligned device pointers");
  }
  // (a strided input or pool takes what lies between its rows along: outputs there are refused alike)
  const size_t per_req = static_cast<size_t>(in->n_req) * 4, per_tok = static_cast<size_t>(tokens) * 4;
  auto span = [](const void* a, int64_t elems) { return Span{a, static_cast<size_t>(elems) * 2}; };
  const Span qi = span(in->q, (tokens - 1) * str[0] + row[0]), ki = span(in->k, (tokens - 1) * str[1] + row[1]),
             vi = has_v ? span(in->v, (tokens - 1) * str[2] + row[2]) : Span{nullptr, 0}, qo = span(q_out, tokens * q_row),
             wq = span(in->q_norm, d), wk = span(in->k_norm, d), pos = {in->pos, per_tok}, n_new = {in->n_new, per_req};
  bool bad;
  if (cache) {  // (the two pools may be interleaved)
    const size_t meta = static_cast<size_t>(in->n_req) * in->n_kv_heads * p.pages.cap * 4;
    const Span kp = span(cache->k, p.pages.extent), vp = span(cache->v, p.pages.extent);
    const Span first = {start, per_req}, table = {cache->table, per_req * cache->max_pages};
    bad = any_overlap({qo, {acc, meta}, {slot_pos, meta}, {cache->status, 4}},
                      {qi, ki, vi, kp, vp, wq, wk, pos, n_new, first, table});
    for (const Span& pool : {kp, vp}) bad = bad || any_overlap({pool}, {qi, ki, vi, wq, wk, pos, n_new, first, table});
  } else {
    bad = any_overlap({qo, span(k_out, tokens * kv_row), span(v_out, tokens * kv_row), {in->status, 4}},
                      {qi, ki, vi, wq, wk, pos, n_new});
  }
  if (bad) return paged_fail(SVX_ERR_INVALID_ARG, "an output overlaps an input or another output");

  PagedDevice dev(in->device);
  if (!dev.ok) return paged_fail(SVX_ERR_CUDA, "cannot use device %d", in->device);
  const void* ptrs[] = {in->q,   in->k,    in->v, in->q_norm, in->k_norm, in->pos, in->n_new, in->status,
                        q_out,   k_out,    v_out, start,      acc,        slot_pos, cache ? cache->k : nullptr,
                        cache ? cache->v : nullptr, cache ? cache->table : nullptr, cache ? cache->status : nullptr};
  for (const void* x : ptrs)
    if (x && !(in->flags & SVX_POINTERS_CHECKED) && !on_device(x, in->device))
      return paged_fail(SVX_ERR_INVALID_ARG, "a pointer is not memory of device %d", in->device);

  p.q = in->q;
  p.k = in->k;
  p.v = in->v;
  p.q_stride = str[0];
  p.k_stride = str[1];
  p.v_stride = str[2];
  p.q_norm = in->q_norm;
  p.k_norm = in->k_norm;
  p.pos = in->pos;
  p.n_new = in->n_new;
  if (!cache) p.status = in->status;
  p.q_out = q_out;
  p.k_out = k_out;
  p.v_out = v_out;
  p.start = start;
  p.acc = acc;
  p.slot_pos = slot_pos;
  for (int i = 0; i < 64; ++i) p.turns[i] = rope->turns[i];
  p.tokens = tokens;
  p.q_ext = clipped(kClipInputs, (tokens - 1) * str[0] + row[0]);
  p.k_ext = clipped(kClipInputs, (tokens - 1) * str[1] + row[1]);
  p.v_ext = has_v ? clipped(kClipInputs, (tokens - 1) * str[2] + row[2]) : 0;
  p.q_out_ext = clipped(kClipOutputs, tokens * q_row);
  p.kv_out_ext = clipped(kClipOutputs, tokens * kv_row);
  p.pages.extent = clipped(kClipPool, p.pages.extent);
  p.eps = in->eps;
  p.scale = rope->scale;
  p.n_tok = in->n_tok;
  p.n_q = in->n_q_heads;
  p.n_kv = in->n_kv_heads;
  p.rot_dim = rope->rot_dim;
  p.neighbours = rope->neighbours;
  p.norm = in->eps >= 0.f;
  const int sms = sm_count(in->device);
  if (sms <= 0) return paged_fail(SVX_ERR_CUDA, "cannot read the SM count");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (in->dtype == SVX_BF16)
    e = d == 128 ? launch<__nv_bfloat16, 128>(p, s, sms) : launch<__nv_bfloat16, 64>(p, s, sms);
  else
    e = d == 128 ? launch<__half, 128>(p, s, sms) : launch<__half, 64>(p, s, sms);
  if (e != cudaSuccess) return paged_fail(SVX_ERR_CUDA, "heads kernel launch failed: %s", cudaGetErrorString(e));
  return SVX_OK;
}

}  // namespace
}  // namespace svx

extern "C" svx_status svx_qk_norm_rope(const svx_heads* in, const svx_rope* rope, void* q_out, void* k_out, void* v_out,
                                       void* stream) {
  return svx::run_heads(in, rope, nullptr, nullptr, q_out, k_out, v_out, nullptr, nullptr, stream);
}

extern "C" svx_status svx_paged_append(const svx_heads* in, const svx_rope* rope, const svx_pages* cache,
                                       const int32_t* start, void* q_out, float* acc, int32_t* slot_pos, void* stream) {
  if (!cache) return svx::paged_fail(SVX_ERR_INVALID_ARG, "cache is NULL");
  return svx::run_heads(in, rope, cache, start, q_out, nullptr, nullptr, acc, slot_pos, stream);
}
