// The residual stream between two blocks of a decoder layer, in one pass.
//
//   u  = y, or y rsqrt(mean y^2 + post_eps) post_norm       (the norm after the block)
//   h' = alpha h + beta act(gate) u                          (the gate, and the scaled residual sum)
//   x  = h' rsqrt(mean h'^2 + eps) norm                      (the norm before the next block)
//
// A row is held on the SM from its loads to its stores (kVec elements, 16 bytes of a 16-bit type, at a time), so that h, y and a
// gate per element are read once and h', x written once: those bytes are the floor.  Two sums over the row, each a
// shuffle within the warps and one exchange through shared memory between them.  Everything is fp32, rounded once on the way out; x is
// the norm of the unrounded h'.
//
// Blocks stay on their SM and take rows in turn, the next ones on their way through shared memory by cp.async, so that the loads of a
// row run under the sums of the one before it (a block a row and loads into registers: 32768 x 4096 with both norms and a gate per
// element 269 us, 20000 x 5120 295).
// What bounds it: the copy rate, 32768 x 4096 with both norms and a gate per element (1.34 GB) 215 to 222 us = 6040 to 6240 GB/s, 90 to 93%
// of the measured copy rate.  Rows that are not a power of two of threads keep fewer on their way: 20000 x 5120 with a gate per
// channel 152 us (80%), with a 32-bit stream 250 (73%); weights kept in shared memory, or three blocks an SM of 56 registers a thread, moved
// these by -6 to +2%.  Few rows: the start and whole turns of the blocks (4 us the first ones): 777 x 5128 17.5 us where the bytes are
// 7, one row 3.2.
#include "svx_paged.h"

#include <algorithm>
#include <atomic>
#include <cmath>

namespace svx {
namespace {

constexpr int kVec = 8;
constexpr int kMaxThreads = 512;  // (128 registers a thread)
constexpr int kMaxDim = 16384;

enum GateKind : int { kGateNone = 0, kGateScalar = 1, kGateRow = 2 };

struct ResidualParams {
  const void* h;
  const void* y;
  const void* gate;
  const void* norm;
  const void* post_norm;
  void* h_out;
  void* x_out;
  int64_t h_stride, y_stride, gate_stride, h_out_stride, x_stride;
  int64_t rows;
  int32_t vecs;  // of a row
  int32_t gate_kind, act;
  int32_t stages;  // rows that a block has on their way
  bool wide;       // (fp32) pieces of h_out lie on the grid of 32 bytes
  float alpha, beta, eps, post_eps;  // eps < 0: no such norm
  float inv_dim;
};

// Values are worked on two at a time (fp32 pairs: half the instructions, which took longer than the bytes).  kVec elements as they
// lie in memory: one 16-byte plane, or (fp32) two.
constexpr int kPairs = kVec / 2;
__device__ __forceinline__ uint64_t widen(__nv_bfloat16, uint32_t w) {
  return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint64_t widen(__half, uint32_t w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pair(f.x, f.y);
}
__device__ __forceinline__ uint32_t narrow(__nv_bfloat16, uint64_t x) {
  float a, b;
  unpair(x, a, b);
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint32_t narrow(__half, uint64_t x) {
  float a, b;
  unpair(x, a, b);
  const __half2 p = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}
template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, uint64_t (&f)[kPairs]) {
  f[0] = widen(T(), v.x), f[1] = widen(T(), v.y), f[2] = widen(T(), v.z), f[3] = widen(T(), v.w);
}
template <typename T>
struct Raw {
  static __device__ __forceinline__ void get(const uint4& a, const uint4&, uint64_t (&f)[kPairs]) { unpack<T>(a, f); }
  static __device__ __forceinline__ void store(T* p, const uint64_t (&f)[kPairs], bool) {
    *reinterpret_cast<uint4*>(p) = make_uint4(narrow(T(), f[0]), narrow(T(), f[1]), narrow(T(), f[2]), narrow(T(), f[3]));
  }
};
template <>
struct Raw<float> {
  static __device__ __forceinline__ void get(const uint4& a, const uint4& b, uint64_t (&f)[kPairs]) {
    const uint32_t w[kVec] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < kPairs; ++e) f[e] = pair(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
  }
  static __device__ __forceinline__ void store(float* p, const uint64_t (&f)[kPairs], bool wide) {
    if (wide) {  // a whole sector
      asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(p), "l"(f[0]), "l"(f[1]), "l"(f[2]), "l"(f[3]) : "memory");
      return;
    }
    float v[kVec];
#pragma unroll
    for (int e = 0; e < kPairs; ++e) unpair(f[e], v[2 * e], v[2 * e + 1]);
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};

__device__ __forceinline__ uint64_t both(float x) { return pair(x, x); }
// 2^x and 1 / x, each within 2^-22 of itself
__device__ __forceinline__ uint64_t exp2_2(uint64_t x) {
  float a, b;
  unpair(x, a, b);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
  return pair(a, b);
}
__device__ __forceinline__ uint64_t inverse2(uint64_t x) {
  float a, b;
  unpair(x, a, b);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
  return pair(a, b);
}
// tanh and the sigmoid, within 2^-19 of themselves; the sigmoid loses up to 2^-17 where it is below e^-60 (its argument's product
// with log2 e is off by 2^-24 of itself).  tanh: 1 - 2 / (1 + e^2g), and where that cancels, below 1/4, the series up to g^9.
__device__ __forceinline__ uint64_t activate2(uint64_t g, int act) {
  constexpr float kLog2e = 1.44269504089f;
  if (act == SVX_ACT_SIGMOID) return inverse2(add2(both(1.f), exp2_2(mul2(g, both(-kLog2e)))));
  if (act == SVX_ACT_TANH) {
    const uint64_t far = fma2(both(-2.f), inverse2(add2(both(1.f), exp2_2(mul2(g, both(2.f * kLog2e))))), both(1.f));
    const uint64_t x = mul2(g, g);
    uint64_t s = fma2(x, both(62.f / 2835.f), both(-17.f / 315.f));
    s = fma2(x, s, both(2.f / 15.f));
    s = fma2(x, s, both(-1.f / 3.f));
    s = fma2(mul2(x, s), g, g);
    float g0, g1, f0, f1, s0, s1;
    unpair(g, g0, g1);
    unpair(far, f0, f1);
    unpair(s, s0, s1);
    return pair(fabsf(g0) < 0.25f ? s0 : f0, fabsf(g1) < 0.25f ? s1 : f1);
  }
  return g;
}

// The sum over the threads of a row: LANES of a warp, or (0) the block (every thread gets it; `s`: not the last call's).
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float* s) {
#pragma unroll
  for (int o = LANES ? LANES / 2 : 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (LANES == 0) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) s[warp] = v;
    __syncthreads();
    v = lane < (blockDim.x >> 5) ? s[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}

__device__ __forceinline__ void bring16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void brought(int newer) {  // all but the `newer` last groups are in
  if (newer == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (newer == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 2;" ::: "memory");
}

// T: block outputs and weights; H: the residual stream.  LANES: a row to so many lanes of a warp, or (0) to each block.  N: the most
// kVec-element pieces of a row that a thread holds.  A block takes every gridDim.x-th row (or as many at a time as it has).  Rows come in through shared
// memory, P.stages of them ahead; a thread brings in what it will read itself, or (32-bit h) its warp does, so no warp waits for another's
// copies.
template <typename T, typename H, int LANES, int N>
__global__ void __launch_bounds__(LANES ? 128 : kMaxThreads, LANES ? 8 : N > 2 ? 1 : 2) residual_kernel(const __grid_constant__ ResidualParams P) {
  constexpr int HP = sizeof(H) / 2;  // 16-byte planes of a piece of h
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float s_sum[2][32];
  constexpr int LANE_ROWS = LANES ? 32 / LANES : 1;  // rows of a warp
  constexpr int PER = LANES ? LANES : 1;
  const int threads = blockDim.x, t = LANES ? threadIdx.x % PER : threadIdx.x, step = LANES ? LANES : threads;
  const int64_t rows_at_once = LANES ? static_cast<int64_t>(gridDim.x) * (threads / PER) : gridDim.x;
  int64_t row = LANES ? static_cast<int64_t>(blockIdx.x) * (threads / PER) + threadIdx.x / PER : blockIdx.x;
  const int nth = LANES ? (threadIdx.x & 31) / PER : 0;  // this thread's row among its warp's, whose loop ends with the first of them
  // planes of 16 bytes a thread: [stage][piece][y, h (one or two), gate]
  const bool has_y = P.y != nullptr, has_g = P.gate_kind == kGateRow && P.gate_stride != 0;
  const int planes = HP + (has_y ? 1 : 0) + (has_g ? 1 : 0);
  auto plane = [&](int stage, int i, int k) { return ((stage * N + i) * planes + k) * threads + static_cast<int>(threadIdx.x); };
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  const uint4* const held = reinterpret_cast<const uint4*>(smem);
  auto bring = [&](int64_t r, int stage) {
    if (r < P.rows) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = t + i * step;
        if (v >= P.vecs) continue;
        if constexpr (HP == 1) bring16(base + plane(stage, i, 0) * 16, static_cast<const H*>(P.h) + r * P.h_stride + v * kVec);
        if (has_y) bring16(base + plane(stage, i, HP) * 16, static_cast<const T*>(P.y) + r * P.y_stride + v * kVec);
        if (has_g) bring16(base + plane(stage, i, planes - 1) * 16, static_cast<const T*>(P.gate) + r * P.gate_stride + v * kVec);
      }
    }
    // two planes of a thread: a warp's copies in order of their addresses, 512 bytes at a time (its own 32 a thread would fetch
    // every sector twice)
    if (HP == 2 && (LANE_ROWS > 1 || r < P.rows)) {
      const int lane = threadIdx.x & 31;
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int c = q * 32 + lane, other = (c >> 1) - lane;
          const int v = (LANE_ROWS > 1 ? (c >> 1) % PER : t + other) + i * step;
          const int64_t ro = r + (LANE_ROWS > 1 ? (c >> 1) / PER - nth : 0);
          if (v < P.vecs && (LANE_ROWS == 1 || ro < P.rows))
            bring16(base + (plane(stage, i, c & 1) + other) * 16, static_cast<const H*>(P.h) + ro * P.h_stride + v * kVec + (c & 1) * 4);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  grid_dependency_wait();
  allow_dependents();
  for (int k = 0; k < P.stages; ++k) bring(row + k * rows_at_once, k);
  float scalar = P.beta;
  if (P.gate_kind == kGateScalar) {
    float a, b;
    unpair(activate2(both(static_cast<float>(*static_cast<const T*>(P.gate))), P.act), a, b);
    scalar *= a;
  }
  // sums use two places in turn: one is written again only behind the other's barrier, when all have read it
  int place = 0, stage = 0;
  for (; row - nth < P.rows; row += rows_at_once) {
    const int vecs = LANE_ROWS > 1 && row >= P.rows ? 0 : P.vecs;
    brought(P.stages - 1);
    if constexpr (HP == 2) __syncwarp();
    uint64_t z[N][kPairs], u[N][kPairs];  // h' and the block's output; of pieces past the row's end: zeros
    uint64_t sum2 = 0;
    float lo, hi;
    float factor = scalar;
    if (has_y) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (t + i * step < vecs) unpack<T>(held[plane(stage, i, HP)], u[i]);
        else u[i][0] = u[i][1] = u[i][2] = u[i][3] = 0;
      }
      if (P.post_eps >= 0.f) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int e = 0; e < kPairs; ++e) sum2 = fma2(u[i][e], u[i][e], sum2);
        unpair(sum2, lo, hi);
        factor *= rsqrtf(fmaf(row_sum<LANES>(lo + hi, s_sum[place]), P.inv_dim, P.post_eps));
        place ^= 1;
      }
    }
    sum2 = 0;
    const uint64_t factor2 = both(factor), alpha2 = both(P.alpha);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int v = t + i * step;
      if (v >= vecs) continue;
      Raw<H>::get(held[plane(stage, i, 0)], held[plane(stage, i, HP - 1)], z[i]);
      if (has_y) {
        uint64_t w[kPairs];
        if (P.post_norm) {
          unpack<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(P.post_norm) + v * kVec), w);
#pragma unroll
          for (int e = 0; e < kPairs; ++e) u[i][e] = mul2(u[i][e], w[e]);
        }
        if (P.gate_kind == kGateRow) {
          unpack<T>(has_g ? held[plane(stage, i, planes - 1)] : *reinterpret_cast<const uint4*>(static_cast<const T*>(P.gate) + v * kVec), w);
#pragma unroll
          for (int e = 0; e < kPairs; ++e) u[i][e] = mul2(u[i][e], activate2(w[e], P.act));
        }
#pragma unroll
        for (int e = 0; e < kPairs; ++e) z[i][e] = fma2(z[i][e], alpha2, mul2(u[i][e], factor2));
      } else {
#pragma unroll
        for (int e = 0; e < kPairs; ++e) z[i][e] = mul2(z[i][e], alpha2);
      }
#pragma unroll
      for (int e = 0; e < kPairs; ++e) sum2 = fma2(z[i][e], z[i][e], sum2);
    }
    if constexpr (HP == 2) __syncwarp();
    bring(row + P.stages * rows_at_once, stage);  // (into places that this thread, or its warp, has read)
    stage = stage + 1 == P.stages ? 0 : stage + 1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int v = t + i * step;
      if (v < vecs && P.h_out) Raw<H>::store(static_cast<H*>(P.h_out) + row * P.h_out_stride + v * kVec, z[i], P.wide);
    }
    if (!P.x_out) continue;
    unpair(sum2, lo, hi);
    const uint64_t r = both(rsqrtf(fmaf(row_sum<LANES>(lo + hi, s_sum[place]), P.inv_dim, P.eps)));
    place ^= 1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int v = t + i * step;
      if (v >= vecs) continue;
#pragma unroll
      for (int e = 0; e < kPairs; ++e) z[i][e] = mul2(z[i][e], r);
      if (P.norm) {
        uint64_t w[kPairs];
        unpack<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(P.norm) + v * kVec), w);
#pragma unroll
        for (int e = 0; e < kPairs; ++e) z[i][e] = mul2(z[i][e], w[e]);
      }
      Raw<T>::store(static_cast<T*>(P.x_out) + row * P.x_stride + v * kVec, z[i], false);
    }
  }
  brought(0);
}

constexpr int kSmem = 200 * 1024;  // of rows on their way, of an SM

template <typename T, typename H, int LANES, int N>
cudaError_t launch_of(ResidualParams p, int threads, int device, cudaStream_t s) {
  static std::atomic<bool> done[64];
  if (device >= 64 || !done[device].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(residual_kernel<T, H, LANES, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (device < 64) done[device].store(true, std::memory_order_release);
  }
  const int planes = sizeof(H) / 2 + (p.y ? 1 : 0) + (p.gate_kind == kGateRow && p.gate_stride ? 1 : 0);
  const int bytes = threads * N * planes * 16;  // of a stage
  const int at_once = LANES ? threads / (LANES ? LANES : 1) : 1;  // rows of a block
  const int64_t blocks = (p.rows + at_once - 1) / at_once;
  const int sms = sm_count(device), resident = std::min(std::max(1024 / threads, 1), kSmem / bytes);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(blocks, static_cast<int64_t>(std::max(sms, 1)) * resident));
  p.stages = std::min<int64_t>(std::min(kSmem / (resident * bytes), 3), (blocks + grid - 1) / grid);
  return launch_pdl(residual_kernel<T, H, LANES, N>, dim3(grid), dim3(threads), p.stages * bytes, s, p);
}

template <typename T, typename H>
cudaError_t launch_residual(const ResidualParams& p, int device, cudaStream_t s) {
  // A warp holds rows of up to 512 elements, or several shorter ones (67108864 elements with a gate per element, d = 64: a row to a warp
  // 405 us, four 127; d = 120: 223, two 129); else a block does, two pieces to a thread, but one where two would leave more idle (d = 520:
  // 195 us, 176; d = 768: 137, 125; with more than four warps the other way round, d = 2056: 139, 154), and three or four of long rows
  // (d = 12288: three 137 us, four 143).
  if (p.vecs <= 8) return launch_of<T, H, 8, 1>(p, 128, device, s);
  if (p.vecs <= 16) return launch_of<T, H, 16, 1>(p, 128, device, s);
  if (p.vecs <= 32) return launch_of<T, H, 32, 1>(p, 128, device, s);
  if (p.vecs <= 64) return launch_of<T, H, 32, 2>(p, 128, device, s);
  auto threads = [&](int n) { return ((p.vecs + n - 1) / n + 31) / 32 * 32; };
  if (p.vecs <= 128 && threads(1) < 2 * threads(2)) return launch_of<T, H, 0, 1>(p, threads(1), device, s);
  if (p.vecs <= 1024) return launch_of<T, H, 0, 2>(p, threads(2), device, s);
  if (p.vecs <= 1536) return launch_of<T, H, 0, 3>(p, threads(3), device, s);
  return launch_of<T, H, 0, 4>(p, 512, device, s);
}

}  // namespace
}  // namespace svx

extern "C" svx_status svx_residual_norm(const svx_residual* in, void* stream) {
  using svx::paged_fail;
  if (!in) return paged_fail(SVX_ERR_INVALID_ARG, "the arguments are NULL");
  const svx_residual& a = *in;
  if (a.dtype != SVX_BF16 && a.dtype != SVX_FP16)
    return paged_fail(SVX_ERR_UNSUPPORTED, "dtype must be SVX_BF16 or SVX_FP16");
  if (a.stream_dtype != a.dtype && a.stream_dtype != SVX_FP32)
    return paged_fail(SVX_ERR_UNSUPPORTED, "the residual stream's type must be dtype or SVX_FP32");
  if (a.dim < 8 || a.dim % 8 || a.dim > svx::kMaxDim)
    return paged_fail(SVX_ERR_UNSUPPORTED, "dim must be a multiple of 8 in [8, %d]", svx::kMaxDim);
  if (a.rows < 1 || a.rows > 0x7fffffff) return paged_fail(SVX_ERR_INVALID_ARG, "rows must be in [1, 2^31)");
  if (!a.h) return paged_fail(SVX_ERR_INVALID_ARG, "h is NULL");
  if (!a.h_out && !a.x_out) return paged_fail(SVX_ERR_INVALID_ARG, "h_out and x_out are both NULL");
  if (a.gate_kind < SVX_GATE_NONE || a.gate_kind > SVX_GATE_ELEMENT || a.act < SVX_ACT_NONE || a.act > SVX_ACT_SIGMOID)
    return paged_fail(SVX_ERR_INVALID_ARG, "unknown gate_kind or act");
  if ((a.gate_kind != SVX_GATE_NONE) != (a.gate != nullptr))
    return paged_fail(SVX_ERR_INVALID_ARG, "a gate needs its kind, and a kind its gate");
  if (a.act != SVX_ACT_NONE && !a.gate) return paged_fail(SVX_ERR_INVALID_ARG, "act needs a gate");
  if (!a.y && (a.gate || a.post_eps >= 0.f)) return paged_fail(SVX_ERR_INVALID_ARG, "a gate and a norm after the block need y");
  if (!std::isfinite(a.alpha) || !std::isfinite(a.beta) || !std::isfinite(a.eps) || !std::isfinite(a.post_eps))
    return paged_fail(SVX_ERR_INVALID_ARG, "alpha, beta, eps and post_eps must be finite");
  if (a.x_out && !(a.eps >= 0.f)) return paged_fail(SVX_ERR_INVALID_ARG, "eps must be >= 0");
  if (a.norm && !a.x_out) return paged_fail(SVX_ERR_INVALID_ARG, "norm needs x_out");
  if (a.post_norm && !(a.post_eps >= 0.f)) return paged_fail(SVX_ERR_INVALID_ARG, "post_norm needs post_eps >= 0");
  for (const void* p : {a.h, a.y, a.norm, a.post_norm, static_cast<const void*>(a.h_out), static_cast<const void*>(a.x_out)})
    if (!svx::is_aligned(p, 16)) return paged_fail(SVX_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
  if (!svx::is_aligned(a.gate, a.gate_kind == SVX_GATE_SCALAR ? 2 : 16))
    return paged_fail(SVX_ERR_INVALID_ARG, "the gate must be 16-byte aligned (a scalar: 2)");
  const size_t stream_size = a.stream_dtype == SVX_FP32 ? 4 : 2;
  const int64_t most = (int64_t{1} << 60) / a.rows;
  struct {
    const void* p;
    int64_t stride;
    bool out;
  } rows[] = {{a.h, a.h_stride, false}, {a.y, a.y_stride, false}, {a.gate_kind == SVX_GATE_ELEMENT ? a.gate : nullptr, a.gate_stride, false},
              {a.h_out, a.h_out_stride, true}, {a.x_out, a.x_stride, true}};
  for (const auto& r : rows)
    if (r.p && a.rows > 1 && (r.stride < (r.out ? a.dim : 0) || r.stride % 8 || r.stride > most))
      return paged_fail(SVX_ERR_INVALID_ARG, "row strides must be multiples of 8 elements, those of outputs at least dim");
  auto span = [&](const void* p, int64_t stride, size_t size) {
    return svx::Span{p, static_cast<size_t>((a.rows - 1) * (a.rows > 1 ? stride : 0) + a.dim) * size};
  };
  const bool h_in_place = a.h_out == a.h && (a.rows == 1 || a.h_out_stride == a.h_stride);
  const bool y_in_place = a.y && a.x_out == a.y && (a.rows == 1 || a.x_stride == a.y_stride);
  const svx::Span h = span(a.h, a.h_stride, stream_size), y = span(a.y, a.y_stride, 2);
  const svx::Span gate = {a.gate, a.gate_kind == SVX_GATE_SCALAR    ? 2
                                  : a.gate_kind == SVX_GATE_CHANNEL ? static_cast<size_t>(a.dim) * 2
                                                                    : span(a.gate, a.gate_stride, 2).bytes};
  const svx::Span h_out = span(a.h_out, a.h_out_stride, stream_size), x_out = span(a.x_out, a.x_stride, 2);
  const svx::Span weights[2] = {{a.norm, static_cast<size_t>(a.dim) * 2}, {a.post_norm, static_cast<size_t>(a.dim) * 2}};
  const svx::Span none = {nullptr, 0};
  if (svx::any_overlap({h_out}, {x_out, h_in_place ? none : h, y, gate, weights[0], weights[1]}) ||
      svx::any_overlap({x_out}, {h, y_in_place ? none : y, gate, weights[0], weights[1]}))
    return paged_fail(SVX_ERR_INVALID_ARG, "an output overlaps an input or the other output (h_out may be h, x_out may be y)");
  svx::PagedDevice dev(a.device);
  if (!dev.ok) return paged_fail(SVX_ERR_CUDA, "cannot use device %d", a.device);
  for (const void* p : {a.h, a.y, a.gate, a.norm, a.post_norm, static_cast<const void*>(a.h_out), static_cast<const void*>(a.x_out)})
    if (p && !(a.flags & SVX_POINTERS_CHECKED) && !svx::on_device(p, a.device))
      return paged_fail(SVX_ERR_INVALID_ARG, "a pointer is not memory of device %d", a.device);

  svx::ResidualParams p = {};
  p.h = a.h;
  p.y = a.y;
  p.gate = a.gate;
  p.norm = a.norm;
  p.post_norm = a.post_norm;
  p.h_out = a.h_out;
  p.x_out = a.x_out;
  p.h_stride = a.h_stride;
  p.y_stride = a.y_stride;
  p.gate_stride = a.gate_kind == SVX_GATE_ELEMENT ? a.gate_stride : 0;
  p.h_out_stride = a.h_out_stride;
  p.x_stride = a.x_stride;
  p.rows = a.rows;
  p.vecs = a.dim / svx::kVec;
  p.gate_kind = a.gate_kind == SVX_GATE_NONE ? svx::kGateNone : a.gate_kind == SVX_GATE_SCALAR ? svx::kGateScalar : svx::kGateRow;
  p.act = a.act;
  p.alpha = a.alpha;
  p.beta = a.beta;
  p.eps = a.eps;
  p.post_eps = a.post_eps;
  p.wide = svx::is_aligned(a.h_out, 32);
  p.inv_dim = 1.f / static_cast<float>(a.dim);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a.dtype == SVX_BF16)
    e = a.stream_dtype == SVX_FP32 ? svx::launch_residual<__nv_bfloat16, float>(p, a.device, s) : svx::launch_residual<__nv_bfloat16, __nv_bfloat16>(p, a.device, s);
  else
    e = a.stream_dtype == SVX_FP32 ? svx::launch_residual<__half, float>(p, a.device, s) : svx::launch_residual<__half, __half>(p, a.device, s);
  if (e != cudaSuccess) return paged_fail(SVX_ERR_CUDA, "residual kernel launch failed: %s", cudaGetErrorString(e));
  return SVX_OK;
}
