// The residual stream between two blocks of a decoder layer, in one pass.
//
//   u  = y, or y rsqrt(mean y^2 + post_eps) post_norm       (the norm after the block)
//   h' = alpha h + beta act(gate) u                          (the gate, and the scaled residual sum)
//   x  = h' rsqrt(mean h'^2 + eps) norm                      (the norm before the next block)
//
// A row is held in registers from its loads to its stores (kVec elements, 16 bytes of a 16-bit type, at a time), so that h, y and a
// gate per element are read once and h', x written once: those bytes are the floor.  Two sums over the row, each a
// shuffle within the warps and one exchange through shared memory between them.  Everything is fp32, rounded once on the way out; x is
// the norm of the unrounded h'.
#include "svx_paged.h"

#include <cfloat>
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
  float alpha, beta, eps, post_eps;  // eps < 0: no such norm
  float inv_dim;
};

template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[kVec]);
template <>
__device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4& v, float (&f)[kVec]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void unpack<__half>(const uint4& v, float (&f)[kVec]) {
  const __half2* p = reinterpret_cast<const __half2*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = __half22float2(p[i]);
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}
__device__ __forceinline__ uint32_t pack2(__nv_bfloat16, float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint32_t pack2(__half, float a, float b) {
  const __half2 p = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// kVec elements as they lie in memory.
template <typename T>
struct Raw {
  uint4 v;
  __device__ __forceinline__ void load(const T* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&f)[kVec]) const { unpack<T>(v, f); }
  static __device__ __forceinline__ void store(T* p, const float (&f)[kVec]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack2(T(), f[0], f[1]), pack2(T(), f[2], f[3]), pack2(T(), f[4], f[5]), pack2(T(), f[6], f[7]));
  }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&f)[kVec]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&f)[kVec]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

__device__ __forceinline__ float activate(float g, int act) {
  return act == SVX_ACT_TANH ? tanhf(g) : act == SVX_ACT_SIGMOID ? 1.f / (1.f + expf(-g)) : g;
}

// The sum over the threads of a row: a warp, or the block (every thread gets it; `s` is used once a call).
template <bool WARP_ROW>
__device__ __forceinline__ float row_sum(float v, float* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (!WARP_ROW) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) s[warp] = v;
    __syncthreads();
    v = lane < (blockDim.x >> 5) ? s[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}

// T: block outputs and weights; H: the residual stream.  WARP_ROW: a row to each warp, else to each block.  N: the most
// kVec-element pieces of a row that a thread holds.
template <typename T, typename H, bool WARP_ROW, int N>
__global__ void __launch_bounds__(WARP_ROW ? 128 : kMaxThreads) residual_kernel(const __grid_constant__ ResidualParams P) {
  __shared__ float s_post[32], s_pre[32];
  const int64_t row = WARP_ROW ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5) : blockIdx.x;
  const int t = WARP_ROW ? threadIdx.x & 31 : threadIdx.x, step = WARP_ROW ? 32 : blockDim.x;
  grid_dependency_wait();
  allow_dependents();
  if (row >= P.rows) return;  // (whole warps, and no barrier follows for them)
  Raw<H> h[N];
  Raw<T> y[N], g[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int v = t + i * step;
    if (v >= P.vecs) continue;
    if (P.y) y[i].load(static_cast<const T*>(P.y) + row * P.y_stride + v * kVec);
    h[i].load(static_cast<const H*>(P.h) + row * P.h_stride + v * kVec);
    if (P.gate_kind == kGateRow) g[i].load(static_cast<const T*>(P.gate) + row * P.gate_stride + v * kVec);
  }
  float factor = P.beta;
  if (P.y && P.post_eps >= 0.f) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (t + i * step >= P.vecs) continue;
      float f[kVec];
      y[i].get(f);
#pragma unroll
      for (int e = 0; e < kVec; ++e) sum = fmaf(f[e], f[e], sum);
    }
    factor *= rsqrtf(fmaf(row_sum<WARP_ROW>(sum, s_post), P.inv_dim, P.post_eps));
  }
  if (P.gate_kind == kGateScalar) factor *= activate(static_cast<float>(*static_cast<const T*>(P.gate)), P.act);
  float z[N][kVec];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int v = t + i * step;
    if (v >= P.vecs) continue;
    h[i].get(z[i]);
#pragma unroll
    for (int e = 0; e < kVec; ++e) z[i][e] *= P.alpha;
    if (P.y) {
      float u[kVec], w[kVec];
      y[i].get(u);
#pragma unroll
      for (int e = 0; e < kVec; ++e) u[e] *= factor;
      if (P.post_norm) {
        Raw<T> r;
        r.load(static_cast<const T*>(P.post_norm) + v * kVec);
        r.get(w);
#pragma unroll
        for (int e = 0; e < kVec; ++e) u[e] *= w[e];
      }
      if (P.gate_kind == kGateRow) {
        g[i].get(w);
#pragma unroll
        for (int e = 0; e < kVec; ++e) u[e] *= activate(w[e], P.act);
      }
#pragma unroll
      for (int e = 0; e < kVec; ++e) z[i][e] += u[e];
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) sum = fmaf(z[i][e], z[i][e], sum);
    if (P.h_out) Raw<H>::store(static_cast<H*>(P.h_out) + row * P.h_out_stride + v * kVec, z[i]);
  }
  if (!P.x_out) return;
  const float r = rsqrtf(fmaf(row_sum<WARP_ROW>(sum, s_pre), P.inv_dim, P.eps));
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int v = t + i * step;
    if (v >= P.vecs) continue;
#pragma unroll
    for (int e = 0; e < kVec; ++e) z[i][e] *= r;
    if (P.norm) {
      float w[kVec];
      Raw<T> raw;
      raw.load(static_cast<const T*>(P.norm) + v * kVec);
      raw.get(w);
#pragma unroll
      for (int e = 0; e < kVec; ++e) z[i][e] *= w[e];
    }
    Raw<T>::store(static_cast<T*>(P.x_out) + row * P.x_stride + v * kVec, z[i]);
  }
}

template <typename T, typename H>
cudaError_t launch_residual(const ResidualParams& p, cudaStream_t s) {
  // a warp holds rows of up to 1024 elements; else as few threads as hold the row four pieces each
  if (p.vecs <= 128) {
    const dim3 grid(static_cast<unsigned>((p.rows + 3) / 4));
    return p.vecs <= 32 ? launch_pdl(residual_kernel<T, H, true, 1>, grid, dim3(128), 0, s, p)
                        : launch_pdl(residual_kernel<T, H, true, 4>, grid, dim3(128), 0, s, p);
  }
  const int threads = ((p.vecs + 3) / 4 + 31) / 32 * 32;
  return launch_pdl(residual_kernel<T, H, false, 4>, dim3(static_cast<unsigned>(p.rows)), dim3(threads), 0, s, p);
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
  p.inv_dim = 1.f / static_cast<float>(a.dim);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a.dtype == SVX_BF16)
    e = a.stream_dtype == SVX_FP32 ? svx::launch_residual<__nv_bfloat16, float>(p, s) : svx::launch_residual<__nv_bfloat16, __nv_bfloat16>(p, s);
  else
    e = a.stream_dtype == SVX_FP32 ? svx::launch_residual<__half, float>(p, s) : svx::launch_residual<__half, __half>(p, s);
  if (e != cudaSuccess) return paged_fail(SVX_ERR_CUDA, "residual kernel launch failed: %s", cudaGetErrorString(e));
  return SVX_OK;
}
