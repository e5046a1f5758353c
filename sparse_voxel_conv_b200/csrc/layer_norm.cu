// Layer norm over the channels of each row, with an optional affine map and
// activation, and its backward pass.
//
// Per row x[0 .. C): mean = sum x / C, var = sum (x - mean)^2 / C (two passes:
// no cancellation), rstd = 1 / sqrt(var + eps), xhat = (x - mean) rstd,
// z = xhat w + b, y = act(z).  Everything is fp32 until the one rounding of y.
//
// Backward, with dz = dy act'(z) and g = dz w:
//   db = sum over rows dz, dw = sum over rows dz xhat,
//   dx = rstd (g - mean(g) - xhat mean(g xhat)).
//
// These are the kernels for any width and alignment: a block a row, scalar
// loads, the row read again from the caches for every pass.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "epilogue.cuh"
#include "internal.h"

namespace subm3d {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Element i of a weight or bias vector of either type.
__device__ __forceinline__ float affine_at(const void* p, bool bf16, int64_t i) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
              : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ float activate_rt(int act, float z) {
  return act == kActGelu ? activate<kActGelu>(z)
                         : (act == kActSilu ? activate<kActSilu>(z) : z);
}

// act'(z).  GELU: Phi(z) + z phi(z); SiLU: s (1 + z (1 - s)), s = sigmoid(z).
// Phi as in gelu_erf (epilogue.cuh): its Gaussian factor exp(-z^2 / 2) is also
// phi's.
__device__ __forceinline__ float act_slope_rt(int act, float z) {
  if (act == kActGelu) {
    const float u = fabsf(z) * 0.70710678118654752f;
    const float t = __fdividef(1.0f, __fmaf_rn(0.3275911f, u, 1.0f));
    float poly = __fmaf_rn(t, 1.061405429f, -1.453152027f);
    poly = __fmaf_rn(t, poly, 1.421413741f);
    poly = __fmaf_rn(t, poly, -0.284496736f);
    poly = t * __fmaf_rn(t, poly, 0.254829592f);
    const float e = __expf(-u * u);
    const float half_ec = 0.5f * poly * e;
    return __fmaf_rn(z, 0.39894228040143268f * e, z >= 0.0f ? 1.0f - half_ec : half_ec);
  }
  if (act == kActSilu) {
    const float s = __fdividef(1.0f, 1.0f + __expf(-z));
    return s * __fmaf_rn(z, 1.0f - s, 1.0f);
  }
  return 1.0f;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sums of two values over the block, in every thread.  `sh` holds 2 * kWarps
// floats; the barriers let it be used again right after.
__device__ __forceinline__ float2 block_sum2(float a, float b, float* sh) {
  a = warp_sum(a);
  b = warp_sum(b);
  const int w = threadIdx.x / 32;
  __syncthreads();
  if (threadIdx.x % 32 == 0) {
    sh[w] = a;
    sh[kWarps + w] = b;
  }
  __syncthreads();
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    s.x += sh[i];
    s.y += sh[kWarps + i];
  }
  return s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_any_kernel(LayerNormArgs a) {
  __shared__ float sh[2 * kWarps];
  pdl_wait();
  const float inv_c = 1.0f / static_cast<float>(a.c);
  for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
    T* y = static_cast<T*>(a.y) + r * a.c;
    float s = 0.0f;
    for (int c = threadIdx.x; c < a.c; c += kThreads) s += to_f32(x[c]);
    const float mean = block_sum2(s, 0.0f, sh).x * inv_c;
    float q = 0.0f;
    for (int c = threadIdx.x; c < a.c; c += kThreads) {
      const float d = to_f32(x[c]) - mean;
      q = __fmaf_rn(d, d, q);
    }
    const float rstd = 1.0f / sqrtf(block_sum2(q, 0.0f, sh).x * inv_c + a.eps);
    for (int c = threadIdx.x; c < a.c; c += kThreads) {
      float z = (to_f32(x[c]) - mean) * rstd;
      if (a.weight) z *= affine_at(a.weight, a.affine_bf16, c);
      if (a.bias) z += affine_at(a.bias, a.affine_bf16, c);
      y[c] = from_f32<T>(activate_rt(a.act, z));
    }
    if (a.mean && threadIdx.x == 0) {
      a.mean[r] = mean;
      a.rstd[r] = rstd;
    }
  }
}

// dz and xhat of one element.
template <typename T>
__device__ __forceinline__ float2 slope_at(const LayerNormGradArgs& a, const T* x, const T* dy,
                                           int c, float mean, float rstd, float w) {
  const float xhat = (to_f32(x[c]) - mean) * rstd;
  float dz = to_f32(dy[c]);
  if (a.act != kActNone) {
    const float b = a.bias ? affine_at(a.bias, a.affine_bf16, c) : 0.0f;
    dz *= act_slope_rt(a.act, __fmaf_rn(xhat, w, b));
  }
  return make_float2(dz, xhat);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_dx_any_kernel(LayerNormGradArgs a) {
  __shared__ float sh[2 * kWarps];
  pdl_wait();
  const float inv_c = 1.0f / static_cast<float>(a.c);
  for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
    const T* dy = static_cast<const T*>(a.dy) + r * a.dy_stride;
    T* dx = static_cast<T*>(a.dx) + r * a.c;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float s0 = 0.0f, s1 = 0.0f;
    for (int c = threadIdx.x; c < a.c; c += kThreads) {
      const float w = a.weight ? affine_at(a.weight, a.affine_bf16, c) : 1.0f;
      const float2 v = slope_at(a, x, dy, c, mean, rstd, w);
      s0 += v.x * w;
      s1 = __fmaf_rn(v.x * w, v.y, s1);
    }
    const float2 s = block_sum2(s0, s1, sh);
    for (int c = threadIdx.x; c < a.c; c += kThreads) {
      const float w = a.weight ? affine_at(a.weight, a.affine_bf16, c) : 1.0f;
      const float2 v = slope_at(a, x, dy, c, mean, rstd, w);
      dx[c] = from_f32<T>(rstd * (v.x * w - s.x * inv_c - v.y * (s.y * inv_c)));
    }
  }
}

// Column sums of dz xhat and dz over a chunk of rows: 32 columns a block, 8 rows
// at a time, into partial[chunk][2][C].
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_dw_any_kernel(LayerNormGradArgs a,
                                                               int64_t rows_per_chunk) {
  __shared__ float sh[2][kWarps][33];
  pdl_wait();
  const int lane = threadIdx.x % 32, ty = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  const int64_t r0 = blockIdx.y * rows_per_chunk;
  const int64_t r1 = min(r0 + rows_per_chunk, a.n);
  float dw = 0.0f, db = 0.0f;
  if (c < a.c) {
    const float w = a.weight ? affine_at(a.weight, a.affine_bf16, c) : 1.0f;
    for (int64_t r = r0 + ty; r < r1; r += kWarps) {
      const float2 v = slope_at(a, static_cast<const T*>(a.x) + r * a.x_stride,
                                static_cast<const T*>(a.dy) + r * a.dy_stride, c, a.mean[r],
                                a.rstd[r], w);
      dw = __fmaf_rn(v.x, v.y, dw);
      db += v.x;
    }
  }
  sh[0][ty][lane] = dw;
  sh[1][ty][lane] = db;
  __syncthreads();
  if (ty < 2 && c < a.c) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) s += sh[ty][i][lane];
    a.partial[(static_cast<int64_t>(blockIdx.y) * 2 + ty) * a.c + c] = s;
  }
}

// dw (blockIdx.y = 0) and db (1): the chunks' partial sums, in a fixed order.
__global__ void __launch_bounds__(kThreads) norm_dw_join_kernel(const float* partial, int chunks,
                                                                int32_t channels, float* dw,
                                                                float* db) {
  __shared__ float sh[kWarps][33];
  pdl_wait();
  const int lane = threadIdx.x % 32, ty = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  float* out = blockIdx.y == 0 ? dw : db;
  float s = 0.0f;
  if (out && c < channels)
    for (int k = ty; k < chunks; k += kWarps)
      s += partial[(static_cast<int64_t>(k) * 2 + blockIdx.y) * channels + c];
  sh[ty][lane] = s;
  __syncthreads();
  if (ty == 0 && out && c < channels) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) t += sh[i][lane];
    out[c] = t;
  }
}

constexpr int64_t kMaxChunks = 592;  // four blocks on each of 148 SMs

}  // namespace

int64_t layer_norm_chunks(int64_t n) {
  const int64_t c = (n + 63) / 64;
  return c < kMaxChunks ? c : kMaxChunks;
}

cudaError_t launch_layer_norm(const LayerNormArgs& a, int num_sms, cudaStream_t stream) {
  const int64_t most = static_cast<int64_t>(num_sms) * 8;
  const dim3 grid(static_cast<unsigned>(a.n < most ? a.n : most));
  return a.bf16 ? launch_pdl(norm_any_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, stream, a)
                : launch_pdl(norm_any_kernel<float>, grid, dim3(kThreads), 0, stream, a);
}

cudaError_t launch_layer_norm_grad(const LayerNormGradArgs& a, int num_sms, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (a.dx) {
    const int64_t most = static_cast<int64_t>(num_sms) * 8;
    const dim3 grid(static_cast<unsigned>(a.n < most ? a.n : most));
    e = a.bf16 ? launch_pdl(norm_dx_any_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, stream, a)
               : launch_pdl(norm_dx_any_kernel<float>, grid, dim3(kThreads), 0, stream, a);
    if (e != cudaSuccess) return e;
  }
  if (!a.dweight && !a.dbias) return e;
  const int64_t chunks = layer_norm_chunks(a.n);
  const int64_t rows = (a.n + chunks - 1) / chunks;
  const unsigned cols = static_cast<unsigned>((a.c + 31) / 32);
  const dim3 grid(cols, static_cast<unsigned>(chunks));
  e = a.bf16 ? launch_pdl(norm_dw_any_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, stream, a,
                          rows)
             : launch_pdl(norm_dw_any_kernel<float>, grid, dim3(kThreads), 0, stream, a, rows);
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_dw_join_kernel, dim3(cols, 2), dim3(kThreads), 0, stream,
                    static_cast<const float*>(a.partial), static_cast<int>(chunks), a.c,
                    a.dweight, a.dbias);
}

}  // namespace subm3d
