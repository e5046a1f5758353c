// Rotary positions with up to four axes.
//
// A head vector of D channels is D / 2 pairs.  The first axis_pairs[0] pairs
// turn with the first axis of the row's position, the next axis_pairs[1] with
// the second, and so on; pairs behind the axes' are copied.  Pair j of an axis
// with n pairs turns by position * theta^(-j / n):
//   (x0, x1) -> (x0 cos - x1 sin, x0 sin + x1 cos),
// the inverse (and the gradient) by the opposite angle.  Pairs are neighbours
// (2p, 2p + 1) or lie half a vector apart (p, p + D / 2).
//
// The angle of a far position has to be known to a small part of one turn, so
// it is formed in fp64 and in turns: position * (theta^(-j/n) / 2 pi), minus
// the nearest whole number (exact); the rest, within [-1/2, 1/2], goes through
// sincospif.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace subm3d {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// cos and sin of pair p < a.pairs at row r.
__device__ __forceinline__ float2 cos_sin(const RotaryArgs& a, int64_t r, int p) {
  int axis = 0, first = a.axis_pairs[0];
  while (p >= first) first += a.axis_pairs[++axis];
  const double pos = a.pos_f32
                         ? static_cast<double>(static_cast<const float*>(a.pos)[r * a.pos_stride + axis])
                         : static_cast<double>(static_cast<const int32_t*>(a.pos)[r * a.pos_stride + axis]);
  const double turns = pos * a.turns[p];
  const float rest = static_cast<float>(turns - rint(turns));
  float s, c;
  sincospif(2.0f * rest, &s, &c);
  return make_float2(c, a.inverse ? -s : s);
}

// A thread a pair of one head.
template <typename T>
__global__ void __launch_bounds__(kThreads) rotary_any_kernel(const __grid_constant__ RotaryArgs a) {
  pdl_wait();
  const int half = a.head_dim / 2;
  const int64_t total = a.n * a.heads * half;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int p = static_cast<int>(i % half);
    const int64_t rh = i / half;
    const int64_t r = rh / a.heads;
    const int64_t h = rh % a.heads;
    const T* x = static_cast<const T*>(a.x) + r * a.x_row + h * a.x_head;
    T* y = static_cast<T*>(a.y) + r * a.y_row + h * a.y_head;
    const int i0 = a.halves ? p : 2 * p, i1 = a.halves ? p + half : 2 * p + 1;
    const T x0 = x[i0], x1 = x[i1];
    if (p >= a.pairs) {
      y[i0] = x0;
      y[i1] = x1;
      continue;
    }
    const float2 cs = cos_sin(a, r, p);
    const float f0 = to_f32(x0), f1 = to_f32(x1);
    store(y + i0, f0 * cs.x - f1 * cs.y);
    store(y + i1, f0 * cs.y + f1 * cs.x);
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int num_sms, cudaStream_t stream) {
  const int64_t total = a.n * a.heads * (a.head_dim / 2);
  const int64_t want = (total + kThreads - 1) / kThreads;
  const int64_t most = static_cast<int64_t>(num_sms) * 16;
  const dim3 grid(static_cast<unsigned>(want < most ? want : most));
  return a.bf16 ? launch_pdl(rotary_any_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, stream, a)
                : launch_pdl(rotary_any_kernel<float>, grid, dim3(kThreads), 0, stream, a);
}

}  // namespace subm3d
