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
// Rows up to some thousands of elements are held in registers and read once (row
// kernels, below); wider ones take the kernels for any width: a block a row, the
// row read again from the caches for every pass.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "epilogue.cuh"
#include "internal.h"

namespace subm3d {

// Blocks that leave partial column sums: four on each of 148 SMs, fewer for few rows.
int64_t layer_norm_chunks(int64_t n) { return std::min<int64_t>((n + 15) / 16, 592); }

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

// ---------------------------------------------------------------- row kernels ----
//
// A team works on one row: 2^k lanes of a warp, or several whole warps.  A lane
// holds kLane = V x E elements of the row in registers: V loads of E elements,
// 16-byte loads where the rows allow it and single elements otherwise.  The row is
// read once; its sums go over the team by shuffles, and between warps through one
// exchange in shared memory.  Teams walk over the rows with their columns' weights
// in registers and load the next row before they work on this one.

constexpr int kMaxRowWarps = 16;  // forward: rows up to 16 * 32 * 16 = 8,192 elements
constexpr int kMaxGradWarps = 8;  // backward: 4,096

using f2 = unsigned long long;  // two fp32 values
__device__ __forceinline__ f2 f2_set(float v) { return f2_pack(v, v); }
__device__ __forceinline__ float f2_sum(f2 v) {
  float a, b;
  f2_unpack(v, a, b);
  return a + b;
}

// E elements as they lie in memory.  (Coherent loads in volatile asm: they stay
// behind pdl_wait() and in front of the work on the row before.)
template <typename T, int E>
struct Raw;
template <>
struct Raw<__nv_bfloat16, 8> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(p));
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      o[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
  }
};
template <>
struct Raw<float, 4> {
  float w[4];
  __device__ __forceinline__ void load(const float* p) {
    asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(w[0]), "=f"(w[1]), "=f"(w[2]), "=f"(w[3])
                 : "l"(p));
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0.0f; }
  __device__ __forceinline__ float at(int i) const { return w[i]; }
  static __device__ __forceinline__ void store(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct Raw<__nv_bfloat16, 1> {
  uint16_t w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    asm volatile("ld.global.b16 %0, [%1];" : "=h"(w) : "l"(p));
  }
  __device__ __forceinline__ void zero() { w = 0; }
  __device__ __forceinline__ float at(int) const {
    return __uint_as_float(static_cast<uint32_t>(w) << 16);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) {
    *p = __float2bfloat16_rn(v[0]);
  }
};
template <>
struct Raw<float, 1> {
  float w;
  __device__ __forceinline__ void load(const float* p) {
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(w) : "l"(p));
  }
  __device__ __forceinline__ void zero() { w = 0.0f; }
  __device__ __forceinline__ float at(int) const { return w; }
  static __device__ __forceinline__ void store(float* p, const float* v) { *p = v[0]; }
};

// A thread's place.  `lanes` = threads of a team: a power of two up to 32, or whole
// warps.  The loop over rows is a warp's: `base` is its first team's row, and rows
// from a.n on (the last round of teams inside a warp) are computed on zeros and not
// stored, so that all lanes take part in every shuffle.
struct Team {
  int lanes, warps;     // warps: of a team of whole warps, else 1
  int first, step;      // the lane's vectors: first + k step
  int warp;             // the warp's number in its team
  int id;               // the team's number in the block
  bool leader;          // the team's first lane
  int64_t base, stride;  // the loop over rows
  int sub;              // the team's number in the warp
};
template <int V, bool WIDE>
__device__ __forceinline__ Team team_of(int lanes) {
  Team t;
  const int l = threadIdx.x % lanes;
  t.lanes = lanes;
  t.id = threadIdx.x / lanes;
  t.leader = l == 0;
  const int teams = blockDim.x / lanes;
  t.step = WIDE ? 32 : lanes;
  t.warps = WIDE ? lanes / 32 : 1;
  t.warp = WIDE ? l / 32 : 0;
  t.first = t.warp * 32 * V + l % t.step;
  t.sub = WIDE ? 0 : (threadIdx.x % 32) / lanes;
  t.base = static_cast<int64_t>(blockIdx.x) * teams + (t.id - t.sub);
  t.stride = static_cast<int64_t>(gridDim.x) * teams;
  return t;
}

// Sum over the lanes of a team inside a warp (over the warp for wider teams).
template <bool WIDE>
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2)
    if (WIDE || lanes > o) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// The barrier of one team of several warps (barrier 0 is __syncthreads').
__device__ __forceinline__ void team_barrier(const Team& t) {
  asm volatile("bar.sync %0, %1;" ::"r"(t.id + 1), "r"(t.lanes) : "memory");
}

template <typename T, int E, int V>
__device__ __forceinline__ void load_row(Raw<T, E> (&raw)[V], const T* p, const Team& t, int vecs) {
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int v = t.first + k * t.step;
    if (v < vecs)
      raw[k].load(p + v * E);
    else
      raw[k].zero();
  }
}
template <typename T, int E, int V>
__device__ __forceinline__ void zero_row(Raw<T, E> (&raw)[V]) {
#pragma unroll
  for (int k = 0; k < V; ++k) raw[k].zero();
}

// A lane's columns of a weight or bias vector; `none` without one, 0 behind the row.
template <int E, int V>
__device__ __forceinline__ void load_affine(float (&w)[V * E], const void* p, bool bf16, float none,
                                            const Team& t, int vecs) {
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int v = t.first + k * t.step;
#pragma unroll
    for (int i = 0; i < E; ++i)
      w[k * E + i] = v < vecs ? (p ? affine_at(p, bf16, static_cast<int64_t>(v) * E + i) : none)
                              : 0.0f;
  }
}

template <typename T, int E, int V, int ACT, bool WIDE>
__global__ void __launch_bounds__(WIDE ? kMaxRowWarps * 32 : kThreads, WIDE ? 1 : 3)
    norm_row_kernel(LayerNormArgs a, int lanes) {
  // warps' sums and squares, two buffers in turn: one is written again only behind the
  // other's barrier
  __shared__ float2 slot[2][kMaxRowWarps];
  constexpr int N = V * E;
  pdl_wait();
  const Team t = team_of<V, WIDE>(lanes);
  const int vecs = a.c / E;
  const bool full = vecs == V * lanes;
  const float inv_c = 1.0f / static_cast<float>(a.c);
  // elements in each warp of a team: all but the last one are full
  const float last_count = static_cast<float>(a.c - (t.warps - 1) * 32 * N);
  const float my_count = t.warp + 1 < t.warps ? 32.0f * N : last_count;
  const float inv_mine = 1.0f / my_count, inv_last = 1.0f / last_count;
  float w[N], b[N];
  load_affine<E, V>(w, a.weight, a.affine_bf16, 1.0f, t, vecs);
  load_affine<E, V>(b, a.bias, a.affine_bf16, 0.0f, t, vecs);
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.y);
  Raw<T, E> next[V];
  zero_row(next);
  if (t.base + t.sub < a.n) load_row<T, E, V>(next, x + (t.base + t.sub) * a.x_stride, t, vecs);
  int turn = 0;
  for (int64_t base = t.base; base < a.n; base += t.stride) {
    const int64_t r = base + t.sub;
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = next[i / E].at(i % E);
    if (r + t.stride < a.n) load_row<T, E, V>(next, x + (r + t.stride) * a.x_stride, t, vecs);
    f2 s = f2_set(0.0f);
#pragma unroll
    for (int i = 0; i < N; i += 2) s = f2_add(s, f2_pack(v[i], v[i + 1]));
    const float sum = lanes_sum<WIDE>(f2_sum(s), lanes);
    float mean = sum * inv_mine;  // the warp's, and the row's in a team of one warp
    f2 q = f2_set(0.0f);
    const f2 shift = f2_set(-mean);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      f2 d = f2_add(f2_pack(v[i], v[i + 1]), shift);
      f2_unpack(d, v[i], v[i + 1]);
      if (!full) {  // columns behind the row's end do not count
        if (t.first + i / E * t.step >= vecs) v[i] = 0.0f;
        if (t.first + (i + 1) / E * t.step >= vecs) v[i + 1] = 0.0f;
        d = f2_pack(v[i], v[i + 1]);
      }
      q = f2_fma(d, d, q);
    }
    float sq = lanes_sum<WIDE>(f2_sum(q), lanes);
    if (WIDE) {
      // the squares around the row's mean from those around the warps' means
      const int first = t.id * t.warps;
      if (threadIdx.x % 32 == 0) slot[turn][first + t.warp] = make_float2(sum, sq);
      team_barrier(t);
      float whole = 0.0f;
      for (int i = 0; i < t.warps; ++i) whole += slot[turn][first + i].x;
      whole *= inv_c;
      sq = 0.0f;
      for (int i = 0; i < t.warps; ++i) {
        const float2 e = slot[turn][first + i];
        const bool end = i + 1 == t.warps;
        const float d = __fmaf_rn(e.x, end ? inv_last : 1.0f / (32 * N), -whole);
        sq += __fmaf_rn(d * d, end ? last_count : 32.0f * N, e.y);
      }
      turn ^= 1;
      const f2 moved = f2_set(mean - whole);
#pragma unroll
      for (int i = 0; i < N; i += 2)
        f2_unpack(f2_add(f2_pack(v[i], v[i + 1]), moved), v[i], v[i + 1]);
      mean = whole;
    }
    const float rstd = 1.0f / sqrtf(__fmaf_rn(sq, inv_c, a.eps));
    const f2 rs = f2_set(rstd);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      f2_unpack(f2_fma(f2_mul(f2_pack(v[i], v[i + 1]), rs), f2_pack(w[i], w[i + 1]),
                       f2_pack(b[i], b[i + 1])),
                v[i], v[i + 1]);
      if (ACT == kActGelu) {
        gelu_erf2(v[i], v[i + 1]);
      } else {
        v[i] = activate<ACT>(v[i]);
        v[i + 1] = activate<ACT>(v[i + 1]);
      }
    }
    if (r < a.n) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c = t.first + k * t.step;
        if (c < vecs) Raw<T, E>::store(y + r * a.c + c * E, &v[k * E]);
      }
      if (a.mean && t.leader) {
        a.mean[r] = mean;
        a.rstd[r] = rstd;
      }
    }
  }
}

// dx of the team's rows, and the block's column sums of dz xhat and dz into
// partial[block][2][C] (or straight into dweight and dbias, for a grid of one).
template <typename T, int E, int V, int ACT, bool WIDE>
__global__ void __launch_bounds__(kMaxGradWarps * 32, 2)
    norm_grad_row_kernel(LayerNormGradArgs a, int lanes) {
  __shared__ float2 slot[2][kMaxGradWarps];
  extern __shared__ float sums[];  // [2][C]
  constexpr int N = V * E;
  pdl_wait();
  const Team t = team_of<V, WIDE>(lanes);
  const int vecs = a.c / E;
  const float inv_c = 1.0f / static_cast<float>(a.c);
  float w[N], b[N], dw[N], db[N];
  load_affine<E, V>(w, a.weight, a.affine_bf16, 1.0f, t, vecs);
  if (ACT != kActNone) load_affine<E, V>(b, a.bias, a.affine_bf16, 0.0f, t, vecs);
#pragma unroll
  for (int i = 0; i < N; ++i) dw[i] = db[i] = 0.0f;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  T* dx = static_cast<T*>(a.dx);
  Raw<T, E> nx[V], ny[V];
  zero_row(nx);
  zero_row(ny);
  float next_mean = 0.0f, next_rstd = 0.0f;
  const auto fetch = [&](int64_t r) {
    next_mean = a.mean[r];
    next_rstd = a.rstd[r];
    load_row<T, E, V>(nx, x + r * a.x_stride, t, vecs);
    load_row<T, E, V>(ny, dy + r * a.dy_stride, t, vecs);
  };
  if (t.base + t.sub < a.n) fetch(t.base + t.sub);
  int turn = 0;
  for (int64_t base = t.base; base < a.n; base += t.stride) {
    const int64_t r = base + t.sub;
    const float rstd = next_rstd;
    const f2 shift = f2_set(-next_mean), rs = f2_set(rstd);
    f2 xh[N / 2], g[N / 2];
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      xh[i / 2] = f2_pack(nx[i / E].at(i % E), nx[(i + 1) / E].at((i + 1) % E));
      g[i / 2] = f2_pack(ny[i / E].at(i % E), ny[(i + 1) / E].at((i + 1) % E));
    }
    if (r + t.stride < a.n) {
      fetch(r + t.stride);
    } else {  // a warp's last round may have teams without a row
      zero_row(ny);
    }
    f2 s0 = f2_set(0.0f), s1 = f2_set(0.0f);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const f2 h = f2_mul(f2_add(xh[i / 2], shift), rs);
      const f2 wp = f2_pack(w[i], w[i + 1]);
      f2 dz = g[i / 2];
      if (ACT != kActNone) {
        float z0, z1;
        f2_unpack(f2_fma(h, wp, f2_pack(b[i], b[i + 1])), z0, z1);
        dz = f2_mul(dz, f2_pack(act_slope_rt(ACT, z0), act_slope_rt(ACT, z1)));
      }
      f2_unpack(f2_add(f2_pack(db[i], db[i + 1]), dz), db[i], db[i + 1]);
      f2_unpack(f2_fma(dz, h, f2_pack(dw[i], dw[i + 1])), dw[i], dw[i + 1]);
      xh[i / 2] = h;
      g[i / 2] = f2_mul(dz, wp);
      s0 = f2_add(s0, g[i / 2]);
      s1 = f2_fma(g[i / 2], h, s1);
    }
    float m0 = lanes_sum<WIDE>(f2_sum(s0), lanes), m1 = lanes_sum<WIDE>(f2_sum(s1), lanes);
    if (WIDE) {
      const int first = t.id * t.warps;
      if (threadIdx.x % 32 == 0) slot[turn][first + t.warp] = make_float2(m0, m1);
      team_barrier(t);
      m0 = m1 = 0.0f;
      for (int i = 0; i < t.warps; ++i) {
        m0 += slot[turn][first + i].x;
        m1 += slot[turn][first + i].y;
      }
      turn ^= 1;
    }
    if (r < a.n && dx) {
      const f2 c0 = f2_set(-m0 * inv_c * rstd), c1 = f2_set(-m1 * inv_c * rstd);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        float o[E];
#pragma unroll
        for (int i = 0; i < E; i += 2) {
          if (E > 1) {
            const int j = (k * E + i) / 2;
            f2_unpack(f2_fma(xh[j], c1, f2_fma(g[j], rs, c0)), o[i], o[(i + 1) % E]);
          } else {
            float p0, p1;
            f2_unpack(f2_fma(xh[k / 2], c1, f2_fma(g[k / 2], rs, c0)), p0, p1);
            o[0] = k % 2 ? p1 : p0;
          }
        }
        const int c = t.first + k * t.step;
        if (c < vecs) Raw<T, E>::store(dx + r * a.c + c * E, o);
      }
    }
  }
  if (!a.partial) return;
  // The lanes with the same columns: first the teams of a warp, then, one after
  // another, the block's warps or wider teams.
#pragma unroll
  for (int o = 16; o > 0; o /= 2)
    if (!WIDE && o >= lanes) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        dw[i] += __shfl_xor_sync(0xFFFFFFFFu, dw[i], o);
        db[i] += __shfl_xor_sync(0xFFFFFFFFu, db[i], o);
      }
    }
  const int rounds = WIDE ? blockDim.x / lanes : blockDim.x / 32;
  const int mine = WIDE ? t.id : static_cast<int>(threadIdx.x) / 32;
  for (int round = 0; round < rounds; ++round) {
    if (round == mine && t.sub == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = t.first + i / E * t.step;
        if (v < vecs) {
          float* p = sums + v * E + i % E;
          p[0] = round ? p[0] + dw[i] : dw[i];
          p[a.c] = round ? p[a.c] + db[i] : db[i];
        }
      }
    }
    __syncthreads();
  }
  if (gridDim.x == 1) {
    for (int c = threadIdx.x; c < a.c; c += blockDim.x) {
      if (a.dweight) a.dweight[c] = sums[c];
      if (a.dbias) a.dbias[c] = sums[a.c + c];
    }
  } else {
    float* p = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.c;
    for (int c = threadIdx.x; c < 2 * a.c; c += blockDim.x) p[c] = sums[c];
  }
}

// How a row kernel lies on the rows.
struct RowPlan {
  int vec = 0;    // elements a load: 16 bytes' or 1
  int v = 0;      // loads a lane
  int lanes = 0;  // threads of a team; 0: the row is too wide
  int threads = 0;
  int64_t teams = 0;  // of a block
};

// Rows whose starts and width are multiples of 16 bytes take 16-byte loads.  A lane
// holds 16 elements (8 or 4 single ones: a narrow row still spreads over lanes, and
// a lane's columns cost registers); teams are as small as that allows.
RowPlan row_plan(int32_t c, bool bf16, bool vector, int max_warps) {
  RowPlan p;
  const int wide = bf16 ? 8 : 4;
  p.vec = vector && c % wide == 0 ? wide : 1;
  const int vecs = c / p.vec;
  p.v = p.vec > 1 ? 16 / p.vec : (vecs <= 128 ? 4 : 8);
  if (vecs <= 32 * p.v) {
    p.lanes = 1;
    while (p.lanes * p.v < vecs) p.lanes *= 2;
    p.threads = 256;
  } else {
    const int warps = (vecs + 32 * p.v - 1) / (32 * p.v);
    if (warps > max_warps) return p;
    p.lanes = warps * 32;
    const int teams = warps < 8 ? 8 / warps : 1;
    p.threads = teams * p.lanes;
  }
  p.teams = p.threads / p.lanes;
  return p;
}

// Blocks for n rows: as many as there are teams for, up to what fits on the device
// at once (teams walk on from there) and `most`.
template <typename Kernel>
int64_t resident_blocks(Kernel kernel, const RowPlan& p, int64_t n, size_t smem, int num_sms,
                        int64_t most) {
  int per_sm = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, p.threads, smem) !=
          cudaSuccess ||
      per_sm < 1)
    per_sm = 1;
  return std::min({(n + p.teams - 1) / p.teams, static_cast<int64_t>(per_sm) * num_sms, most});
}

bool rows_of_16_bytes(const void* p, int64_t stride, bool bf16) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % (bf16 ? 8 : 4) == 0;
}

template <typename T, int E, int V>
cudaError_t launch_norm_rows(const LayerNormArgs& a, const RowPlan& p, int num_sms,
                             cudaStream_t stream) {
  const auto go = [&](auto kernel) {
    const int64_t blocks = resident_blocks(kernel, p, a.n, 0, num_sms, 0x7FFFFFFF);
    return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(p.threads), 0, stream, a,
                      p.lanes);
  };
  const auto pick = [&](auto wide) {
    constexpr bool W = decltype(wide)::value;
    if (a.act == kActGelu) return go(norm_row_kernel<T, E, V, kActGelu, W>);
    if (a.act == kActSilu) return go(norm_row_kernel<T, E, V, kActSilu, W>);
    return go(norm_row_kernel<T, E, V, kActNone, W>);
  };
  return p.lanes > 32 ? pick(std::true_type{}) : pick(std::false_type{});
}

// The gradient's row kernel and the join of its blocks' column sums.
template <typename T, int E, int V>
cudaError_t launch_grad_rows(const LayerNormGradArgs& a, const RowPlan& p, int num_sms,
                             cudaStream_t stream) {
  const auto go = [&](auto kernel) {
    const size_t smem = a.partial ? static_cast<size_t>(a.c) * 8 : 0;
    const int64_t blocks = resident_blocks(kernel, p, a.n, smem, num_sms, layer_norm_chunks(a.n));
    const cudaError_t e = launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)),
                                     dim3(p.threads), smem, stream, a, p.lanes);
    if (e != cudaSuccess || !a.partial || blocks == 1) return e;
    return launch_pdl(norm_dw_join_kernel, dim3(static_cast<unsigned>((a.c + 31) / 32), 2),
                      dim3(kThreads), 0, stream, static_cast<const float*>(a.partial),
                      static_cast<int>(blocks), a.c, a.dweight, a.dbias);
  };
  const auto pick = [&](auto wide) {
    constexpr bool W = decltype(wide)::value;
    if (a.act == kActGelu) return go(norm_grad_row_kernel<T, E, V, kActGelu, W>);
    if (a.act == kActSilu) return go(norm_grad_row_kernel<T, E, V, kActSilu, W>);
    return go(norm_grad_row_kernel<T, E, V, kActNone, W>);
  };
  return p.lanes > 32 ? pick(std::true_type{}) : pick(std::false_type{});
}

// f<T, E, V> of a plan.
#define SUBM3D_ROW_PLAN(f, p, bf16, ...)                                        \
  ((bf16) ? ((p).vec > 1 ? f<__nv_bfloat16, 8, 2>(__VA_ARGS__)                  \
                         : ((p).v == 4 ? f<__nv_bfloat16, 1, 4>(__VA_ARGS__)    \
                                       : f<__nv_bfloat16, 1, 8>(__VA_ARGS__))) \
          : ((p).vec > 1 ? f<float, 4, 4>(__VA_ARGS__)                          \
                         : ((p).v == 4 ? f<float, 1, 4>(__VA_ARGS__)            \
                                       : f<float, 1, 8>(__VA_ARGS__))))

}  // namespace

cudaError_t launch_layer_norm(const LayerNormArgs& a, int num_sms, cudaStream_t stream) {
  const bool vector =
      rows_of_16_bytes(a.x, a.x_stride, a.bf16) && rows_of_16_bytes(a.y, a.c, a.bf16);
  const RowPlan p = row_plan(a.c, a.bf16, vector, kMaxRowWarps);
  if (p.lanes > 0) return SUBM3D_ROW_PLAN(launch_norm_rows, p, a.bf16, a, p, num_sms, stream);
  const dim3 grid(static_cast<unsigned>(std::min(a.n, static_cast<int64_t>(num_sms) * 8)));
  return a.bf16 ? launch_pdl(norm_any_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, stream, a)
                : launch_pdl(norm_any_kernel<float>, grid, dim3(kThreads), 0, stream, a);
}

cudaError_t launch_layer_norm_grad(const LayerNormGradArgs& in, int num_sms, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  LayerNormGradArgs a = in;
  if (!a.dweight && !a.dbias) a.partial = nullptr;
  const bool vector = rows_of_16_bytes(a.x, a.x_stride, a.bf16) &&
                      rows_of_16_bytes(a.dy, a.dy_stride, a.bf16) &&
                      rows_of_16_bytes(a.dx, a.c, a.bf16);
  const RowPlan p = row_plan(a.c, a.bf16, vector, kMaxGradWarps);
  if (p.lanes > 0) return SUBM3D_ROW_PLAN(launch_grad_rows, p, a.bf16, a, p, num_sms, stream);
  if (a.dx) {
    const int64_t blocks = std::min(a.n, static_cast<int64_t>(num_sms) * 8);
    const dim3 grid(static_cast<unsigned>(blocks));
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
