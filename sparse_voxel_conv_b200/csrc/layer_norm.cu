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
//
// Both directions are bound by HBM where there is no activation (329,839 x 128 bf16:
// forward 29.3 us, 5.8 TB/s; backward 43.4 us, 5.8 TB/s).  SiLU adds two instructions
// of the special-function pipe an element (19 us of it): 32 us and 48 us in a
// sustained run.  The steps from 568 and 913 us: one read by a block a row -> rows in
// registers of small teams (36 / 90) -> rows ahead by cp.async, pairs (30 / 63) ->
// no recomputed addresses and no branches in the copies (30 / 47) -> one block an SM
// and a wider join of the column sums (30 / 43).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "epilogue.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace subm3d {

constexpr int kMaxRowElements = 8192;  // of a row kernel

// The most blocks that leave partial column sums: four on each of 148 SMs.  Fewer for
// the widest rows, whose sums take the more room the fewer the rows.  Up to
// kOneBlock elements (a round of a block's lanes) one block sums them all: no partial
// sums, no workspace and no second launch, which spares the caller some 4 us.  (4,096
// elements: 3.6 us by one block, 3.8 by many and their join; 16,384: 6.4 and 3.8.)
constexpr int64_t kOneBlock = 8192;
int64_t layer_norm_chunks(int64_t n, int32_t channels) {
  if (channels <= kMaxRowElements / 2 && n * std::max(channels, 64) <= kOneBlock) return 1;
  return std::min<int64_t>(channels <= kMaxRowElements ? n : (n + 63) / 64, 592);
}

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
// at a time, into partial[chunk][2][C] (one chunk: into dweight and dbias).
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
    if (gridDim.y > 1) {
      a.partial[(static_cast<int64_t>(blockIdx.y) * 2 + ty) * a.c + c] = s;
    } else {
      float* out = ty == 0 ? a.dweight : a.dbias;
      if (out) out[c] = s;
    }
  }
}

// dw (blockIdx.y = 0) and db (1): the chunks' partial sums, in a fixed order: 32
// columns a block, its warps take the chunks in turn, eight loads at a time.
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(kJoinWarps * 32) norm_dw_join_kernel(const float* partial,
                                                                      int chunks, int32_t channels,
                                                                      float* dw, float* db) {
  __shared__ float sh[kJoinWarps][33];
  pdl_wait();
  const int lane = threadIdx.x % 32, ty = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  float* out = blockIdx.y == 0 ? dw : db;
  float s = 0.0f;
  if (out && c < channels) {
    const float* p = partial + static_cast<int64_t>(blockIdx.y) * channels + c;
    const int64_t step = 2 * static_cast<int64_t>(channels);
    for (int k = ty; k < chunks; k += 8 * kJoinWarps) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int chunk = k + i * kJoinWarps;
        v[i] = chunk < chunks ? p[chunk * step] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
  }
  sh[ty][lane] = s;
  __syncthreads();
  // lane l of warp w takes warp l's sum of column w
  const float t = warp_sum(sh[lane][ty]);
  const int col = blockIdx.x * 32 + ty;
  if (lane == 0 && out && col < channels) out[col] = t;
}

cudaError_t launch_join(const LayerNormGradArgs& a, int chunks, cudaStream_t stream) {
  return launch_pdl(norm_dw_join_kernel, dim3(static_cast<unsigned>((a.c + 31) / 32), 2),
                    dim3(kJoinWarps * 32), 0, stream, static_cast<const float*>(a.partial), chunks,
                    a.c, a.dweight, a.dbias);
}

// ---------------------------------------------------------------- row kernels ----
//
// A team works on one row: 2^k lanes of a warp, or several whole warps (WIDE;
// LANES = 0).  A lane holds N = V x E elements of the row: V loads of E elements, as
// wide as the rows' alignment allows.  The row is read once; its sums go over the
// team by shuffles, and between warps through one exchange in shared memory.  Teams
// walk over the rows with their columns' weights in registers.  Each lane copies its
// own part of the rows ahead into its own shared-memory slots (cp.async): no
// barrier, and the bytes in flight do not cost registers, which are what limits the
// warps on an SM.  Single-element loads go to registers instead, one row ahead: as
// copies they are twice as many shared-memory operations as the row has elements
// (50,021 x 203 fp32: 18.3 us by copies, 15.9 by loads).

// Rows a lane has under way, its present one included.  More cost shared memory and
// gain nothing (gradient at 329,839 x 128 bf16: 43.3 us with 3, 44.3 with 4); 64-byte
// parts (fp32) have room for 2.
constexpr int kRowStages = 4;
template <typename T, int E, int V>
constexpr int kGradStages = sizeof(T) * E * V >= 64 ? 2 : 3;
constexpr int kMaxRowWarps = 16;  // of a team: 16 * 32 lanes of 16 elements
static_assert(kMaxRowWarps * 32 * 16 == kMaxRowElements, "");
// Rows are counted in 32 bits, some strides of all teams beyond the last one included.
constexpr int64_t kMaxRows = (int64_t(1) << 31) - (1 << 20);
constexpr int kFewestLanes = 4;   // of a team: 16 bytes of 64 channels a lane and load
// Registers of a thread and threads of an SM: forward as many threads as hold their
// elements of a row without spilling (single-element loads hold half as many), the
// gradient 128 registers.  A forward block has up to kRowBlock threads, or one wider
// team; the gradient's blocks fill an SM each, so that few partial sums are left to
// join (16,384 x 1,536 bf16 over three warps a row: 33.4 us; 40.3 with two blocks an SM
// and a slower join).
constexpr int row_registers(int e) { return e > 1 ? 80 : 64; }
constexpr int row_threads(int e) { return e > 1 ? 768 : 1024; }
constexpr int kRowBlock = 256, kGradThreads = 512;

using f2 = unsigned long long;  // two fp32 values
__device__ __forceinline__ f2 f2_set(float v) { return f2_pack(v, v); }
__device__ __forceinline__ float f2_sum(f2 v) {
  float a, b;
  f2_unpack(v, a, b);
  return a + b;
}
__device__ __forceinline__ f2 bf16_pair(uint32_t w) {
  return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t to_bf16_pair(f2 v) {
  float a, b;
  f2_unpack(v, a, b);
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// One instruction each (no handling of subnormal inputs and results, which the
// uses below do not need).
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ f2 exp2_pair(f2 v) {
  float a, b;
  f2_unpack(v, a, b);
  return f2_pack(exp2_fast(a), exp2_fast(b));
}
__device__ __forceinline__ f2 rcp_pair(f2 v) {
  float a, b;
  f2_unpack(v, a, b);
  return f2_pack(rcp_fast(a), rcp_fast(b));
}

// sigmoid(z) of a pair: 1 / (1 + 2^(-z log2 e)).
__device__ __forceinline__ f2 sigmoid_pair(f2 z) {
  return rcp_pair(f2_add(exp2_pair(f2_mul(z, f2_set(-1.4426950408889634f))), f2_set(1.0f)));
}

// Phi(z) and exp(-z^2 / 2) of a pair: the rational-times-Gaussian form that
// gelu_erf uses (epilogue.cuh: Abramowitz & Stegun, eq. 7.1.26, erfc off by at most
// 1.5e-7), with the factor 1/2 of Phi in its coefficients.  With its fp32 roundings Phi
// is off by up to 5 units of 2^-24 (an erf in fp32: 1); the convolution's
// epilogue and this norm give one GELU.
__device__ __forceinline__ f2 phi_pair(f2 z, f2& gauss) {
  const f2 mag = z & 0x7FFFFFFF7FFFFFFFull;
  const f2 t = rcp_pair(f2_fma(mag, f2_set(0.3275911f * 0.70710678118654752f), f2_set(1.0f)));
  f2 q = f2_fma(t, f2_set(0.5f * 1.061405429f), f2_set(0.5f * -1.453152027f));
  q = f2_fma(t, q, f2_set(0.5f * 1.421413741f));
  q = f2_fma(t, q, f2_set(0.5f * -0.284496736f));
  q = f2_fma(t, q, f2_set(0.5f * 0.254829592f));
  gauss = exp2_pair(f2_mul(f2_mul(z, z), f2_set(-0.5f * 1.4426950408889634f)));
  const f2 tail = f2_mul(f2_mul(t, q), gauss);
  float z0, z1, t0, t1, u0, u1;
  f2_unpack(z, z0, z1);
  f2_unpack(tail, t0, t1);
  f2_unpack(f2_fma(tail, f2_set(-1.0f), f2_set(1.0f)), u0, u1);
  return f2_pack(z0 >= 0.0f ? u0 : t0, z1 >= 0.0f ? u1 : t1);
}

template <int ACT>
__device__ __forceinline__ f2 act_pair(f2 z) {
  if (ACT == kActSilu) return f2_mul(z, sigmoid_pair(z));
  if (ACT == kActGelu) {
    f2 gauss;
    return f2_mul(z, phi_pair(z, gauss));
  }
  return z;
}
// act'(z): s (1 + z (1 - s)) = s + (z s) (1 - s); Phi(z) + z phi(z).
template <int ACT>
__device__ __forceinline__ f2 slope_pair(f2 z) {
  if (ACT == kActSilu) {
    const f2 s = sigmoid_pair(z);
    return f2_fma(f2_mul(z, s), f2_fma(s, f2_set(-1.0f), f2_set(1.0f)), s);
  }
  f2 gauss;
  const f2 phi = phi_pair(z, gauss);
  return f2_fma(z, f2_mul(gauss, f2_set(0.39894228040143268f)), phi);
}

// A thread's place.  `lanes` = threads of a team: a power of two up to 32, or whole
// warps.  The loop over rows is a warp's: rows from a.n on (the last round of teams
// inside a warp) are computed on zeros and not stored, so that all lanes take part in
// every shuffle.
struct Team {
  int lanes, warps;      // warps: of a team of whole warps, else 1
  int first, step;       // the lane's vectors: first + k step
  int warp;              // the warp's number in its team
  int id;                // the team's number in the block
  bool leader;           // the team's first lane
  uint32_t row, stride;  // the loop over rows (below 2^31)
  int sub;               // the team's number in the warp
};
template <int V, int LANES>
__device__ __forceinline__ Team team_of(int lanes) {
  constexpr bool WIDE = LANES == 0;
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
  t.row = blockIdx.x * teams + t.id;
  t.stride = gridDim.x * teams;
  return t;
}

// v, in a register: not to be computed again at each use (which costs more
// instructions than the register saves).
__device__ __forceinline__ uint32_t kept(uint32_t v) {
  asm volatile("mov.b32 %0, %0;" : "+r"(v));
  return v;
}

// A lane's parts of the rows ahead.  Parts of several elements are copied into the
// lane's own shared-memory slots (S stages, kStage bytes apart; a warp's slots lie
// together, [S][V][32] parts); single elements are held in registers, one row ahead.
template <typename T, int E, int V, int S>
struct Ahead {
  static constexpr int kBytes = static_cast<int>(sizeof(T)) * E;
  static constexpr bool kAsync = E > 1;
  static constexpr int N = V * E;
  static constexpr int kFront = kAsync ? S - 1 : 1;  // rows on their way
  const char* src;  // the lane's first vector of row 0
  uint32_t mine;
  uint32_t held[kAsync ? 1 : V];
  bool on[V];        // the vector lies in the row

  static constexpr uint32_t kStage = kAsync ? 32 * V * kBytes : 0;
  static constexpr uint32_t kWarp = S * kStage;  // bytes of a warp

  // smem: the warp's slots
  __device__ __forceinline__ void init(uint32_t smem, const void* x, const Team& t, int vecs) {
    mine = kept(smem + threadIdx.x % 32 * kBytes);
    src = static_cast<const char*>(x) + static_cast<int64_t>(t.first) * kBytes;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      on[k] = t.first + k * t.step < vecs;
      if (!on[k]) {  // columns behind the row's end are zeros for good
        held[kAsync ? 0 : k] = 0u;
        if constexpr (kAsync)
          for (int s = 0; s < S; ++s) zero(s * kStage, k);
      }
    }
  }
  __device__ __forceinline__ void zero(uint32_t at, int k) {
    const uint32_t dst = mine + at + k * 32 * kBytes;
#pragma unroll
    for (int i = 0; i < kBytes; i += 4)
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + i), "r"(0) : "memory");
  }
  // Starts on row r, into the stage at byte offset `at`; zeros where there is none.
  // (Predicated copies that fill with zeros: no branch.)
  __device__ __forceinline__ void fetch(uint32_t at, uint32_t r, uint32_t row_bytes, bool live,
                                        const Team& t) {
    const char* row = src + static_cast<uint64_t>(live ? r : 0u) * row_bytes;
    const int bytes = live ? kBytes : 0;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const char* p = row + k * t.step * kBytes;
      if constexpr (!kAsync) {
        held[k] = 0u;
        if (live && on[k]) {
          if constexpr (kBytes == 2) {
            uint16_t h;
            asm volatile("ld.global.b16 %0, [%1];" : "=h"(h) : "l"(p));
            held[k] = h;
          } else {
            asm volatile("ld.global.b32 %0, [%1];" : "=r"(held[k]) : "l"(p));
          }
        }
      } else {
        const uint32_t dst = mine + at + k * 32 * kBytes;
        if constexpr (kBytes == 16)
          asm volatile(
              "{\n .reg .pred q;\n setp.ne.s32 q, %3, 0;\n"
              " @q cp.async.cg.shared.global [%0], [%1], 16, %2;\n}" ::"r"(dst),
              "l"(p), "r"(bytes), "r"(static_cast<int>(on[k]))
              : "memory");
        else
          asm volatile(
              "{\n .reg .pred q;\n setp.ne.s32 q, %4, 0;\n"
              " @q cp.async.ca.shared.global [%0], [%1], %2, %3;\n}" ::"r"(dst),
              "l"(p), "n"(kBytes), "r"(bytes), "r"(static_cast<int>(on[k]))
              : "memory");
      }
    }
  }
  __device__ __forceinline__ void read(uint32_t at, f2 (&v)[N / 2]) const {
    uint32_t w[kAsync ? V * kBytes / 4 : V];
    if constexpr (kAsync) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const uint32_t from = mine + at + k * 32 * kBytes;
        uint32_t* o = w + k * kBytes / 4;
        if constexpr (kBytes == 16)
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
                       : "r"(from)
                       : "memory");
        else
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(o[0]) : "r"(from) : "memory");
      }
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) w[k] = held[k];
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if constexpr (sizeof(T) == 4)
        v[i] = f2_pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
      else if constexpr (kAsync)
        v[i] = bf16_pair(w[i]);
      else
        v[i] = f2_pack(__uint_as_float(w[2 * i] << 16), __uint_as_float(w[2 * i + 1] << 16));
    }
  }
};
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int PENDING>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// The lane's vectors into its row, p = where its first one goes; `live`: there is one.
template <typename T, int E, int V>
__device__ __forceinline__ void store_row(T* p, const f2 (&v)[V * E / 2], const bool (&on)[V],
                                          bool live, const Team& t) {
#pragma unroll
  for (int k = 0; k < V; ++k) {
    T* q = p + k * t.step * E;
    const int go = on[k] && live, j = k * E / 2;
    float lo, hi;
    f2_unpack(v[j], lo, hi);
    if constexpr (sizeof(T) * E == 16) {
      uint32_t w[4];
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = to_bf16_pair(v[j + i]);
      } else {
        float l1, h1;
        f2_unpack(v[j + 1], l1, h1);
        w[0] = __float_as_uint(lo);
        w[1] = __float_as_uint(hi);
        w[2] = __float_as_uint(l1);
        w[3] = __float_as_uint(h1);
      }
      asm volatile(
          "{\n .reg .pred q;\n setp.ne.s32 q, %5, 0;\n"
          " @q st.global.v4.b32 [%0], {%1, %2, %3, %4};\n}" ::"l"(q),
          "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(go)
          : "memory");
    } else if constexpr (E == 2) {
      if (go) *reinterpret_cast<uint32_t*>(q) = to_bf16_pair(v[j]);
    } else {
      if (go) *q = from_f32<T>(k % 2 ? hi : lo);
    }
  }
}

// Sum over the lanes of a team inside a warp (over the warp for wider teams).
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2)
    if (LANES == 0 || LANES > o) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// The barrier of one team of several warps (barrier 0 is __syncthreads').
__device__ __forceinline__ void team_barrier(const Team& t) {
  asm volatile("bar.sync %0, %1;" ::"r"(t.id + 1), "r"(t.lanes) : "memory");
}

// A lane's columns of a weight or bias vector; `none` without one, 0 behind the row.
// Vectors that start on 16 bytes are read in 16-byte loads (they are on the way to a
// block's first row).
template <int E, int V>
__device__ __forceinline__ void load_affine(f2 (&w)[V * E / 2], const void* p, bool bf16,
                                            float none, const Team& t, int vecs) {
  const bool whole = reinterpret_cast<uintptr_t>(p) % 16 == 0;
  float v[V * E];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int64_t c = static_cast<int64_t>(t.first + k * t.step) * E;
    const bool on = t.first + k * t.step < vecs;
#pragma unroll
    for (int i = 0; i < E; ++i) v[k * E + i] = on ? none : 0.0f;
    if (!p || !on) continue;
    if (E % 4 == 0 && whole && !bf16) {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + c);
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const float4 f = q[i];
        v[k * E + 4 * i] = f.x;
        v[k * E + 4 * i + 1] = f.y;
        v[k * E + 4 * i + 2] = f.z;
        v[k * E + 4 * i + 3] = f.w;
      }
    } else if (E == 8 && whole) {
      const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + c);
      const uint32_t words[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const uint32_t word = words[i / 2 % 4];
        v[k * E + i] = __uint_as_float(i % 2 ? word & 0xFFFF0000u : word << 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) v[k * E + i] = affine_at(p, bf16, c + i);
    }
  }
#pragma unroll
  for (int i = 0; i < V * E; i += 2) w[i / 2] = f2_pack(v[i], v[i + 1]);
}

template <typename T, int E, int V, int ACT, int LANES>
__global__ void __maxnreg__(row_registers(E)) norm_row_kernel(LayerNormArgs a, int team_lanes) {
  constexpr bool WIDE = LANES == 0;
  const int lanes = WIDE ? team_lanes : LANES;
  // warps' sums and squares, two buffers in turn: one is written again only behind the
  // other's barrier
  __shared__ float2 slot[2][WIDE ? kMaxRowWarps : 1];
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr int N = V * E;
  constexpr int S = kRowStages;
  pdl_wait();
  const Team t = team_of<V, LANES>(lanes);
  const int vecs = a.c / E;
  const bool full = vecs == V * lanes;
  const float inv_c = 1.0f / static_cast<float>(a.c);
  // elements in each warp of a team: all but the last one are full
  const float last_count = static_cast<float>(a.c - (t.warps - 1) * 32 * N);
  const float my_count = t.warp + 1 < t.warps ? 32.0f * N : last_count;
  const float inv_mine = 1.0f / my_count, inv_last = 1.0f / last_count;
  using A = Ahead<T, E, V, S>;
  A ahead;
  ahead.init(smem_u32(ring) + threadIdx.x / 32 * A::kWarp, a.x, t, vecs);
  const uint32_t n = static_cast<uint32_t>(a.n);
  const auto fetch = [&](uint32_t at, uint32_t r) {
    ahead.fetch(at, r, a.row_bytes, r < n, t);
    if constexpr (A::kAsync) copies_commit();
  };
  constexpr uint32_t stage = A::kStage, last_stage = (S - 1) * stage;
#pragma unroll
  for (int s = 0; s < A::kFront; ++s) fetch(s * stage, t.row + s * t.stride);
  f2 w[N / 2], b[N / 2];
  load_affine<E, V>(w, a.weight, a.affine_bf16, 1.0f, t, vecs);
  load_affine<E, V>(b, a.bias, a.affine_bf16, 0.0f, t, vecs);
  T* y = static_cast<T*>(a.y) + t.first * E;
  int turn = 0;
  uint32_t cur = 0, freed = last_stage;
  for (uint32_t r = t.row; r - t.sub < n; r += t.stride) {
    f2 v[N / 2];
    if constexpr (A::kAsync) copies_wait<A::kFront - 1>();
    ahead.read(cur, v);
    fetch(freed, r + A::kFront * t.stride);
    freed = cur;
    cur = cur == last_stage ? 0 : cur + stage;
    f2 s = v[0];
#pragma unroll
    for (int i = 1; i < N / 2; ++i) s = f2_add(s, v[i]);
    const float sum = lanes_sum<LANES>(f2_sum(s));
    float mean = sum * inv_mine;  // the warp's, and the row's in a team of one warp
    f2 q = f2_set(0.0f);
    const f2 shift = f2_set(-mean);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) v[i] = f2_add(v[i], shift);
    if (!full) {  // columns behind the row's end do not count
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        float lo, hi;
        f2_unpack(v[i], lo, hi);
        v[i] = f2_pack(ahead.on[2 * i / E] ? lo : 0.0f, ahead.on[(2 * i + 1) / E] ? hi : 0.0f);
      }
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) q = f2_fma(v[i], v[i], q);
    float sq = lanes_sum<LANES>(f2_sum(q));
    f2 moved = f2_set(0.0f);
    if (WIDE) {
      // the squares around the row's mean from those around the warps' means
      const int first = t.id * t.warps;
      if (threadIdx.x % 32 == 0) slot[turn][first + t.warp] = make_float2(sum, sq);
      team_barrier(t);
      float whole = 0.0f;
      sq = 0.0f;
      for (int i = 0; i < t.warps; ++i) whole += slot[turn][first + i].x;
      whole *= inv_c;
      for (int i = 0; i < t.warps; ++i) {
        const float2 e = slot[turn][first + i];
        const bool end = i + 1 == t.warps;
        const float d = __fmaf_rn(e.x, end ? inv_last : 1.0f / (32 * N), -whole);
        sq += __fmaf_rn(d * d, end ? last_count : 32.0f * N, e.y);
      }
      turn ^= 1;
      moved = f2_set(mean - whole);
      mean = whole;
    }
    const float rstd = rsqrtf(__fmaf_rn(sq, inv_c, a.eps));
    const f2 rs = f2_set(rstd);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const f2 d = WIDE ? f2_add(v[i], moved) : v[i];
      v[i] = act_pair<ACT>(f2_fma(f2_mul(d, rs), w[i], b[i]));
    }
    store_row<T, E, V>(y + static_cast<uint64_t>(r) * static_cast<uint32_t>(a.c), v, ahead.on,
                       r < n, t);
    if (a.mean && t.leader && r < n) {
      a.mean[r] = mean;
      a.rstd[r] = rstd;
    }
  }
  // the copies behind the last row (zeros) have landed before the block gives up its
  // shared memory
  if constexpr (A::kAsync) copies_wait<0>();
}

// The block's column sums of dw and db into partial[block][2][C] (or straight into dweight
// and dbias, for a grid of one); all threads of the block, done with the rows' slots.
template <typename T, int E, int V, int LANES>
__device__ __forceinline__ void leave_sums(const LayerNormGradArgs& a, const Team& t,
                                           const bool (&on)[V], f2 (&dw)[V * E / 2],
                                           f2 (&db)[V * E / 2], uint8_t* ring) {
  constexpr bool WIDE = LANES == 0;
  constexpr int N = V * E;
  // The lanes with the same columns: first the teams of a warp by shuffles, then the
  // block's warps (or wider teams) through shared memory, where the rows' slots hold
  // their sums now, [groups][2][C].
  if (!WIDE) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2)
      if (o >= LANES) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          dw[i] = f2_add(dw[i], __shfl_xor_sync(0xFFFFFFFFu, dw[i], o));
          db[i] = f2_add(db[i], __shfl_xor_sync(0xFFFFFFFFu, db[i], o));
        }
      }
  }
  __syncthreads();
  float* sums = reinterpret_cast<float*>(ring);
  const int groups = WIDE ? blockDim.x / t.lanes : blockDim.x / 32;
  if (t.sub == 0) {
    float* mine = sums + (WIDE ? t.id : static_cast<int>(threadIdx.x) / 32) * 2 * a.c +
                  t.first * E;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (!on[k]) continue;
      float* at = mine + k * t.step * E;
      if constexpr (E % 4 == 0) {  // 16 bytes: single words would meet in an eighth of the banks
#pragma unroll
        for (int i = 0; i < E; i += 4) {
          const int j = (k * E + i) / 2;
          float4 f;
          f2_unpack(dw[j], f.x, f.y);
          f2_unpack(dw[j + 1], f.z, f.w);
          *reinterpret_cast<float4*>(at + i) = f;
          f2_unpack(db[j], f.x, f.y);
          f2_unpack(db[j + 1], f.z, f.w);
          *reinterpret_cast<float4*>(at + a.c + i) = f;
        }
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const int e = k * E + i;
          float lo, hi;
          f2_unpack(dw[e / 2], lo, hi);
          at[i] = e % 2 ? hi : lo;
          f2_unpack(db[e / 2], lo, hi);
          at[a.c + i] = e % 2 ? hi : lo;
        }
      }
    }
  }
  __syncthreads();
  const int group = 2 * a.c, step = blockDim.x;
  // the groups' sums of `count` columns from `first` on, four columns under way
  const auto add_up = [&](float* out, int first, int count) {
    const float* from = sums + first;
    for (int c = threadIdx.x; c < count; c += 4 * step) {
      float sum[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] = c + j * step < count ? from[c + j * step] : 0.0f;
      for (int k = 1; k < groups; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c + j * step < count) sum[j] += from[k * group + c + j * step];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j * step < count) out[c + j * step] = sum[j];
    }
  };
  if (gridDim.x > 1) {
    add_up(a.partial + static_cast<int64_t>(blockIdx.x) * group, 0, group);
  } else {
    if (a.dweight) add_up(a.dweight, 0, a.c);
    if (a.dbias) add_up(a.dbias, a.c, a.c);
  }
}

// Shared memory of a warp of the gradient kernel.
template <typename T, int E, int V, int ACT>
__host__ __device__ constexpr uint32_t grad_warp_bytes() {
  constexpr int S = kGradStages<T, E, V>;
  return 2 * Ahead<T, E, V, S>::kWarp + S * 256 + (ACT != kActNone ? V * E * 128 : 0);
}

// dx of the team's rows, and the block's column sums of dz xhat and dz.
template <typename T, int E, int V, int ACT, int LANES>
__global__ void __launch_bounds__(kGradThreads, 1)
    norm_grad_row_kernel(LayerNormGradArgs a, int team_lanes) {
  constexpr bool WIDE = LANES == 0;
  const int lanes = WIDE ? team_lanes : LANES;
  __shared__ float2 slot[2][WIDE ? kMaxRowWarps : 1];
  extern __shared__ __align__(16) uint8_t ring[];  // rows ahead; at the end the sums
  constexpr int N = V * E;
  constexpr int S = kGradStages<T, E, V>;
  pdl_wait();
  const Team t = team_of<V, LANES>(lanes);
  const int vecs = a.c / E;
  const float inv_c = 1.0f / static_cast<float>(a.c);
  using A = Ahead<T, E, V, S>;
  A ax, ay;
  // a warp's part: the two rows' slots, a row's mean and rstd [S][2][32], the bias
  constexpr uint32_t kStats = 2 * A::kWarp, kBias = kStats + S * 256;
  const uint32_t warp_part =
      smem_u32(ring) + threadIdx.x / 32 * grad_warp_bytes<T, E, V, ACT>();
  ax.init(warp_part, a.x, t, vecs);
  ay.init(warp_part + A::kWarp, a.dy, t, vecs);
  const uint32_t stats = kept(warp_part + kStats + threadIdx.x % 32 * 4);
  constexpr uint32_t stage = A::kAsync ? A::kStage : 256;
  constexpr uint32_t last_stage = A::kFront * stage;
  const uint32_t n = static_cast<uint32_t>(a.n);
  // stages are told apart by the byte offset of their rows' slots (single elements,
  // which are not copied: by that of their statistics)
  const auto stats_at = [&](uint32_t at) { return stats + at / stage * 256; };
  const auto fetch = [&](uint32_t at, uint32_t r) {
    const bool live = r < n;
    ax.fetch(at, r, a.x_row_bytes, live, t);
    ay.fetch(at, r, a.dy_row_bytes, live, t);
    const uint32_t to = stats_at(at), row = live ? r : 0u;
    const int bytes = live ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(a.mean + row),
                 "r"(bytes)
                 : "memory");
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + 128),
                 "l"(a.rstd + row), "r"(bytes)
                 : "memory");
    copies_commit();
  };
#pragma unroll
  for (int s = 0; s < A::kFront; ++s) fetch(s * stage, t.row + s * t.stride);
  f2 w[N / 2], dw[N / 2], db[N / 2];
  load_affine<E, V>(w, a.weight, a.affine_bf16, 1.0f, t, vecs);
  // the bias waits in the lane's slots, 8 bytes a pair of elements: in registers it
  // would be the sixth array of N
  uint32_t bias = 0;
  if (ACT != kActNone) {
    f2 b[N / 2];
    load_affine<E, V>(b, a.bias, a.affine_bf16, 0.0f, t, vecs);
    bias = kept(warp_part + kBias + threadIdx.x % 32 * 16);
#pragma unroll
    for (int i = 0; i < N / 2; i += 2)
      asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(bias + i / 2 * 512),
                   "l"(b[i]), "l"(b[i + 1])
                   : "memory");
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) dw[i] = db[i] = f2_set(0.0f);
  T* dx = static_cast<T*>(a.dx) + t.first * E;
  int turn = 0;
  uint32_t cur = 0, freed = last_stage;
  for (uint32_t r = t.row; r - t.sub < n; r += t.stride) {
    f2 h[N / 2], g[N / 2];
    copies_wait<A::kFront - 1>();
    ax.read(cur, h);
    ay.read(cur, g);
    float mean, rstd;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(mean) : "r"(stats_at(cur)) : "memory");
    asm volatile("ld.shared.f32 %0, [%1];"
                 : "=f"(rstd)
                 : "r"(stats_at(cur) + 128)
                 : "memory");
    fetch(freed, r + A::kFront * t.stride);
    freed = cur;
    cur = cur == last_stage ? 0 : cur + stage;
    const f2 shift = f2_set(-mean), rs = f2_set(rstd);
    f2 s0 = f2_set(0.0f), s1 = f2_set(0.0f);
    f2 b[2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      h[i] = f2_mul(f2_add(h[i], shift), rs);
      if (ACT != kActNone) {
        if (i % 2 == 0)
          asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];"
                       : "=l"(b[0]), "=l"(b[1])
                       : "r"(bias + i / 2 * 512)
                       : "memory");
        g[i] = f2_mul(g[i], slope_pair<ACT>(f2_fma(h[i], w[i], b[i % 2])));
      }
      db[i] = f2_add(db[i], g[i]);
      dw[i] = f2_fma(g[i], h[i], dw[i]);
      g[i] = f2_mul(g[i], w[i]);
      s0 = f2_add(s0, g[i]);
      s1 = f2_fma(g[i], h[i], s1);
    }
    float m0 = lanes_sum<LANES>(f2_sum(s0)), m1 = lanes_sum<LANES>(f2_sum(s1));
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
    const f2 c0 = f2_set(-m0 * inv_c * rstd), c1 = f2_set(-m1 * inv_c * rstd);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) g[i] = f2_fma(h[i], c1, f2_fma(g[i], rs, c0));
    store_row<T, E, V>(dx + static_cast<uint64_t>(r) * static_cast<uint32_t>(a.c), g, ax.on,
                       r < n && a.dx, t);
  }
  copies_wait<0>();  // also those behind the last row: the slots are free now
  if (!a.sums) return;
  leave_sums<T, E, V, LANES>(a, t, ax.on, dw, db, ring);
}

// The same for bf16 rows of 32 V x 8 elements at most, V > 2, without an activation: a
// warp a row.  Only dw and db stay in registers (16 V of them); xhat and g cost a few
// instructions a pair, so they are formed again from the row's slots for dx, and the
// weights lie in shared memory.  As many instructions a row as over several warps,
// but no exchange: warps wait for nobody and hide one another's latency (46 % of the
// issue slots against 34 %).  A block has more sums to join, so it takes kLongRows rows
// a warp to pay (768 channels: 32,768 rows 32.9 us, 39.2 over several warps; 8,192 rows
// 14.3 and 14.4; 4,096 rows of 1,536 channels 15.2 and 14.2).
constexpr int long_warps(int v) { return v > 4 ? 12 : 16; }  // that the registers allow
constexpr int kLongRows = 4;
template <int V>
__host__ __device__ constexpr uint32_t long_weight_bytes() {
  return V * 32 * 8 * 4;
}
template <int V>
__global__ void __launch_bounds__(long_warps(V) * 32, 1)
    norm_grad_long_kernel(LayerNormGradArgs a) {
  using T = __nv_bfloat16;
  constexpr int E = 8, N = V * E;
  using A = Ahead<T, E, V, 2>;
  static_assert(A::kAsync && A::kFront == 1, "one row ahead, in the other stage");
  extern __shared__ __align__(16) uint8_t ring[];  // weights, rows; at the end the sums
  pdl_wait();
  const Team t = team_of<V, 32>(32);
  const int vecs = a.c / E, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const float inv_c = 1.0f / static_cast<float>(a.c);
  const uint32_t weights = kept(smem_u32(ring) + lane * 16);  // [V][2][32] x 4 floats
  const uint32_t rows = smem_u32(ring) + long_weight_bytes<V>() + warp * 2 * A::kWarp;
  A ax, ay;
  ax.init(rows, a.x, t, vecs);
  ay.init(rows + A::kWarp, a.dy, t, vecs);
  const uint32_t n = static_cast<uint32_t>(a.n);
  float next_mean = 0.0f, next_rstd = 0.0f;
  const auto fetch = [&](uint32_t at, uint32_t r) {
    const bool live = r < n;
    ax.fetch(at, r, a.x_row_bytes, live, t);
    ay.fetch(at, r, a.dy_row_bytes, live, t);
    copies_commit();
    if (live) {
      next_mean = *static_cast<const volatile float*>(a.mean + r);
      next_rstd = *static_cast<const volatile float*>(a.rstd + r);
    }
  };
  fetch(0, t.row);
  for (int i = threadIdx.x; i < V * 256; i += blockDim.x) {
    // float i % 4 of half i / 4 % 2 of the part that lane i / 8 % 32 holds k-th
    const float w = i < a.c ? (a.weight ? affine_at(a.weight, a.affine_bf16, i) : 1.0f) : 0.0f;
    const int k = i / 256, of = i / 8 % 32, half = i / 4 % 2;
    reinterpret_cast<float*>(ring)[((k * 2 + half) * 32 + of) * 4 + i % 4] = w;
  }
  __syncthreads();
  f2 dw[N / 2], db[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) dw[i] = db[i] = f2_set(0.0f);
  T* dx = static_cast<T*>(a.dx) + t.first * E;
  uint32_t cur = 0;
  f2 shift, rs;
  // Zero, by way of the part before: the assembler would load all parts at once, into
  // more registers than there are.  (a.zero is 0, which it does not know.)
  uint32_t chain = 0;
  // xhat, dz and dz w of the k-th part
  const auto part = [&](int k, f2 (&h)[4], f2 (&z)[4], f2 (&g)[4]) {
    uint32_t x[4], y[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(ax.mine + cur + chain + k * 512)
                 : "memory");
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
                 : "r"(ay.mine + cur + chain + k * 512)
                 : "memory");
    f2 w[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2)
      asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];"
                   : "=l"(w[i]), "=l"(w[i + 1])
                   : "r"(weights + chain + (k * 2 + i / 2) * 512)
                   : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = f2_mul(f2_add(bf16_pair(x[i]), shift), rs);
      z[i] = bf16_pair(y[i]);
      g[i] = f2_mul(z[i], w[i]);
    }
    chain = (x[0] ^ static_cast<uint32_t>(g[3])) & a.zero;
  };
  for (uint32_t r = t.row; r < n; r += t.stride) {
    copies_wait<0>();
    shift = f2_set(-next_mean);
    rs = f2_set(next_rstd);
    fetch(cur ^ A::kStage, r + t.stride);
    f2 s0 = f2_set(0.0f), s1 = f2_set(0.0f);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      f2 h[4], z[4], g[4];
      part(k, h, z, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        db[k * 4 + i] = f2_add(db[k * 4 + i], z[i]);
        dw[k * 4 + i] = f2_fma(z[i], h[i], dw[k * 4 + i]);
        s0 = f2_add(s0, g[i]);
        s1 = f2_fma(g[i], h[i], s1);
      }
    }
    const float m0 = lanes_sum<32>(f2_sum(s0)), m1 = lanes_sum<32>(f2_sum(s1));
    if (a.dx) {
      float rstd, unused;
      f2_unpack(rs, rstd, unused);
      const f2 c0 = f2_set(-m0 * inv_c * rstd), c1 = f2_set(-m1 * inv_c * rstd);
      T* to = dx + static_cast<uint64_t>(r) * static_cast<uint32_t>(a.c);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        f2 h[4], z[4], g[4];
        part(k, h, z, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = f2_fma(h[i], c1, f2_fma(g[i], rs, c0));
        if (ax.on[k])
          *reinterpret_cast<uint4*>(to + k * 256) = make_uint4(
              to_bf16_pair(g[0]), to_bf16_pair(g[1]), to_bf16_pair(g[2]), to_bf16_pair(g[3]));
      }
    }
    cur ^= A::kStage;
  }
  copies_wait<0>();
  if (!a.sums) return;
  leave_sums<T, E, V, 32>(a, t, ax.on, dw, db, ring);
}

// How a row kernel lies on the rows.
struct RowPlan {
  int vec = 0;    // elements a load
  int v = 0;      // loads a lane
  int lanes = 0;  // threads of a team; 0: the row is too wide
};

// Loads of 16 bytes where the rows' starts and widths are multiples of that, else of
// 4 where they are (bf16), else of an element.  A lane holds 16 elements (8 single
// ones); teams are as small as that allows.
RowPlan row_plan(int32_t c, bool bf16, int align) {
  RowPlan p;
  p.vec = align == 16 ? (bf16 ? 8 : 4) : (align == 4 && bf16 ? 2 : 1);
  p.v = p.vec > 1 ? 16 / p.vec : 8;
  const int vecs = c / p.vec;
  if (vecs <= 32 * p.v) {
    p.lanes = kFewestLanes;
    while (p.lanes * p.v < vecs) p.lanes *= 2;
  } else {
    const int warps = (vecs + 32 * p.v - 1) / (32 * p.v);
    if (warps <= kMaxRowWarps) p.lanes = warps * 32;
  }
  return p;
}

// Threads of a block: whole teams, up to `most` (or one team); fewer where there would
// be fewer blocks than SMs, down to four warps.
int block_threads(int lanes, int64_t n, int most, int num_sms) {
  const int unit = std::max(lanes, 32);
  int threads = std::max(most / unit, 1) * unit;
  while (threads >= 2 * unit && threads > 128 &&
         threads / lanes * static_cast<int64_t>(num_sms) > n)
    threads = threads / 2 / unit * unit;
  return threads;
}

// Of a gradient's only block: a team a row, up to the most.
int one_block_threads(int lanes, int64_t n) {
  const int unit = std::max(lanes, 32);
  const int64_t wanted = (n * lanes + unit - 1) / unit;
  return static_cast<int>(std::min<int64_t>(wanted, std::max(kGradThreads / unit, 1))) * unit;
}

// Blocks for n rows: as many as there are teams for, up to what fits on the device
// at once (teams walk on from there) and `most`.
int64_t blocks_for(int lanes, int threads, int64_t n, int sm_threads, int num_sms, int64_t most) {
  const int64_t teams = threads / lanes;
  const int64_t resident = static_cast<int64_t>(std::max(1, sm_threads / threads)) * num_sms;
  return std::min({(n + teams - 1) / teams, resident, most});
}

// The largest of 16, 4 and the element's bytes that every row's start is a multiple of.
int rows_align(const void* p, int64_t stride, bool bf16) {
  const uint64_t bytes = static_cast<uint64_t>(stride) * (bf16 ? 2 : 4);
  const uint64_t both = reinterpret_cast<uintptr_t>(p) | bytes;
  return both % 16 == 0 ? 16 : (both % 4 == 0 ? 4 : 2);
}

// More than 48 KB of shared memory, static included, is allowed to a kernel once a device.
template <auto KERNEL>
cudaError_t allow_smem(size_t bytes) {
  if (bytes <= 47 * 1024) return cudaSuccess;
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
  return e;
}

template <typename T, int E, int V, int ACT, int LANES>
cudaError_t launch_norm_rows(const LayerNormArgs& a, const RowPlan& p, int num_sms,
                             cudaStream_t stream) {
  const int threads = block_threads(p.lanes, a.n, kRowBlock, num_sms);
  const size_t smem = threads / 32 * Ahead<T, E, V, kRowStages>::kWarp;
  constexpr auto kernel = norm_row_kernel<T, E, V, ACT, LANES>;
  const cudaError_t e = allow_smem<kernel>(smem);
  if (e != cudaSuccess) return e;
  const int64_t blocks = blocks_for(p.lanes, threads, a.n, row_threads(E), num_sms, 0x7FFFFFFF);
  return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(threads), smem, stream, a,
                    p.lanes);
}

// The gradient's row kernel and the join of its blocks' column sums.
template <typename T, int E, int V, int ACT, int LANES>
cudaError_t launch_grad_rows(const LayerNormGradArgs& a, const RowPlan& p, int num_sms,
                             cudaStream_t stream) {
  const int threads = layer_norm_chunks(a.n, a.c) > 1
                          ? block_threads(p.lanes, a.n, kGradThreads, num_sms)
                          : one_block_threads(p.lanes, a.n);
  const size_t groups = LANES == 0 ? threads / p.lanes : threads / 32;
  const size_t smem =
      std::max<size_t>(threads / 32 * grad_warp_bytes<T, E, V, ACT>(), groups * a.c * 8);
  constexpr auto kernel = norm_grad_row_kernel<T, E, V, ACT, LANES>;
  cudaError_t e = allow_smem<kernel>(smem);
  if (e != cudaSuccess) return e;
  const int64_t blocks =
      blocks_for(p.lanes, threads, a.n, kGradThreads, num_sms, layer_norm_chunks(a.n, a.c));
  e = launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(threads), smem, stream, a,
                 p.lanes);
  if (e != cudaSuccess || !a.sums || blocks == 1) return e;
  return launch_join(a, static_cast<int>(blocks), stream);
}

template <int V>
cudaError_t launch_grad_long(const LayerNormGradArgs& a, int num_sms, cudaStream_t stream) {
  const int threads = block_threads(32, a.n, long_warps(V) * 32, num_sms);
  const size_t rows = 2 * Ahead<__nv_bfloat16, 8, V, 2>::kWarp;
  const size_t warps = threads / 32;
  const size_t smem = std::max(long_weight_bytes<V>() + warps * rows, warps * a.c * 8);
  constexpr auto kernel = norm_grad_long_kernel<V>;
  cudaError_t e = allow_smem<kernel>(smem);
  if (e != cudaSuccess) return e;
  const int64_t blocks =
      blocks_for(32, threads, a.n, long_warps(V) * 32, num_sms, layer_norm_chunks(a.n, a.c));
  e = launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(threads), smem, stream, a);
  if (e != cudaSuccess || !a.sums || blocks == 1) return e;
  return launch_join(a, static_cast<int>(blocks), stream);
}

// f<T, E, V, ACT, LANES> of a plan (LANES 0: teams of several warps).
#define SUBM3D_ROW_LANES(f, T, E, V, ACT, p, ...)                   \
  ((p).lanes > 32    ? f<T, E, V, ACT, 0>(__VA_ARGS__)              \
   : (p).lanes == 32 ? f<T, E, V, ACT, 32>(__VA_ARGS__)             \
   : (p).lanes == 16 ? f<T, E, V, ACT, 16>(__VA_ARGS__)             \
   : (p).lanes == 8  ? f<T, E, V, ACT, 8>(__VA_ARGS__)              \
                     : f<T, E, V, ACT, kFewestLanes>(__VA_ARGS__))
#define SUBM3D_ROW_ACT(f, T, E, V, act, p, ...)                                        \
  ((act) == kActGelu ? SUBM3D_ROW_LANES(f, T, E, V, kActGelu, p, __VA_ARGS__)           \
                     : ((act) == kActSilu ? SUBM3D_ROW_LANES(f, T, E, V, kActSilu, p, __VA_ARGS__) \
                                          : SUBM3D_ROW_LANES(f, T, E, V, kActNone, p, __VA_ARGS__)))
#define SUBM3D_ROW_PLAN(f, a, p, ...)                                                         \
  ((a).bf16 ? ((p).vec == 8 ? SUBM3D_ROW_ACT(f, __nv_bfloat16, 8, 2, (a).act, p, __VA_ARGS__) \
               : (p).vec == 2 ? SUBM3D_ROW_ACT(f, __nv_bfloat16, 2, 8, (a).act, p, __VA_ARGS__) \
                              : SUBM3D_ROW_ACT(f, __nv_bfloat16, 1, 8, (a).act, p, __VA_ARGS__)) \
            : ((p).vec == 4 ? SUBM3D_ROW_ACT(f, float, 4, 4, (a).act, p, __VA_ARGS__)         \
                            : SUBM3D_ROW_ACT(f, float, 1, 8, (a).act, p, __VA_ARGS__)))

}  // namespace

cudaError_t launch_layer_norm(const LayerNormArgs& in, int num_sms, cudaStream_t stream) {
  LayerNormArgs a = in;
  const int align = std::min(rows_align(a.x, a.x_stride, a.bf16), rows_align(a.y, a.c, a.bf16));
  const RowPlan p = row_plan(a.c, a.bf16, align);
  const int64_t row_bytes = a.x_stride * (a.bf16 ? 2 : 4);
  a.row_bytes = static_cast<uint32_t>(row_bytes);
  if (p.lanes > 0 && a.n <= kMaxRows && row_bytes <= 0xFFFFFFFFll)
    return SUBM3D_ROW_PLAN(launch_norm_rows, a, p, a, p, num_sms, stream);
  const dim3 grid(static_cast<unsigned>(std::min(a.n, static_cast<int64_t>(num_sms) * 8)));
  return a.bf16 ? launch_pdl(norm_any_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, stream, a)
                : launch_pdl(norm_any_kernel<float>, grid, dim3(kThreads), 0, stream, a);
}

cudaError_t launch_layer_norm_grad(const LayerNormGradArgs& in, int num_sms, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  LayerNormGradArgs a = in;
  a.sums = a.dweight || a.dbias;
  const int align = std::min({rows_align(a.x, a.x_stride, a.bf16),
                              rows_align(a.dy, a.dy_stride, a.bf16),
                              rows_align(a.dx, a.c, a.bf16)});
  const RowPlan p = row_plan(a.c, a.bf16, align);
  const int64_t x_bytes = a.x_stride * (a.bf16 ? 2 : 4), dy_bytes = a.dy_stride * (a.bf16 ? 2 : 4);
  a.x_row_bytes = static_cast<uint32_t>(x_bytes);
  a.dy_row_bytes = static_cast<uint32_t>(dy_bytes);
  const bool fits = p.lanes > 0 && a.n <= kMaxRows && std::max(x_bytes, dy_bytes) <= 0xFFFFFFFFll;
  if (fits && p.lanes > 32 && a.bf16 && p.vec == 8 && a.act == kActNone) {
    const int v = a.c <= 4 * 256 ? 4 : 6;
    if (a.c <= v * 256 && a.n >= static_cast<int64_t>(kLongRows) * num_sms * long_warps(v))
      return v == 4 ? launch_grad_long<4>(a, num_sms, stream)
                    : launch_grad_long<6>(a, num_sms, stream);
  }
  if (fits)
    return SUBM3D_ROW_PLAN(launch_grad_rows, a, p, a, p, num_sms, stream);
  if (a.dx) {
    const int64_t blocks = std::min(a.n, static_cast<int64_t>(num_sms) * 8);
    const dim3 grid(static_cast<unsigned>(blocks));
    e = a.bf16 ? launch_pdl(norm_dx_any_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, stream, a)
               : launch_pdl(norm_dx_any_kernel<float>, grid, dim3(kThreads), 0, stream, a);
    if (e != cudaSuccess) return e;
  }
  if (!a.sums) return e;
  const int64_t chunks = layer_norm_chunks(a.n, a.c);
  const int64_t rows = (a.n + chunks - 1) / chunks;
  const unsigned cols = static_cast<unsigned>((a.c + 31) / 32);
  const dim3 grid(cols, static_cast<unsigned>(chunks));
  e = a.bf16 ? launch_pdl(norm_dw_any_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, stream, a,
                          rows)
             : launch_pdl(norm_dw_any_kernel<float>, grid, dim3(kThreads), 0, stream, a, rows);
  if (e != cudaSuccess || chunks == 1) return e;
  return launch_join(a, static_cast<int>(chunks), stream);
}

}  // namespace subm3d
