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
//
// Bound by HBM: x is read and y written once (131,072 x 24 of 36 x 128 bf16: 245 us,
// 6.6 TB/s).  A thread takes the P pairs of one load, as wide as the head vectors'
// alignment allows up to 16 bytes (two loads half a vector apart in the halves
// layout), computes their cos and sin once, while its first loads are on their way,
// and keeps them in registers over a run of the row's heads.  With a head or two a
// row the angles bound it instead (131,072 x 1 x 64 bf16: 22 us, its bytes 5.4).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"

namespace subm3d {
namespace {

constexpr int kThreads = 256;


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

// E elements of T: in one access of 2 to 16 bytes (WHOLE), or element by element.
// Volatile loads: they stay in front of the angles' arithmetic.
template <typename T, int E, bool WHOLE>
struct Part {
  static constexpr int kBytes = static_cast<int>(sizeof(T)) * E;
  alignas(kBytes) T v[E];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (!WHOLE) {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = p[i];
    } else if constexpr (kBytes == 16) {
      uint4 w;
      asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                   : "l"(p)
                   : "memory");
      *reinterpret_cast<uint4*>(v) = w;
    } else if constexpr (kBytes == 8) {
      uint2 w;
      asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "l"(p) : "memory");
      *reinterpret_cast<uint2*>(v) = w;
    } else if constexpr (kBytes == 4) {
      uint32_t w;
      asm volatile("ld.global.b32 %0, [%1];" : "=r"(w) : "l"(p) : "memory");
      *reinterpret_cast<uint32_t*>(v) = w;
    } else {
      uint16_t w;
      asm volatile("ld.global.b16 %0, [%1];" : "=h"(w) : "l"(p) : "memory");
      *reinterpret_cast<uint16_t*>(v) = w;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (!WHOLE) {
#pragma unroll
      for (int i = 0; i < E; ++i) p[i] = v[i];
    } else if constexpr (kBytes == 16) {
      *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(v);
    } else if constexpr (kBytes == 4) {
      *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(v);
    } else {
      *p = v[0];
    }
  }
};

// cos and sin of P pairs from p0 on at row r; 0 and 0 marks a pair that is copied.
template <int P>
__device__ __forceinline__ void cos_sin(const RotaryArgs& a, const double* turns, int64_t r, int p0,
                                        float (&c)[P], float (&s)[P]) {
  double pos[kRotaryMaxAxes];
#pragma unroll
  for (int i = 0; i < kRotaryMaxAxes; ++i) {
    pos[i] = 0.0;
    if (i < a.axes) {
      const int64_t at = r * a.pos_stride + i;
      pos[i] = a.pos_f32 ? static_cast<double>(static_cast<const float*>(a.pos)[at])
                         : static_cast<double>(static_cast<const int32_t*>(a.pos)[at]);
    }
  }
  const int e0 = a.axis_pairs[0], e1 = e0 + a.axis_pairs[1], e2 = e1 + a.axis_pairs[2];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = p0 + i;
    c[i] = s[i] = 0.0f;
    if (p < a.pairs) {
      const double at = p < e0 ? pos[0] : (p < e1 ? pos[1] : (p < e2 ? pos[2] : pos[3]));
      const double t = at * turns[p];
      // the nearest whole number, by the rounding of a sum in [2^52, 2^53) (a
      // conversion instruction runs at a fraction of the adds' rate)
      constexpr double kWhole = 6755399441055744.0;  // 1.5 * 2^52
      const double whole = __dadd_rn(__dadd_rn(t, kWhole), -kWhole);
      sincospif(2.0f * static_cast<float>(t - whole), &s[i], &c[i]);
      if (a.inverse) s[i] = -s[i];
    }
  }
}

// Heads loaded before the first is stored (twice the registers a head for halves).
// 16-byte parts: 33,331 x 5 x 72 fp32 halves 17.2 us with 3, 19.7 with 4; 131,072 x 24 x
// 128 bf16 interleaved 243 with 4, 260 with 2.  Narrower parts take more.
__host__ __device__ constexpr int unroll_of(int bytes, bool halves) {
  if (halves) return bytes == 16 ? 3 : 4;
  return bytes == 16 ? 4 : (bytes == 8 ? 6 : 8);
}

// Items: (row, run of heads, P pairs).  HALVES: the pairs' second elements lie half a
// vector behind the first ones.
template <typename T, int P, bool HALVES, bool WHOLE>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  extern __shared__ double turns[];
  for (int i = threadIdx.x; i < a.pairs; i += kThreads) turns[i] = a.turns[i];
  pdl_wait();
  __syncthreads();
  constexpr int E = HALVES ? P : 2 * P;
  constexpr int kUnroll = unroll_of(static_cast<int>(sizeof(T)) * E, HALVES);
  const uint32_t half = a.head_dim / 2, slots = half / P, runs = a.runs, run = a.run_heads;
  const int64_t total = a.n * runs * slots;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    int64_t r;
    uint32_t h0, slot;
    if (total <= 0xFFFFFFFFll) {
      const uint32_t j = static_cast<uint32_t>(i), q = j / slots;
      slot = j - q * slots;
      const uint32_t row = q / runs;
      h0 = (q - row * runs) * run;
      r = row;
    } else {
      const int64_t q = i / slots;
      slot = static_cast<uint32_t>(i - q * slots);
      r = q / runs;
      h0 = static_cast<uint32_t>(q - r * runs) * run;
    }
    const uint32_t h1 = min(h0 + run, static_cast<uint32_t>(a.heads));
    const T* x = static_cast<const T*>(a.x) + r * a.x_row + slot * E;
    T* y = static_cast<T*>(a.y) + r * a.y_row + slot * E;
    Part<T, E, WHOLE> lo[kUnroll], hi[HALVES ? kUnroll : 1];
    const auto load = [&](uint32_t h) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (h + u < h1) {
          lo[u].load(x + (h + u) * a.x_head);
          if (HALVES) hi[HALVES ? u : 0].load(x + (h + u) * a.x_head + half);
        }
    };
    load(h0);  // on its way while the angles are computed
    float c[P], s[P];
    cos_sin<P>(a, turns, r, slot * P, c, s);
    for (uint32_t h = h0; h < h1; h += kUnroll) {
      if (h > h0) load(h);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (h + u >= h1) continue;
        T* first = lo[u].v;
        T* second = HALVES ? hi[HALVES ? u : 0].v : lo[u].v + 1;
#pragma unroll
        for (int k = 0; k < P; ++k) {
          T& e0 = first[HALVES ? k : 2 * k];
          T& e1 = second[HALVES ? k : 2 * k];
          const float f0 = to_f32(e0), f1 = to_f32(e1);
          const bool turned = slot * P + k < static_cast<uint32_t>(a.pairs);
          const T g0 = from_f32<T>(f0 * c[k] - f1 * s[k]), g1 = from_f32<T>(f0 * s[k] + f1 * c[k]);
          e0 = turned ? g0 : e0;
          e1 = turned ? g1 : e1;
        }
        lo[u].store(y + (h + u) * a.y_head);
        if (HALVES) hi[HALVES ? u : 0].store(y + (h + u) * a.y_head + half);
      }
    }
  }
}

template <typename T, int P, bool HALVES, bool WHOLE>
cudaError_t launch(RotaryArgs a, int num_sms, cudaStream_t stream) {
  // As many heads in one run as leave every SM its threads (2,048): fewer angles to
  // compute, but a short call is spread over the device.
  const int64_t slots = a.head_dim / 2 / P;
  const int64_t want = static_cast<int64_t>(num_sms) * 2048;
  const int64_t most_runs = (a.heads + 3) / 4;
  int64_t runs = std::min(std::max<int64_t>(want / (a.n * slots), 1), most_runs);
  a.run_heads = static_cast<int32_t>((a.heads + runs - 1) / runs);
  a.runs = (a.heads + a.run_heads - 1) / a.run_heads;
  const int64_t total = a.n * a.runs * slots;
  const int64_t blocks = std::min((total + kThreads - 1) / kThreads,
                                  static_cast<int64_t>(num_sms) * 64);
  return launch_pdl(rotary_kernel<T, P, HALVES, WHOLE>, dim3(static_cast<unsigned>(blocks)),
                    dim3(kThreads), a.pairs * sizeof(double), stream, a);
}

// The widest access that every part of a head vector is a multiple of.
template <typename T>
cudaError_t pick(const RotaryArgs& a, int align, int num_sms, cudaStream_t stream) {
  constexpr int kEsz = static_cast<int>(sizeof(T));
  if (a.halves) {
    if (align == 16) return launch<T, 16 / kEsz, true, true>(a, num_sms, stream);
    if (align == 8) return launch<T, 8 / kEsz, true, true>(a, num_sms, stream);
    if (align == 4) return launch<T, 4 / kEsz, true, true>(a, num_sms, stream);
    return launch<T, 1, true, true>(a, num_sms, stream);
  }
  if (align == 16) return launch<T, 8 / kEsz, false, true>(a, num_sms, stream);
  if (align == 8) return launch<T, 4 / kEsz, false, true>(a, num_sms, stream);
  if (align == 2 * kEsz) return launch<T, 1, false, true>(a, num_sms, stream);
  return launch<T, 1, false, false>(a, num_sms, stream);  // pairs across a border
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int num_sms, cudaStream_t stream) {
  const int64_t esz = a.bf16 ? 2 : 4;
  uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y);
  bits |= static_cast<uintptr_t>(a.head_dim / (a.halves ? 2 : 1) * esz);
  if (a.n > 1) bits |= static_cast<uintptr_t>((a.x_row | a.y_row) * esz);
  if (a.heads > 1) bits |= static_cast<uintptr_t>((a.x_head | a.y_head) * esz);
  const int align = static_cast<int>(std::min<uintptr_t>(bits & (~bits + 1), 16));
  return a.bf16 ? pick<__nv_bfloat16>(a, align, num_sms, stream)
                : pick<float>(a, align, num_sms, stream);
}

}  // namespace subm3d
