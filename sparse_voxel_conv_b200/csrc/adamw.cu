// One AdamW step over many tensors in one launch.
//
//   m' = b1 m + (1 - b1) g,  v' = b2 v + (1 - b2) g^2,
//   p' = p (1 - lr wd) - lr / (1 - b1^t) * m' / (sqrt(v') / sqrt(1 - b2^t) + eps).
//
// The weight is fp32, or bf16 with or without an fp32 master (with one, the
// step is taken on the master and the bf16 weight is its rounding).
//
// Moments in 8 bits: m and r = sqrt(v) as e4m3, each 32 consecutive elements
// with one power-of-two scale (E8M0): the smallest 2^k, k >= -127, with
// max |value| <= 448 * 2^k.  r instead of v doubles the range of exponents that
// eight bits reach.  With v's 0.1 % steps (b2 = 0.999) against spacings of 6 to
// 12 %, rounding to nearest would leave v where it is for good, so both are
// rounded stochastically, without bias: 20 bits of the fp32 word go, and a
// 16-bit random number (hashed from seed, step, tensor and element, so a step
// is reproducible) is added to them first.  A positive r is never stored as
// zero: the next step divides by it.  A block that holds an infinity or a NaN
// gets the scale 255 (NaN): all its 32 elements are NaN from then on.
//
// The moments' products and sums are rounded one by one (no fma), so that the
// states are the same bits as the formula in elementary fp32 operations gives.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace subm3d {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRowsPerWarp = 8;                             // 32-element blocks a warp takes
constexpr int kChunk = kThreads * kRowsPerWarp;             // elements a block takes

__device__ __forceinline__ uint32_t stir(uint32_t x) {
  x ^= x >> 16;
  x *= 0x9E3779B1u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

struct Hyper {
  float step_size, inv_sqrt_bc2, decay;
  uint32_t key;
};

// The step's factors: from the host, or from the device's step number and rate.
__device__ __forceinline__ Hyper hyper_of(const AdamWStep& a) {
  Hyper h;
  int64_t t = a.step;
  if (a.step_device || a.lr_device) {
    if (a.step_device) t = *static_cast<const volatile int32_t*>(a.step_device);
    const double lr = a.lr_device ? static_cast<double>(*static_cast<const volatile float*>(a.lr_device)) : a.lr;
    const double td = static_cast<double>(t);
    h.step_size = static_cast<float>(lr / -expm1(td * a.log_beta1));
    h.inv_sqrt_bc2 = static_cast<float>(rsqrt(-expm1(td * a.log_beta2)));
    h.decay = static_cast<float>(1.0 - lr * a.weight_decay);
  } else {
    h.step_size = a.step_size;
    h.inv_sqrt_bc2 = a.inv_sqrt_bc2;
    h.decay = a.decay;
  }
  h.key = stir(a.seed + 0x9E3779B9u * static_cast<uint32_t>(t));
  return h;
}

__device__ __forceinline__ uint32_t random_bits(uint32_t k1, uint32_t k2, int64_t i) {
  uint32_t x = static_cast<uint32_t>(i) + static_cast<uint32_t>(i >> 32) * 0x3C6EF373u + k1;
  x ^= x >> 16;
  x = (x * 0x9E3779B1u) ^ k2;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : (byte == 0u ? 0x00400000u : byte << 23));
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3);
  return __half2float(__half(h));
}

// The biased exponent of the block's scale from the largest magnitude's bits.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  if (top >= 0x7F800000u) return 255u;
  const int b = static_cast<int>((top + 0x1FFFFFu) >> 23) - 8;
  return b > 0 ? static_cast<uint32_t>(b) : 0u;
}

// |v| / 2^k as an e4m3 code: the product with 2^-120 puts e4m3's exponents on
// fp32's lowest ones, subnormal numbers included, so the code is the word's top
// bits; `low` is the 16-bit random number.
__device__ __forceinline__ uint32_t e4m3_code(float mag, uint32_t scale, uint32_t low) {
  const float inv = __uint_as_float((254u - scale) << 23);
  const float y = __fmul_rn(__fmul_rn(mag, inv), 0x1p-120f);
  const uint32_t code = (__float_as_uint(y) + (low << 4) + 8u) >> 20;
  return mag > 0.0f ? code : 0u;
}

__device__ __forceinline__ float next_p(const AdamWStep& a, const Hyper& h, float p, float m,
                                        float r) {
  const float denom = __fmaf_rn(r, h.inv_sqrt_bc2, a.eps);
  return __fmaf_rn(-h.step_size, m / denom, p * h.decay);
}

template <bool BITS8, int CAP>
__global__ void __launch_bounds__(kThreads)
    adamw_kernel(const __grid_constant__ AdamWStep a, const __grid_constant__ AdamWList<CAP> l) {
  pdl_wait();
  const Hyper h = hyper_of(a);
  // the tensor this block works on: the last whose first block is not behind it
  int lo = 0, hi = l.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (l.first_block[mid] <= blockIdx.x)
      lo = mid;
    else
      hi = mid - 1;
  }
  const AdamWTensor& t = l.tensors[lo];
  const uint32_t k2 = stir(h.key + 0xBB67AE85u * static_cast<uint32_t>(l.first_tensor + lo + 1));
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t base = static_cast<int64_t>(blockIdx.x - l.first_block[lo]) * kChunk;
  for (int k = 0; k < kRowsPerWarp; ++k) {
    const int64_t b0 = base + (k * kWarps + warp) * 32;  // a 32-element block
    if (b0 >= t.n) break;
    const int64_t i = b0 + lane;
    const bool in = i < t.n;
    float p = 0.0f, g = 0.0f, m = 0.0f, v = 0.0f;
    if (in) {
      p = t.master ? t.master[i]
                   : (a.param_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(t.param)[i])
                                   : static_cast<const float*>(t.param)[i]);
      g = a.grad_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(t.grad)[i])
                      : static_cast<const float*>(t.grad)[i];
      if (BITS8) {
        m = e4m3_value(static_cast<const uint8_t*>(t.exp_avg)[i]) *
            e8m0_value(t.exp_avg_scale[b0 / 32]);
        const float r = e4m3_value(static_cast<const uint8_t*>(t.exp_avg_sq)[i]) *
                        e8m0_value(t.exp_avg_sq_scale[b0 / 32]);
        v = __fmul_rn(r, r);
      } else {
        m = static_cast<const float*>(t.exp_avg)[i];
        v = static_cast<const float*>(t.exp_avg_sq)[i];
      }
    }
    m = __fadd_rn(__fmul_rn(m, a.beta1), __fmul_rn(g, a.one_beta1));
    v = __fadd_rn(__fmul_rn(v, a.beta2), __fmul_rn(__fmul_rn(g, g), a.one_beta2));
    const float r = __fsqrt_rn(v);
    p = next_p(a, h, p, m, r);
    if (in) {
      if (t.master) t.master[i] = p;
      if (a.param_bf16)
        static_cast<__nv_bfloat16*>(t.param)[i] = __float2bfloat16_rn(p);
      else
        static_cast<float*>(t.param)[i] = p;
    }
    if (BITS8) {
      uint32_t tm = __float_as_uint(m) & 0x7FFFFFFFu, tr = __float_as_uint(r) & 0x7FFFFFFFu;
#pragma unroll
      for (int o = 16; o > 0; o /= 2) {
        tm = max(tm, __shfl_xor_sync(0xFFFFFFFFu, tm, o));
        tr = max(tr, __shfl_xor_sync(0xFFFFFFFFu, tr, o));
      }
      const uint32_t sm = scale_byte(tm), sr = scale_byte(tr);
      if (in) {
        const uint32_t rnd = random_bits(h.key, k2, i);
        uint32_t cm = sm == 255u ? 0u : e4m3_code(fabsf(m), sm, rnd & 0xFFFFu);
        uint32_t cr = sr == 255u ? 0u : e4m3_code(r, sr, rnd >> 16);
        if (m < 0.0f) cm |= 128u;
        if (r > 0.0f && cr == 0u) cr = 1u;
        static_cast<uint8_t*>(t.exp_avg)[i] = static_cast<uint8_t>(cm);
        static_cast<uint8_t*>(t.exp_avg_sq)[i] = static_cast<uint8_t>(cr);
        if (lane == 0) {
          t.exp_avg_scale[b0 / 32] = static_cast<uint8_t>(sm);
          t.exp_avg_sq_scale[b0 / 32] = static_cast<uint8_t>(sr);
        }
      }
    } else if (in) {
      static_cast<float*>(t.exp_avg)[i] = m;
      static_cast<float*>(t.exp_avg_sq)[i] = v;
    }
  }
}

}  // namespace

int64_t adamw_chunk() { return kChunk; }

template <int CAP>
cudaError_t launch_adamw(const AdamWStep& a, const AdamWList<CAP>& l, uint32_t blocks, bool bits8,
                         cudaStream_t stream) {
  return bits8 ? launch_pdl(adamw_kernel<true, CAP>, dim3(blocks), dim3(kThreads), 0, stream, a, l)
               : launch_pdl(adamw_kernel<false, CAP>, dim3(blocks), dim3(kThreads), 0, stream, a,
                            l);
}
template cudaError_t launch_adamw(const AdamWStep&, const AdamWList<kAdamWFew>&, uint32_t, bool,
                                  cudaStream_t);
template cudaError_t launch_adamw(const AdamWStep&, const AdamWList<kAdamWMany>&, uint32_t, bool,
                                  cudaStream_t);

}  // namespace subm3d
