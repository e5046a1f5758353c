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
// Bound by HBM.  A thread takes 8 consecutive elements: 16-byte accesses, and a block
// of 32 elements is four lanes', whose largest magnitude two shuffles find.
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
constexpr int kEach = 8;                           // consecutive elements of a thread
constexpr int kRounds = 2;                         // groups of them it takes in turn
constexpr int kChunk = kThreads * kEach * kRounds;  // elements of a block

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

// The biased exponent of the block's scale from the largest magnitude's bits.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  if (top >= 0x7F800000u) return 255u;
  const int b = static_cast<int>((top + 0x1FFFFFu) >> 23) - 8;
  return b > 0 ? static_cast<uint32_t>(b) : 0u;
}

// |v| / 2^k as an e4m3 code, inv = 2^-k: the product with 2^-120 puts e4m3's
// exponents on fp32's lowest ones, subnormal numbers included, so the code is the
// word's top bits; `low` is the 16-bit random number times 16.
__device__ __forceinline__ uint32_t e4m3_code(float mag, float inv, uint32_t low) {
  return (__float_as_uint(__fmul_rn(__fmul_rn(mag, inv), 0x1p-120f)) + low + 8u) >> 20;
}

// kEach elements from i on, `count` of them in the tensor (zeros behind it): in
// 16-byte accesses (8 for codes) where WHOLE, else one by one.
template <bool WHOLE>
__device__ __forceinline__ void load(float (&v)[kEach], const float* p, int count) {
  if constexpr (WHOLE) {
    const float4 lo = reinterpret_cast<const float4*>(p)[0], hi = reinterpret_cast<const float4*>(p)[1];
    v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w;
    v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
  } else {
#pragma unroll
    for (int j = 0; j < kEach; ++j) v[j] = j < count ? p[j] : 0.0f;
  }
}
template <bool WHOLE>
__device__ __forceinline__ void load(float (&v)[kEach], const __nv_bfloat16* p, int count) {
  if constexpr (WHOLE) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kEach; ++j) v[j] = j < count ? __bfloat162float(p[j]) : 0.0f;
  }
}
template <bool WHOLE>
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int count) {
  if constexpr (WHOLE) return *reinterpret_cast<const uint2*>(p);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < kEach; ++j)
    if (j < count) w[j / 4] |= static_cast<uint32_t>(p[j]) << (j % 4 * 8);
  return make_uint2(w[0], w[1]);
}
template <bool WHOLE>
__device__ __forceinline__ void store(float* p, const float (&v)[kEach], int count) {
  if constexpr (WHOLE) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (j < count) p[j] = v[j];
  }
}
template <bool WHOLE>
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[kEach], int count) {
  if constexpr (WHOLE) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (j < count) p[j] = __float2bfloat16_rn(v[j]);
  }
}
template <bool WHOLE>
__device__ __forceinline__ void store_codes(uint8_t* p, uint2 w, int count) {
  if constexpr (WHOLE) {
    *reinterpret_cast<uint2*>(p) = w;
  } else {
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (j < count) p[j] = static_cast<uint8_t>((j < 4 ? w.x : w.y) >> (j % 4 * 8));
  }
}

// Eight e4m3 codes times their scale.
__device__ __forceinline__ void decode(float (&v)[kEach], uint2 codes, float scale) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t two = (j < 2 ? codes.x : codes.y) >> (j % 2 * 16) & 0xFFFFu;
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * j] = f.x * scale;
    v[2 * j + 1] = f.y * scale;
  }
}

// The root for the division alone (32-bit moments): one instruction, off by an ulp.
__device__ __forceinline__ float root_fast(float v) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// One thread's elements i .. i + kEach - 1 of tensor t; all threads of a warp are here
// (a block of 32 elements is four lanes').
template <bool BITS8, bool WHOLE>
__device__ __forceinline__ void step_elements(const AdamWStep& a, const Hyper& h,
                                              const AdamWTensor& t, uint32_t k2, int64_t i,
                                              int count) {
  float p[kEach], g[kEach], m[kEach], v[kEach];
  uint2 cm = make_uint2(0u, 0u), cr = cm;
  uint32_t sm = 0u, sr = 0u;
  if (t.master)
    load<WHOLE>(p, t.master + i, count);
  else if (a.param_bf16)
    load<WHOLE>(p, static_cast<const __nv_bfloat16*>(t.param) + i, count);
  else
    load<WHOLE>(p, static_cast<const float*>(t.param) + i, count);
  if (a.grad_bf16)
    load<WHOLE>(g, static_cast<const __nv_bfloat16*>(t.grad) + i, count);
  else
    load<WHOLE>(g, static_cast<const float*>(t.grad) + i, count);
  if constexpr (BITS8) {
    cm = load_codes<WHOLE>(static_cast<const uint8_t*>(t.exp_avg) + i, count);
    cr = load_codes<WHOLE>(static_cast<const uint8_t*>(t.exp_avg_sq) + i, count);
    if (WHOLE || count > 0) {
      sm = t.exp_avg_scale[i / 32];
      sr = t.exp_avg_sq_scale[i / 32];
    }
    decode(m, cm, e8m0_value(sm));
    decode(v, cr, e8m0_value(sr));
#pragma unroll
    for (int j = 0; j < kEach; ++j) v[j] = __fmul_rn(v[j], v[j]);
  } else {
    load<WHOLE>(m, static_cast<const float*>(t.exp_avg) + i, count);
    load<WHOLE>(v, static_cast<const float*>(t.exp_avg_sq) + i, count);
  }
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    m[j] = __fadd_rn(__fmul_rn(m[j], a.beta1), __fmul_rn(g[j], a.one_beta1));
    v[j] = __fadd_rn(__fmul_rn(v[j], a.beta2), __fmul_rn(__fmul_rn(g[j], g[j]), a.one_beta2));
    const float r = BITS8 ? __fsqrt_rn(v[j]) : root_fast(v[j]);
    const float denom = __fmaf_rn(r, h.inv_sqrt_bc2, a.eps);
    p[j] = __fmaf_rn(-h.step_size, __fdividef(m[j], denom), p[j] * h.decay);
    if (BITS8) v[j] = r;
  }
  if (t.master) store<WHOLE>(t.master + i, p, count);
  if (a.param_bf16)
    store<WHOLE>(static_cast<__nv_bfloat16*>(t.param) + i, p, count);
  else
    store<WHOLE>(static_cast<float*>(t.param) + i, p, count);
  if constexpr (BITS8) {
    uint32_t tm = 0u, tr = 0u;  // the largest magnitudes' bits
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      tm = max(tm, __float_as_uint(m[j]) & 0x7FFFFFFFu);
      tr = max(tr, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    }
#pragma unroll
    for (int o = 1; o < 32 / kEach; o *= 2) {
      tm = max(tm, __shfl_xor_sync(0xFFFFFFFFu, tm, o));
      tr = max(tr, __shfl_xor_sync(0xFFFFFFFFu, tr, o));
    }
    sm = scale_byte(tm);
    sr = scale_byte(tr);
    // a block with a NaN scale keeps any codes: zeros
    const float im = sm == 255u ? 0.0f : __uint_as_float((254u - sm) << 23);
    const float ir = sr == 255u ? 0.0f : __uint_as_float((254u - sr) << 23);
    uint32_t wm[2] = {0u, 0u}, wr[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const uint32_t rnd = random_bits(h.key, k2, i + j);
      const float mag = sm == 255u ? 0.0f : fabsf(m[j]), root = sr == 255u ? 0.0f : v[j];
      const uint32_t sign = __float_as_uint(m[j]) >> 31 << 7;
      const uint32_t code_m = e4m3_code(mag, im, (rnd & 0xFFFFu) << 4) | sign;
      const uint32_t code_r = max(e4m3_code(root, ir, rnd >> 16 << 4), root > 0.0f ? 1u : 0u);
      wm[j / 4] |= code_m << (j % 4 * 8);
      wr[j / 4] |= code_r << (j % 4 * 8);
    }
    store_codes<WHOLE>(static_cast<uint8_t*>(t.exp_avg) + i, make_uint2(wm[0], wm[1]), count);
    store_codes<WHOLE>(static_cast<uint8_t*>(t.exp_avg_sq) + i, make_uint2(wr[0], wr[1]), count);
    if (threadIdx.x % (32 / kEach) == 0 && count > 0) {
      t.exp_avg_scale[i / 32] = static_cast<uint8_t>(sm);
      t.exp_avg_sq_scale[i / 32] = static_cast<uint8_t>(sr);
    }
  } else {
    store<WHOLE>(static_cast<float*>(t.exp_avg) + i, m, count);
    store<WHOLE>(static_cast<float*>(t.exp_avg_sq) + i, v, count);
  }
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
  const AdamWTensor t = l.tensors[lo];
  const uint32_t k2 = stir(h.key + 0xBB67AE85u * static_cast<uint32_t>(l.first_tensor + lo + 1));
  const int64_t base = static_cast<int64_t>(blockIdx.x - l.first_block[lo]) * kChunk;
#pragma unroll 1
  for (int k = 0; k < kRounds; ++k) {
    // the warp's first element: its threads go one way
    const int64_t w = base + (k * kThreads + threadIdx.x / 32 * 32) * kEach;
    if (w >= t.n) break;
    const int64_t i = w + threadIdx.x % 32 * kEach;
    if (t.whole && w + 32 * kEach <= t.n)
      step_elements<BITS8, true>(a, h, t, k2, i, kEach);
    else
      step_elements<BITS8, false>(a, h, t, k2, i,
                                  static_cast<int>(max(int64_t(0), min(t.n - i, int64_t(kEach)))));
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
