// One AdamW step over a list of tensors, up to kAdamWMany of them in a launch.
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
// Bound by HBM: 28 bytes an element with fp32 weights and 32-bit moments (28.3 M
// elements 116 us, 6.8 TB/s, the copy rate), 18.1 with bf16 weights, fp32 gradients
// and masters and 8-bit moments (56.6 M elements 161 us at full clock, 6.4 TB/s; 176
// in a sustained run, whose power lowers the clock: its 67 instructions an element
// count).  A thread takes 8 consecutive elements: 16-byte accesses, and a block of 32
// elements is four lanes', whose largest magnitude two shuffles find.  Arithmetic on
// pairs (f32x2).  Four blocks of 256 threads an SM: with five or six the registers
// spill (178 us), with two groups of elements a thread fewer loads overlap (195).
// These are with the host's step and rate.  With the device's (hyper_of) every thread
// forms the factors in fp64: 119 us for the first case, 219 us for the second, which
// the instructions bound.
//
// The moments' products and sums are rounded one by one (no fma), so that the
// states are the same bits as the formula in elementary fp32 operations gives.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "epilogue.cuh"
#include "internal.h"

namespace subm3d {
namespace {

using f2 = unsigned long long;  // two fp32 values
__device__ __forceinline__ f2 f2_set(float v) { return f2_pack(v, v); }

// A product that keeps its own rounding.  (The assembler joins a mul.f32x2 with the
// add.f32x2 behind it into one fma in spite of their .rn; it cannot join an fma whose
// addend, -0, it does not know: a parameter of the kernel.)
__device__ __forceinline__ f2 product(f2 a, f2 b, f2 minus_zero) {
  return f2_fma(a, b, minus_zero);
}

constexpr int kThreads = 256;
constexpr int kEach = 8;                           // consecutive elements of a thread
constexpr int kPairs = kEach / 2;
constexpr int kChunk = kThreads * kEach;           // elements of a block: one group a thread

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
    double lr = a.lr;
    if (a.lr_device) lr = *static_cast<const volatile float*>(a.lr_device);
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

// The 32 random bits of element i: random_bits(first_word(k1, i), k2), and of the j-th
// after it, with no carry in between (i a multiple of 8, j < 8), + j.
__device__ __forceinline__ uint32_t first_word(uint32_t k1, int64_t i) {
  return static_cast<uint32_t>(i) + static_cast<uint32_t>(i >> 32) * 0x3C6EF373u + k1;
}
__device__ __forceinline__ uint32_t random_bits(uint32_t x, uint32_t k2) {
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

// |v| / 2^k of a pair, inv = 2^-k, times 2^-120: that puts e4m3's exponents on
// fp32's lowest ones, subnormal numbers included, so that an e4m3 code is the bits
// 20 .. 26 of the word.
__device__ __forceinline__ f2 scaled_pair(f2 mag, f2 inv) {
  return f2_mul(f2_mul(mag, inv), f2_set(0x1p-120f));
}
// The stochastically rounded code of such a word in the top byte: the 20 bits below the
// code get the random 16-bit number (half HIGH of rnd) and a half of its last place,
// and the word moves up by 4 bits.
template <bool HIGH>
__device__ __forceinline__ uint32_t code_on_top(float y, uint32_t rnd) {
  const uint32_t add = __byte_perm(rnd, 0x00000080u, HIGH ? 0x5324 : 0x5104);
  return __float_as_uint(y) * 16u + add;
}
// The top bytes of four words.
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// kEach elements from i on, `count` of them in the tensor (zeros behind it): in
// 16-byte accesses (8 for codes) where WHOLE, else one by one.
template <bool WHOLE>
__device__ __forceinline__ void load(f2 (&v)[kPairs], const float* p, int count) {
  if constexpr (WHOLE) {
    const float4 lo = reinterpret_cast<const float4*>(p)[0];
    const float4 hi = reinterpret_cast<const float4*>(p)[1];
    v[0] = f2_pack(lo.x, lo.y), v[1] = f2_pack(lo.z, lo.w);
    v[2] = f2_pack(hi.x, hi.y), v[3] = f2_pack(hi.z, hi.w);
  } else {
#pragma unroll
    for (int j = 0; j < kPairs; ++j)
      v[j] = f2_pack(2 * j < count ? p[2 * j] : 0.0f, 2 * j + 1 < count ? p[2 * j + 1] : 0.0f);
  }
}
template <bool WHOLE>
__device__ __forceinline__ void load(f2 (&v)[kPairs], const __nv_bfloat16* p, int count) {
  if constexpr (WHOLE) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[kPairs] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < kPairs; ++j)
      v[j] = f2_pack(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
  } else {
#pragma unroll
    for (int j = 0; j < kPairs; ++j)
      v[j] = f2_pack(2 * j < count ? __bfloat162float(p[2 * j]) : 0.0f,
                     2 * j + 1 < count ? __bfloat162float(p[2 * j + 1]) : 0.0f);
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
__device__ __forceinline__ void store(float* p, const f2 (&v)[kPairs], int count) {
  float e[kEach];
#pragma unroll
  for (int j = 0; j < kPairs; ++j) f2_unpack(v[j], e[2 * j], e[2 * j + 1]);
  if constexpr (WHOLE) {
    reinterpret_cast<float4*>(p)[0] = make_float4(e[0], e[1], e[2], e[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(e[4], e[5], e[6], e[7]);
  } else {
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (j < count) p[j] = e[j];
  }
}
template <bool WHOLE>
__device__ __forceinline__ void store(__nv_bfloat16* p, const f2 (&v)[kPairs], int count) {
  uint32_t w[kPairs];
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    float lo, hi;
    f2_unpack(v[j], lo, hi);
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  if constexpr (WHOLE) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (j < count) p[j] = __ushort_as_bfloat16(static_cast<uint16_t>(w[j / 2] >> (j % 2 * 16)));
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
__device__ __forceinline__ void decode(f2 (&v)[kPairs], uint2 codes, float scale) {
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    const uint32_t two = (j < 2 ? codes.x : codes.y) >> (j % 2 * 16) & 0xFFFFu;
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[j] = f2_mul(f2_pack(f.x, f.y), f2_set(scale));
  }
}

// For the division alone: one instruction each.  (Denominators lie far from the
// numbers that .ftz drops: a positive root is at least 2^-75, a finite one below 2^65.)
__device__ __forceinline__ float root_fast(float v) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// The correctly rounded roots of a pair of numbers in [2^-100, 2^127): an estimate of
// 1 / sqrt(v), then one step on the root with the remainder v - g^2 formed exactly by an
// fma (Markstein, Computation of elementary functions on the IBM RISC System/6000
// processor, IBM J. Res. Dev. 34, 1990).  All 1,904,214,016
// numbers of that range gave sqrt.rn's bits on a B200.  On pairs it takes half the
// instructions of two sqrt.rn and no branch.
constexpr uint32_t kRootFirst = (127u - 100u) << 23, kRootCount = 227u << 23;
__device__ __forceinline__ f2 root_pair(f2 v) {
  float a, b;
  f2_unpack(v, a, b);
  asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(b));
  const f2 y = f2_pack(a, b), g = f2_mul(v, y);
  return f2_fma(f2_fma(g ^ 0x8000000080000000ull, g, v), f2_mul(y, f2_set(0.5f)), g);
}

// One thread's elements i .. i + kEach - 1 of tensor t; all threads of a warp are here
// (a block of 32 elements is four lanes').
template <bool BITS8, bool PARAM_BF16, bool GRAD_BF16, bool WHOLE>
__device__ __forceinline__ void step_elements(const AdamWStep& a, const Hyper& h,
                                              const AdamWTensor& t, uint32_t k2, int64_t i,
                                              int count) {
  f2 p[kPairs], g[kPairs], m[kPairs], v[kPairs];
  uint2 cm = make_uint2(0u, 0u), cr = cm;
  uint32_t sm = 0u, sr = 0u;
  using Param = std::conditional_t<PARAM_BF16, __nv_bfloat16, float>;
  using Grad = std::conditional_t<GRAD_BF16, __nv_bfloat16, float>;
  if (t.master)
    load<WHOLE>(p, t.master + i, count);
  else
    load<WHOLE>(p, static_cast<const Param*>(t.param) + i, count);
  load<WHOLE>(g, static_cast<const Grad*>(t.grad) + i, count);
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
    for (int j = 0; j < kPairs; ++j) v[j] = f2_mul(v[j], v[j]);
  } else {
    load<WHOLE>(m, static_cast<const float*>(t.exp_avg) + i, count);
    load<WHOLE>(v, static_cast<const float*>(t.exp_avg_sq) + i, count);
  }
  const f2 nz = f2_set(a.minus_zero);
  f2 root[kPairs];
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    m[j] = f2_add(product(m[j], f2_set(a.beta1), nz), product(g[j], f2_set(a.one_beta1), nz));
    v[j] = f2_add(product(v[j], f2_set(a.beta2), nz),
                  product(product(g[j], g[j], nz), f2_set(a.one_beta2), nz));
  }
  bool outside = false;  // roots that root_pair does not take: of zeros, tiny numbers, NaN
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    float lo, hi;
    f2_unpack(v[j], lo, hi);
    if (BITS8) {
      root[j] = root_pair(v[j]);
      const uint32_t from0 = __float_as_uint(lo) - kRootFirst;
      const uint32_t from1 = __float_as_uint(hi) - kRootFirst;
      outside |= max(from0, from1) >= kRootCount;
    } else {
      root[j] = f2_pack(root_fast(lo), root_fast(hi));
    }
  }
  if (BITS8 && outside) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      float lo, hi;
      f2_unpack(v[j], lo, hi);
      root[j] = f2_pack(__fsqrt_rn(lo), __fsqrt_rn(hi));
    }
  }
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    float lo, hi;
    f2_unpack(f2_fma(root[j], f2_set(h.inv_sqrt_bc2), f2_set(a.eps)), lo, hi);
    const f2 step = f2_mul(m[j], f2_pack(rcp_fast(lo), rcp_fast(hi)));
    p[j] = f2_fma(step, f2_set(-h.step_size), f2_mul(p[j], f2_set(h.decay)));
  }
  if (t.master) store<WHOLE>(t.master + i, p, count);
  store<WHOLE>(static_cast<Param*>(t.param) + i, p, count);
  if constexpr (BITS8) {
    uint32_t tm = 0u, tr = 0u;  // the largest magnitudes' bits
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      float lo, hi;
      f2_unpack(m[j], lo, hi);
      tm = max(tm, max(__float_as_uint(lo) & 0x7FFFFFFFu, __float_as_uint(hi) & 0x7FFFFFFFu));
      f2_unpack(root[j], lo, hi);
      tr = max(tr, max(__float_as_uint(lo), __float_as_uint(hi)));
    }
#pragma unroll
    for (int o = 1; o < 32 / kEach; o *= 2) {
      tm = max(tm, __shfl_xor_sync(0xFFFFFFFFu, tm, o));
      tr = max(tr, __shfl_xor_sync(0xFFFFFFFFu, tr, o));
    }
    sm = scale_byte(tm);
    sr = scale_byte(tr);
    // (a block with the scale 255 is NaN whatever its codes are)
    const f2 im = f2_set(__uint_as_float((254u - min(sm, 254u)) << 23));
    const f2 ir = f2_set(__uint_as_float((254u - min(sr, 254u)) << 23));
    const uint32_t word = first_word(h.key, i);
    uint32_t wm[kEach], wr[kEach];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const uint32_t rnd0 = random_bits(word + 2 * j, k2);
      const uint32_t rnd1 = random_bits(word + 2 * j + 1, k2);
      float lo, hi, y0, y1;
      f2_unpack(m[j], lo, hi);
      f2_unpack(scaled_pair(m[j] & 0x7FFFFFFF7FFFFFFFull, im), y0, y1);
      wm[2 * j] = code_on_top<false>(y0, rnd0) | (__float_as_uint(lo) & 0x80000000u);
      wm[2 * j + 1] = code_on_top<false>(y1, rnd1) | (__float_as_uint(hi) & 0x80000000u);
      f2_unpack(root[j], lo, hi);
      f2_unpack(scaled_pair(root[j], ir), y0, y1);
      // at least code 1 for a positive root (whose bits are above 0x01000000)
      wr[2 * j] = max(code_on_top<true>(y0, rnd0), min(__float_as_uint(lo), 0x01000000u));
      wr[2 * j + 1] = max(code_on_top<true>(y1, rnd1), min(__float_as_uint(hi), 0x01000000u));
    }
    cm = make_uint2(top_bytes(wm[0], wm[1], wm[2], wm[3]), top_bytes(wm[4], wm[5], wm[6], wm[7]));
    cr = make_uint2(top_bytes(wr[0], wr[1], wr[2], wr[3]), top_bytes(wr[4], wr[5], wr[6], wr[7]));
    store_codes<WHOLE>(static_cast<uint8_t*>(t.exp_avg) + i, cm, count);
    store_codes<WHOLE>(static_cast<uint8_t*>(t.exp_avg_sq) + i, cr, count);
    if (threadIdx.x % (32 / kEach) == 0 && count > 0) {
      t.exp_avg_scale[i / 32] = static_cast<uint8_t>(sm);
      t.exp_avg_sq_scale[i / 32] = static_cast<uint8_t>(sr);
    }
  } else {
    store<WHOLE>(static_cast<float*>(t.exp_avg) + i, m, count);
    store<WHOLE>(static_cast<float*>(t.exp_avg_sq) + i, v, count);
  }
}

template <bool BITS8, bool PARAM_BF16, bool GRAD_BF16, int CAP>
__global__ void __launch_bounds__(kThreads, 4)
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
  // the warp's first element: its threads go one way
  const int64_t w = base + threadIdx.x / 32 * 32 * kEach;
  if (w >= t.n) return;
  const int64_t i = w + threadIdx.x % 32 * kEach;
  if (t.whole && w + 32 * kEach <= t.n)
    step_elements<BITS8, PARAM_BF16, GRAD_BF16, true>(a, h, t, k2, i, kEach);
  else
    step_elements<BITS8, PARAM_BF16, GRAD_BF16, false>(
        a, h, t, k2, i, static_cast<int>(max(int64_t(0), min(t.n - i, int64_t(kEach)))));
}

}  // namespace

int64_t adamw_chunk() { return kChunk; }

template <int CAP>
cudaError_t launch_adamw(const AdamWStep& a, const AdamWList<CAP>& l, uint32_t blocks, bool bits8,
                         cudaStream_t stream) {
  const auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3(blocks), dim3(kThreads), 0, stream, a, l);
  };
  const auto types = [&](auto bits) {
    constexpr bool B = decltype(bits)::value;
    if (a.param_bf16)
      return a.grad_bf16 ? go(adamw_kernel<B, true, true, CAP>)
                         : go(adamw_kernel<B, true, false, CAP>);
    return a.grad_bf16 ? go(adamw_kernel<B, false, true, CAP>)
                       : go(adamw_kernel<B, false, false, CAP>);
  };
  return bits8 ? types(std::true_type{}) : types(std::false_type{});
}
template cudaError_t launch_adamw(const AdamWStep&, const AdamWList<kAdamWFew>&, uint32_t, bool,
                                  cudaStream_t);
template cudaError_t launch_adamw(const AdamWStep&, const AdamWList<kAdamWMany>&, uint32_t, bool,
                                  cudaStream_t);

}  // namespace subm3d
