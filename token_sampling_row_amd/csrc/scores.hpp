// What the kernels around the logits share (token_logprobs, distill_topk):
// weights of logits against a row's largest, log probabilities, keys of the
// likeliest ids, and the gradient p_j (A + B x_j) with its stores.
#pragma once

#include "device_common.hpp"

namespace tsr {

constexpr double kLn2 = 0.6931471805599453;

// (v - M) log2(e) / T. Held above -2000, where the weight 2^x is 0 anyway, so
// that a logit of -inf gives products of 0 and not NaN.
__device__ __forceinline__ float exponent(float v, float M, float c) {
  return fmaxf((v - M) * c, -2000.0f);
}

// The elements of a chunk as the pass sees them. Passes over the same registers unpack
// bf16 anew: kept from one pass to the next the values would take twice the chunks'
// registers. A shift and a mask that the compiler does not know to be the other pass's
// keep it from that (bf16, 16 chunks: 82 registers against 158).
struct Pass {
  int sixteen;
  uint32_t high;
  __device__ __forceinline__ Pass() {
    asm volatile("s_mov_b32 %0, 16" : "=s"(sixteen));
    asm volatile("s_mov_b32 %0, 0xffff0000" : "=s"(high));
  }
  template <int DT>
  __device__ __forceinline__ void unpack(const uint4 r, float* v) const {
    if constexpr (DT == 0) {
      tsr::unpack<0>(r, v);
    } else {
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << sixteen);
        v[2 * i + 1] = __uint_as_float(w[i] & high);
      }
    }
  }
};

// e^x in 64 bits with few registers (the library's exponential takes dozens, in kernels
// that hold a row in theirs): e^r for r = x / 2^16 from its series to r^4, then squared
// sixteen times. 2^16 times the base's error of 2^-53 and r^5 / 120: under 2^-36 relative
// for |x| < 100, where results are not negligible.
__device__ __forceinline__ double exp_small(double x) {
  const double r = fmax(x, -740.0) * 0x1p-16;
  double y = fma(r, fma(r, fma(r, fma(r, 1.0 / 24.0, 1.0 / 6.0), 0.5), 1.0), 1.0);
#pragma unroll
  for (int i = 0; i < 16; ++i) y *= y;
  return x < -740.0 ? 0.0 : y;
}
// ln a, a > 0: y from the hardware's log2 of a's mantissa m (2^-23 off), then the step to
// y + ln(m e^-y), whose argument is next to 1: exact to 2^-36.
__device__ __forceinline__ double log_small(double a) {
  int e;
  const double m = frexp(a, &e);
  const double y = (double)__builtin_amdgcn_logf((float)m) * kLn2;
  const double d = fma(m, exp_small(-y), -1.0);
  return fma((double)e, kLn2, y + fma(-0.5 * d, d, d));
}

// log p of a logit v: (v - M) / T - log Z, formed in 64 bits and rounded once.
__device__ __forceinline__ float log_prob(float v, float M, double logZ, double inv_t) {
  return (float)(((double)v - (double)M) * inv_t - logZ);
}

constexpr uint32_t kKeyNegInf = 0x007FFFFFu;   // fkey(-inf)
// Keys of ids that order as (value, then the lower id) do; 0 is below all of them.
__device__ __forceinline__ unsigned long long top_key(float v, int id) {
  return ((unsigned long long)fkey(v) << 32) | (0xFFFFFFFFu - (uint32_t)id);
}
__device__ __forceinline__ int top_id(unsigned long long key) {
  return (int)(0xFFFFFFFFu - (uint32_t)key);
}
__device__ __forceinline__ float top_value(unsigned long long key) {
  return key2f((uint32_t)(key >> 32));
}

// A row's gradient: e (A + B X), e = 2^X, X = (z - M) log2(e) / T. X is formed in one fma
// against rc = fl(M c); what it is short of, rc - M c, is the same for the whole row,
// known exactly, and goes into A and B. Where M c is so large that this is no small
// shift, the difference is formed first.
struct GradRow {
  float M, c, rc, A, B;
  bool plain;   // the difference first
  __device__ __forceinline__ GradRow(float M, float c, double A0, double B0) : M(M), c(c) {
    rc = M * c;
    const float off = -fmaf(M, c, -rc);
    plain = !(fabsf(rc) <= 0x1p20f);
    const double f = plain ? 1.0 : (double)__builtin_amdgcn_exp2f(off);
    A = (float)(plain ? A0 : f * (A0 + B0 * (double)off));
    B = (float)(f * B0);
  }
  // Exponents are held above -2000 where B counts: a logit of -inf has a gradient of 0
  template <bool WITH_B, bool PLAIN>
  __device__ __forceinline__ float of(float z) const {
    if constexpr (PLAIN) {
      const float x = exponent(z, M, c);
      return __builtin_amdgcn_exp2f(x) * fmaf(B, x, A);
    }
    float x = fmaf(z, c, -rc);
    if constexpr (!WITH_B) return __builtin_amdgcn_exp2f(x) * A;
    x = fmaxf(x, -2000.0f);
    return __builtin_amdgcn_exp2f(x) * fmaf(B, x, A);
  }
  __device__ __forceinline__ float at(float z) const {
    return plain ? of<true, true>(z) : B != 0.0f ? of<true, false>(z) : of<false, false>(z);
  }
};

// Two floats as bfloat16 in one instruction, each to nearest even; the first below.
typedef float Float2 __attribute__((ext_vector_type(2)));
typedef __bf16 Bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16_both(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(Float2{a, b}, Bf16x2));
}

// A chunk of floats in the rows' type.
template <int DT>
__device__ __forceinline__ uint4 pack(const float* v) {
  if constexpr (DT == 0)
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  else
    return make_uint4(bf16_both(v[0], v[1]), bf16_both(v[2], v[3]), bf16_both(v[4], v[5]),
                      bf16_both(v[6], v[7]));
}

template <int DT>
__device__ __forceinline__ void store_elem(unsigned char* row, long long i, float v) {
  if constexpr (DT == 0)
    *reinterpret_cast<float*>(row + i * 4) = v;
  else
    *reinterpret_cast<uint16_t*>(row + i * 2) = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// The workgroup's largest value, NaN where there is one.
template <int BLOCK>
__device__ __forceinline__ float block_maxn(float v, BlockScratch& s) {
  constexpr int W = BLOCK / kWave;
  v = wave_maxn(v);
  __syncthreads();
  if (__lane_id() == 0) s.f[threadIdx.x / kWave] = v;
  __syncthreads();
  float r = s.f[0];
#pragma unroll
  for (int w = 1; w < W; ++w) r = fmaxn(r, s.f[w]);
  return r;
}

template <int BLOCK>
__device__ __forceinline__ unsigned long long block_max_u64(unsigned long long v,
                                                            BlockScratch& s) {
  constexpr int W = BLOCK / kWave;
  v = wave_reduce(v, [](unsigned long long a, unsigned long long b) { return a > b ? a : b; });
  __syncthreads();
  if (__lane_id() == 0) s.q[threadIdx.x / kWave] = v;
  __syncthreads();
  unsigned long long r = s.q[0];
#pragma unroll
  for (int w = 1; w < W; ++w) r = s.q[w] > r ? s.q[w] : r;
  return r;
}

}  // namespace tsr
