// The RMS norm of rows with the residual's addition, as 8-bit codes
// (norm_quantize_rows): what int8_logits takes, from what a block leaves.
//
//   h = x + residual, rounded once to their type;  t_i = h_i w_i;  m = max |t|
//   code_i = 127 t_i / m to the nearest whole number, ties to even, exactly;
//   scale = m / (127 sqrt(mean(h^2) + eps)).
//
// The row's factor 1 / sqrt(...) is common to all of n_i = t_i / sqrt(...) and to
// their largest, so it cancels in the codes: they need the products alone, and the
// sum of squares and the largest product are formed in one pass. Products are
// formed in 64 bits, exactly; so is the sum of squares (no float32 square of a
// finite value overflows there).
#include "kernels.hpp"
#include "wide_mem.hpp"

namespace tsr {
namespace {

constexpr int kNormBlock = 256;

// 127 |t| / m to the nearest whole number, ties to even, as if the quotient were
// exact. `a` + `low` is 127 |t| without an error. The border between two codes is
// b = floor(quotient) + 1/2, and the sign of 127 |t| - b m says on which side the
// value lies: next to the border that difference is a multiple of the operands'
// last bits and small, so the fma gives it exactly; elsewhere its sign is plain.
__device__ __forceinline__ double exact_code(double t, double m) {
  const double v = fabs(t);
  const double a = 127.0 * v, low = fma(127.0, v, -a);
  const double f = floor(a / m);
  const double d = fma(-(f + 0.5), m, a) + low;
  double q = f;
  if (d > 0.0 || (d == 0.0 && ((int)f & 1))) q += 1.0;
  return copysign(fmin(q, 127.0), t);
}

template <int DT>
__device__ __forceinline__ float stored(float v) {   // rounded to the rows' type
  if constexpr (DT == 0) return v;
  return (float)(__bf16)v;
}

template <int DT>
__device__ __forceinline__ void store_elem(unsigned char* row, long long i, float v) {
  if constexpr (DT == 0)
    *reinterpret_cast<float*>(row + i * 4) = v;
  else
    *reinterpret_cast<uint16_t*>(row + i * 2) = __builtin_bit_cast(uint16_t, (__bf16)v);
}

template <int DT, int WT>
__global__ __launch_bounds__(kNormBlock) void norm_kernel(NormArgs a) {
  __shared__ BlockScratch scratch;
  const long long r = blockIdx.x;
  const unsigned char* x = a.x + r * a.x_stride;
  const unsigned char* res = a.residual ? a.residual + r * a.r_stride : nullptr;
  unsigned char* out_h = a.out_h ? a.out_h + r * a.h_stride : nullptr;
  double ss = 0.0, m = 0.0, bad = 0.0;
  for (int i = threadIdx.x; i < a.width; i += kNormBlock) {
    float h = load_elem<DT>(x, i);
    if (res) h = stored<DT>(h + load_elem<DT>(res, i));
    if (out_h) store_elem<DT>(out_h, i, h);
    const double w = a.weight ? (double)load_elem<WT>(a.weight, i) : 1.0;
    const double t = (double)h * w;
    ss = fma((double)h, (double)h, ss);
    m = fmax(m, fabs(t));
    bad += t * 0.0 + (double)h * 0.0;   // NaN where either is no finite number
  }
  ss = block_sum<kNormBlock>(ss, scratch);
  bad = block_sum<kNormBlock>(bad, scratch);
  // non-negative doubles order as their bits do
  const unsigned long long bits = (unsigned long long)__double_as_longlong(m);
  const uint32_t hi = block_max_u32<kNormBlock>((uint32_t)(bits >> 32), scratch);
  const uint32_t lo = block_max_u32<kNormBlock>(
      (uint32_t)(bits >> 32) == hi ? (uint32_t)bits : 0u, scratch);
  m = __longlong_as_double((long long)((unsigned long long)hi << 32 | lo));
  const bool fine = bad == 0.0;
  if (threadIdx.x == 0)
    a.scale[r] = !fine      ? __uint_as_float(0x7FC00000u)
                 : m == 0.0 ? 0.0f
                            : (float)(m / (127.0 * sqrt(ss / a.width + a.eps)));
  int8_t* q = a.codes + r * a.q_stride;
  for (int i = threadIdx.x; i < a.width; i += kNormBlock) {
    int code = 0;
    if (fine && m > 0.0) {
      float h;
      if (out_h) {   // x or the residual may be there no longer
        h = load_elem<DT>(out_h, i);
      } else {
        h = load_elem<DT>(x, i);
        if (res) h = stored<DT>(h + load_elem<DT>(res, i));
      }
      const double w = a.weight ? (double)load_elem<WT>(a.weight, i) : 1.0;
      code = (int)exact_code((double)h * w, m);
    }
    q[i] = (int8_t)code;
  }
}

}  // namespace

hipError_t launch_norm_quantize(const NormArgs& a, int dtype, int weight_dtype, hipStream_t s) {
  const dim3 grid(a.rows), block(kNormBlock);
  if (dtype == 0 && weight_dtype == 0)
    hipLaunchKernelGGL((norm_kernel<0, 0>), grid, block, 0, s, a);
  else if (dtype == 0)
    hipLaunchKernelGGL((norm_kernel<0, 1>), grid, block, 0, s, a);
  else if (weight_dtype == 0)
    hipLaunchKernelGGL((norm_kernel<1, 0>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((norm_kernel<1, 1>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace tsr
