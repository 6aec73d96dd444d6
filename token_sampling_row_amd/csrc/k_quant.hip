// Per-row 8-bit codes of float rows (quantize_rows): weights per channel,
// hidden states per token.
#include "kernels.hpp"
#include "wide_mem.hpp"

namespace tsr {
namespace {

constexpr int kQuantBlock = 256;

// Codes of one 16-byte chunk. x / s is rounded to the nearest whole number,
// ties to even, as if the quotient were exact: q0 = rint(x * inv) is off by
// at most one, and the remainder r = x - q0 s of a code next to the quotient
// is a multiple of a unit of s below 2^24 of them, so the fma that forms it
// is exact and its comparison with s / 2 decides.
__device__ __forceinline__ int code_of(float x, float s, float inv) {
  float q = rintf(x * inv);
  const float r = fmaf(-q, s, x);
  const float h = 0.5f * s;
  const bool odd = ((int)q & 1) != 0;
  if (r > h || (r == h && odd)) q += 1.0f;
  if (r < -h || (r == -h && odd)) q -= 1.0f;
  return (int)fminf(fmaxf(q, -127.0f), 127.0f);
}

// One workgroup per row: the largest magnitude (as float bits, whose order is
// the values' with infinities and NaN above), then the codes.
template <int DT>
__global__ __launch_bounds__(kQuantBlock) void quant_kernel(const unsigned char* x,
                                                            long long stride_bytes, int width,
                                                            int8_t* q, long long q_stride,
                                                            float* scale) {
  constexpr int EPC = Fmt<DT>::EPC;
  __shared__ uint32_t wmax[kQuantBlock / kWave];
  const long long r = blockIdx.x;
  const unsigned char* row = x + r * stride_bytes;
  int8_t* qrow = q + r * q_stride;
  const int chunks = (width + EPC - 1) / EPC;
  uint32_t m = 0;
  for (int c = threadIdx.x; c < chunks; c += kQuantBlock) {
    float v[EPC];
    unpack<DT>(load_chunk_zero<DT>(row, (long long)c * EPC, width), v);
#pragma unroll
    for (int e = 0; e < EPC; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  }
  m = wave_max_u32(m);
  if ((threadIdx.x & (kWave - 1)) == 0) wmax[threadIdx.x / kWave] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQuantBlock / kWave; ++w) m = max(m, wmax[w]);
  const bool bad = m >= 0x7F800000u;   // an infinity or NaN in the row
  float s = __uint_as_float(m) * (1.0f / 127.0f);
  if (threadIdx.x == 0) scale[r] = bad ? __uint_as_float(0x7FC00000u) : s;
  // scales near or below the smallest normal number: both sides times 2^64,
  // which is exact and leaves every quotient as it is
  const float up = s < 0x1p-64f ? 0x1p64f : 1.0f;
  s *= up;
  const bool zero = bad || s == 0.0f;
  const float inv = zero ? 0.0f : 1.0f / s;
  for (int c = threadIdx.x; c < chunks; c += kQuantBlock) {
    float v[EPC];
    unpack<DT>(load_chunk_zero<DT>(row, (long long)c * EPC, width), v);
    uint32_t w[EPC / 4];
#pragma unroll
    for (int e = 0; e < EPC; e += 4) {
      uint32_t b = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int code = zero ? 0 : code_of(v[e + k] * up, s, inv);
        b |= (uint32_t)(code & 0xFF) << (8 * k);
      }
      w[e / 4] = b;
    }
    const int i0 = c * EPC;
    if (i0 + EPC <= width) {
      store_words<EPC / 4>(qrow + i0, w);
    } else {
      for (int e = 0; i0 + e < width; ++e) qrow[i0 + e] = (int8_t)(w[e / 4] >> (8 * (e % 4)));
    }
  }
}

}  // namespace

hipError_t launch_quantize(const void* x, int dtype, int rows, int width, long long stride_bytes,
                           int8_t* q, long long q_stride, float* scale, hipStream_t s) {
  const unsigned char* p = static_cast<const unsigned char*>(x);
  if (dtype == 0)
    hipLaunchKernelGGL((quant_kernel<0>), dim3(rows), dim3(kQuantBlock), 0, s, p, stride_bytes,
                       width, q, q_stride, scale);
  else
    hipLaunchKernelGGL((quant_kernel<1>), dim3(rows), dim3(kQuantBlock), 0, s, p, stride_bytes,
                       width, q, q_stride, scale);
  return hipGetLastError();
}

}  // namespace tsr
