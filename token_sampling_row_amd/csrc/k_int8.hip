// The 8-bit output projection (int8_logits): out[r][n] = sum_k x[r][k] w[n][k]
// in 32-bit integers, times the row's and the channel's scale.
#include "kernels.hpp"
#include "wide_mem.hpp"

namespace tsr {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v4i as_v4i(uint4 a) {
  return v4i{(int)a.x, (int)a.y, (int)a.z, (int)a.w};
}

// Wavefronts of a workgroup split the width; each holds 16 NT channels by
// 16 MT rows of accumulators, joined in LDS at the end.
//
// v_mfma_i32_16x16x64_i8: lane l gives row l % 16 of the first operand (here
// the weight's channels) and of the second (the hidden rows), 16 bytes at
// (l / 16) * 16 of the 64; it gets channels (l / 16) * 4 + 0..3 of hidden row
// l % 16. Tile t takes channels (i / 4) * 4 NT + t * 4 + i % 4 (i < 16), so
// that a lane ends with 4 NT neighbouring channels of one row.
template <int DT, int MT, int NT, int WV>
__global__ __launch_bounds__(WV* kWave) void int8_rows_kernel(Int8Args a) {
  constexpr int TILES = MT * NT;
  __shared__ v4i part[WV > 1 ? (WV - 1) * TILES * kWave : 1];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int i = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * (16 * NT);
  const int m0 = blockIdx.y * (16 * MT);
  const int8_t* wp[NT];
  const int8_t* xp[MT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int c = min(n0 + (i >> 2) * (4 * NT) + t * 4 + (i & 3), a.vocab - 1);
    wp[t] = a.w + (long long)c * a.w_stride;
  }
#pragma unroll
  for (int t = 0; t < MT; ++t)
    xp[t] = a.x + (long long)min(m0 + t * 16 + i, a.rows - 1) * a.x_stride;
  v4i acc[NT][MT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int u = 0; u < MT; ++u) acc[t][u] = v4i{0, 0, 0, 0};
  const int full = a.width / 64;
#pragma unroll 2
  for (int b = wave; b < full; b += WV) {
    const int k = b * 64 + g * 16;
    v4i wv[NT], xv[MT];
#pragma unroll
    for (int t = 0; t < NT; ++t) wv[t] = as_v4i(load16(wp[t] + k));
#pragma unroll
    for (int t = 0; t < MT; ++t) xv[t] = as_v4i(load16(xp[t] + k));
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int u = 0; u < MT; ++u)
        acc[t][u] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[t], xv[u], acc[t][u], 0, 0, 0);
  }
  if (full * 64 < a.width && wave == full % WV) {   // the partial last block
    const int k = full * 64 + g * 16;
    v4i xv[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) xv[t] = as_v4i(load_bytes_zero(xp[t], k, a.width));
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const v4i wv = as_v4i(load_bytes_zero(wp[t], k, a.width));
#pragma unroll
      for (int u = 0; u < MT; ++u)
        acc[t][u] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv, xv[u], acc[t][u], 0, 0, 0);
    }
  }
  if constexpr (WV > 1) {
    if (wave > 0) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u)
          part[((wave - 1) * TILES + t * MT + u) * kWave + lane] = acc[t][u];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int v = 0; v < WV - 1; ++v)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u) acc[t][u] += part[(v * TILES + t * MT + u) * kWave + lane];
  }
  const int c0 = n0 + g * (4 * NT);
#pragma unroll
  for (int u = 0; u < MT; ++u) {
    const int r = m0 + u * 16 + i;
    if (r >= a.rows) continue;
    const float xs = a.x_scale[r];
    float v[4 * NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = min(c0 + t * 4 + e, a.vocab - 1);
        v[t * 4 + e] = fmaf((float)acc[t][u][e] * xs, a.w_scale[c], a.bias ? a.bias[c] : 0.0f);
      }
    store_row<DT, 4 * NT>(a.out + (long long)r * a.out_stride_bytes, c0, a.vocab, v);
  }
}

template <int DT>
hipError_t launch_int8_dt(const Int8Args& a, hipStream_t s) {
  constexpr int NT = 4, WV = 4;
  const dim3 grid((a.vocab + 16 * NT - 1) / (16 * NT), (a.rows + 63) / 64);
  if (a.rows <= 16)
    hipLaunchKernelGGL((int8_rows_kernel<DT, 1, NT, WV>), grid, dim3(WV * kWave), 0, s, a);
  else if (a.rows <= 32)
    hipLaunchKernelGGL((int8_rows_kernel<DT, 2, NT, WV>), grid, dim3(WV * kWave), 0, s, a);
  else
    hipLaunchKernelGGL((int8_rows_kernel<DT, 4, NT, WV>), grid, dim3(WV * kWave), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8(const Int8Args& a, int dtype, hipStream_t s) {
  return dtype == 0 ? launch_int8_dt<0>(a, s) : launch_int8_dt<1>(a, s);
}

}  // namespace tsr
