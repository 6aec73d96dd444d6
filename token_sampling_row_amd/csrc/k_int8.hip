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

// A buffer of `rows` rows of `width` bytes, `stride` apart (less than 2^32 bytes).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const int8_t* p, uint32_t rows,
                                                            long long stride, int width) {
  const uint32_t bytes = (rows - 1) * (uint32_t)stride + (uint32_t)width;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(p), 0, (int)bytes, 0x00027000);
}
// 16 bytes per lane from byte at + k of a buffer to `p` + 16 lane in LDS. (The
// host pass of the compiler does not know the 16-byte form.)
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t buffer, int8_t* p, uint32_t at,
                                       int k) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer, (__attribute__((address_space(3))) void*)p, 16,
                                           (int)at, k, 0, 0);
#endif
}

constexpr int kTileK = 128;   // bytes of the width a stage holds of each row

// Tiles of BM hidden rows by BN channels, WM x WN wavefronts each MT x NT
// blocks of 16 x 16.
//
// A stage holds kTileK bytes of each row as eight 16-byte chunks; chunk c of
// LDS row r lies at place c ^ (r & 7), so the 16 lanes that read one chunk
// of 16 rows meet every bank once in each group of eight. LDS rows of the
// weight hold channels in the order that leaves a lane with 4 NT neighbouring
// channels (see int8_rows_kernel).
template <int DT, int BM, int BN, int WM, int WN, bool DIRECT>
__global__ __launch_bounds__(WM* WN* kWave) void int8_tile_kernel(Int8Args a, int m_tiles,
                                                                  int tiles) {
  constexpr int WAVES = WM * WN;
  constexpr int MT = BM / (16 * WM), NT = BN / (16 * WN);
  constexpr int XI = BM / 8 / WAVES, WI = BN / 8 / WAVES;   // 1 KiB pieces per wavefront
  static_assert(XI * 8 * WAVES == BM && WI * 8 * WAVES == BN, "pieces");
  __shared__ __attribute__((aligned(1024))) int8_t x0[BM * kTileK];
  __shared__ __attribute__((aligned(1024))) int8_t x1[BM * kTileK];
  __shared__ __attribute__((aligned(1024))) int8_t w0[BN * kTileK];
  __shared__ __attribute__((aligned(1024))) int8_t w1[BN * kTileK];
  // workgroups go round the eight XCDs: each gets a run of tiles, the hidden
  // rows' tiles of one run of channels next to each other (they share its L2)
  const int per = (tiles + 7) / 8;
  const int tile = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (tile >= tiles) return;
  const int m0 = (tile % m_tiles) * BM, n0 = (tile / m_tiles) * BN;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave % WM, wn = wave / WM;
  const int lr = lane >> 3, lc = ((lane & 7) ^ lr) * 16;
  auto channel_of = [](int r) {   // which of the tile's channels LDS row r holds
    const int i = r & 15, t = (r % (16 * NT)) / 16;
    return r / (16 * NT) * (16 * NT) + (i >> 2) * (4 * NT) + t * 4 + (i & 3);
  };
  // from the tile's first row and channel: 32-bit offsets (checked at launch)
  const int8_t* xb = a.x + (long long)m0 * a.x_stride;
  const int8_t* wb = a.w + (long long)n0 * a.w_stride;
  uint32_t xo[XI], wo[WI];
#pragma unroll
  for (int q = 0; q < XI; ++q) {
    const int r = (wave * XI + q) * 8 + lr;
    xo[q] = (uint32_t)min(r, a.rows - 1 - m0) * (uint32_t)a.x_stride + lc;
  }
#pragma unroll
  for (int q = 0; q < WI; ++q) {
    const int r = (wave * WI + q) * 8 + lr;
    wo[q] = (uint32_t)min(channel_of(r), a.vocab - 1 - n0) * (uint32_t)a.w_stride + lc;
  }
  const int whole = a.width / kTileK;
  // the tile's bytes end with the last byte of its last row
  const auto xr = buffer_of(xb, (uint32_t)min(BM, a.rows - m0), a.x_stride, a.width);
  const auto wr = buffer_of(wb, (uint32_t)min(BN, a.vocab - n0), a.w_stride, a.width);

  v4i acc[NT][MT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int u = 0; u < MT; ++u) acc[t][u] = v4i{0, 0, 0, 0};

  // Stage b on its way: straight into LDS, or into registers that `place` puts
  // there.
  uint4 rx[DIRECT ? 1 : XI], rw[DIRECT ? 1 : WI];
  auto fetch = [&](int b, int8_t* xs, int8_t* wsm) {
    const int k = b * kTileK;
    if constexpr (DIRECT) {
#pragma unroll
      for (int q = 0; q < XI; ++q)
        to_lds(xr, xs + (wave * XI + q) * 1024, xo[q], k);
#pragma unroll
      for (int q = 0; q < WI; ++q)
        to_lds(wr, wsm + (wave * WI + q) * 1024, wo[q], k);
    } else {
#pragma unroll
      for (int q = 0; q < XI; ++q) rx[q] = load16(xb + k + xo[q]);
#pragma unroll
      for (int q = 0; q < WI; ++q) rw[q] = load16(wb + k + wo[q]);
    }
  };
  auto place = [&](int8_t* xs, int8_t* wsm) {
    if constexpr (!DIRECT) {
#pragma unroll
      for (int q = 0; q < XI; ++q)
        *reinterpret_cast<uint4*>(xs + (wave * XI + q) * 1024 + lane * 16) = rx[q];
#pragma unroll
      for (int q = 0; q < WI; ++q)
        *reinterpret_cast<uint4*>(wsm + (wave * WI + q) * 1024 + lane * 16) = rw[q];
    }
  };
  const int fr = lane & 15, fg = lane >> 4;
  auto multiply = [&](const int8_t* xs, const int8_t* wsm) {
#pragma unroll
    for (int h = 0; h < kTileK / 64; ++h) {
      const int at = fr * kTileK + (((h * 4 + fg) ^ (fr & 7)) * 16);
      v4i wv[NT], xv[MT];
#pragma unroll
      for (int t = 0; t < NT; ++t)
        wv[t] = *reinterpret_cast<const v4i*>(wsm + (wn * NT + t) * 16 * kTileK + at);
#pragma unroll
      for (int u = 0; u < MT; ++u)
        xv[u] = *reinterpret_cast<const v4i*>(xs + (wm * MT + u) * 16 * kTileK + at);
#pragma unroll
      for (int u = 0; u < MT; ++u)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          acc[t][u] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[t], xv[u], acc[t][u], 0, 0, 0);
      sched_fence();
    }
  };

  if (whole > 0) fetch(0, x0, w0);
  if (whole * kTileK < a.width) {
    // the partial stage comes first, beside the first whole one's loads
    const int k = whole * kTileK + lc;
#pragma unroll 1
    for (int q = 0; q < XI; ++q) {
      const int r = (wave * XI + q) * 8;
      const int8_t* row = xb + (long long)min(r + lr, a.rows - 1 - m0) * a.x_stride;
      *reinterpret_cast<uint4*>(x1 + r * kTileK + lane * 16) = load_bytes_zero(row, k, a.width);
    }
#pragma unroll 1
    for (int q = 0; q < WI; ++q) {
      const int r = (wave * WI + q) * 8;
      const int8_t* row =
          wb + (long long)min(channel_of(r + lr), a.vocab - 1 - n0) * a.w_stride;
      *reinterpret_cast<uint4*>(w1 + r * kTileK + lane * 16) = load_bytes_zero(row, k, a.width);
    }
    __syncthreads();
    multiply(x1, w1);
  }
  if (whole > 0) {
    place(x0, w0);
    __syncthreads();
    int b = 0;
    for (; b + 2 < whole; b += 2) {
      fetch(b + 1, x1, w1);
      multiply(x0, w0);
      place(x1, w1);
      __syncthreads();
      fetch(b + 2, x0, w0);
      multiply(x1, w1);
      place(x0, w0);
      __syncthreads();
    }
    const bool two = b + 1 < whole;
    if (two) fetch(b + 1, x1, w1);
    multiply(x0, w0);
    if (two) {
      place(x1, w1);
      __syncthreads();
      multiply(x1, w1);
    }
  }

  const int c0 = n0 + wn * (16 * NT) + fg * (4 * NT);
  float ws[4 * NT], bs[4 * NT];
#pragma unroll
  for (int e = 0; e < 4 * NT; ++e) {
    const int c = min(c0 + e, a.vocab - 1);
    ws[e] = a.w_scale[c];
    bs[e] = a.bias ? a.bias[c] : 0.0f;
  }
#pragma unroll
  for (int u = 0; u < MT; ++u) {
    const int r = m0 + (wm * MT + u) * 16 + fr;
    if (r >= a.rows) continue;
    const float xs = a.x_scale[r];
    float v[4 * NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[t * 4 + e] = fmaf((float)acc[t][u][e] * xs, ws[t * 4 + e], bs[t * 4 + e]);
    store_row<DT, 4 * NT>(a.out + (long long)r * a.out_stride_bytes, c0, a.vocab, v);
  }
}

template <int DT, int BM, int BN, int WM, int WN>
hipError_t launch_tile(const Int8Args& a, bool direct, hipStream_t s) {
  const int m_tiles = (a.rows + BM - 1) / BM, n_tiles = (a.vocab + BN - 1) / BN;
  const int tiles = m_tiles * n_tiles;
  const dim3 grid((tiles + 7) / 8 * 8), block(WM * WN * kWave);
  if (direct)
    hipLaunchKernelGGL((int8_tile_kernel<DT, BM, BN, WM, WN, true>), grid, block, 0, s, a, m_tiles,
                       tiles);
  else
    hipLaunchKernelGGL((int8_tile_kernel<DT, BM, BN, WM, WN, false>), grid, block, 0, s, a,
                       m_tiles, tiles);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_int8_dt(const Int8Args& a, hipStream_t s) {
  const bool direct = a.width % 16 == 0 && a.x_stride % 16 == 0 && a.w_stride % 16 == 0 &&
                      (uintptr_t)a.x % 16 == 0 && (uintptr_t)a.w % 16 == 0;
  const bool near = a.x_stride < (1 << 23) && a.w_stride < (1 << 23);   // 256 rows within 2^31
  if (near && a.rows > 128) return launch_tile<DT, 256, 256, 2, 4>(a, direct, s);
  if (near && a.rows > 64) return launch_tile<DT, 128, 256, 2, 4>(a, direct, s);
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
