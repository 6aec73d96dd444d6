// Per-row 8-bit codes of float rows (quantize_rows): weights per channel,
// hidden states per token. s = max |x| / 127, q = x / s to the nearest.
//
// Bound by memory: a row is read once, held in registers between its largest
// magnitude and its codes. 32000 x 4096 bf16 (393 MB) 62 us, 6.3 TB/s (a copy
// runs at 5.1, reads alone at 6.9); 333 x 5003 fp32 4.7 us and 5 x 4096 bf16 2.8,
// a launch, one trip to memory and back.
#include "kernels.hpp"
#include "wide_mem.hpp"

namespace tsr {
namespace {

constexpr int kQuantBlock = 256;
// Inputs of more bytes than this are read past the caches, which could not keep
// them: 32000 x 4096 bf16 62 us against 67. Smaller ones may be there still:
// 16384 x 4096 bf16 31 us read from them, 34 past them.
constexpr long long kQuantOnceBytes = 192ll << 20;

// A row's scale from the bits of its largest magnitude (float bits order as the
// values do, infinities and NaN above).
struct RowScale {
  float s, inv, up;   // s and its reciprocal, both sides scaled by up
  float out;          // what is stored
  __device__ __forceinline__ explicit RowScale(uint32_t top) {
    s = __uint_as_float(top) * (1.0f / 127.0f);
    const bool bad = top >= 0x7F800000u;   // an infinity or NaN in the row
    out = bad ? __uint_as_float(0x7FC00000u) : s;
    // scales near or below the smallest normal number: both sides times 2^64,
    // which is exact and leaves every quotient as it is
    up = s < 0x1p-64f ? 0x1p64f : 1.0f;
    s *= up;
    if (bad) s = 0.0f;
    inv = s == 0.0f ? 0.0f : 1.0f / s;   // 0: every code is 0
  }
};

// x / s to the nearest whole number, ties to even, as if the quotient were
// exact: q = rint(x * inv) is off by at most one, the remainder r = x - q s is
// exact where it is near s / 2 (a multiple of a unit of s, below 2^24 of them),
// and decides.
__device__ __forceinline__ float nearest(float x, const RowScale& a) {
  float q = rintf(x * a.inv);
  const float r = fmaf(-q, a.s, x);
  const float h = 0.5f * a.s;
  const bool odd = ((int)q & 1) != 0;
  if (r > h || (r == h && odd)) q += 1.0f;
  if (r < -h || (r == -h && odd)) q -= 1.0f;
  return q;
}

// Codes of one chunk, four to a word. The remainders are looked at together:
// only a chunk with one at or past s / 2 takes the corrected quotients.
template <int DT>
__device__ __forceinline__ void codes_of(uint4 chunk, const RowScale& a, uint32_t* words) {
  constexpr int EPC = Fmt<DT>::EPC;
  float v[EPC], q[EPC];
  unpack<DT>(chunk, v);
  float far = 0.0f;
#pragma unroll
  for (int e = 0; e < EPC; ++e) {
    v[e] *= a.up;
    q[e] = rintf(v[e] * a.inv);
    far = fmaxf(far, fabsf(fmaf(-q[e], a.s, v[e])));
  }
  if (far >= 0.5f * a.s) {
#pragma unroll
    for (int e = 0; e < EPC; ++e) q[e] = a.s == 0.0f ? 0.0f : nearest(v[e], a);
  }
#pragma unroll
  for (int e = 0; e < EPC; e += 4) {
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)   // code + 128 as an unsigned byte
      w = __builtin_amdgcn_cvt_pk_u8_f32(fminf(fmaxf(q[e + k], -127.0f), 127.0f) + 128.0f, k, w);
    words[e / 4] = w ^ 0x80808080u;
  }
}

template <int DT>
__device__ __forceinline__ uint32_t top_of(uint4 chunk) {
  float v[Fmt<DT>::EPC];
  unpack<DT>(chunk, v);
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < Fmt<DT>::EPC; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  return m;
}

template <int DT>
__device__ __forceinline__ void store_codes(int8_t* row, int i0, int width, const uint32_t* w) {
  constexpr int EPC = Fmt<DT>::EPC;
  if (i0 + EPC <= width) {
    store_words<EPC / 4>(row + i0, w);
  } else {
#pragma unroll
    for (int e = 0; e < EPC; ++e)
      if (i0 + e < width) row[i0 + e] = (int8_t)(w[e / 4] >> (8 * (e % 4)));
  }
}

// The largest of `m` over the WPR wavefronts of a row, neighbours in the workgroup.
template <int WPR>
__device__ __forceinline__ uint32_t row_top(uint32_t m) {
  m = wave_max_u32(m);
  if constexpr (WPR > 1) {
    __shared__ uint32_t each[kQuantBlock / kWave];
    if ((threadIdx.x & (kWave - 1)) == 0) each[threadIdx.x / kWave] = m;
    __syncthreads();
    const int first = threadIdx.x / (WPR * kWave) * WPR;
#pragma unroll
    for (int w = 0; w < WPR; ++w) m = max(m, each[first + w]);
  }
  return m;
}

// Rows of up to NC chunks a lane, in registers; WPR wavefronts to a row, four in
// a workgroup. ONCE: read past the caches.
template <int DT, int WPR, int NC, bool ONCE>
__global__ __launch_bounds__(kQuantBlock) void quant_kernel(const unsigned char* x,
                                                            long long stride_bytes, int rows,
                                                            int width, int8_t* q,
                                                            long long q_stride, float* scale) {
  constexpr int EPC = Fmt<DT>::EPC, T = WPR * kWave, RPB = kQuantBlock / T;
  const int part = __builtin_amdgcn_readfirstlane(threadIdx.x / T);
  const int t = threadIdx.x % T;
  const long long r = (long long)blockIdx.x * RPB + part;
  const unsigned char* row = x + min(r, (long long)rows - 1) * stride_bytes;
  const int whole = width / EPC;   // at least one
  uint4 c[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) {   // chunks past the last whole one repeat it
    const unsigned char* p = row + (long long)min(j * T + t, whole - 1) * 16;
    c[j] = ONCE ? load16_once(p) : load16(p);
  }
  uint4 rest{};
  const bool partial = whole * EPC < width && t == whole % T;
  if (partial) rest = load_chunk_zero<DT>(row, (long long)whole * EPC, width);
  uint32_t m = top_of<DT>(rest);
#pragma unroll
  for (int j = 0; j < NC; ++j) m = max(m, top_of<DT>(c[j]));
  const RowScale a(row_top<WPR>(m));
  if (r >= rows) return;
  if (t == 0) scale[r] = a.out;
  int8_t* out = q + r * q_stride;
  uint32_t w[EPC / 4];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    if (j * T + t < whole) {
      codes_of<DT>(c[j], a, w);
      store_words<EPC / 4>(out + (long long)(j * T + t) * EPC, w);
    }
  }
  if (partial) {
    codes_of<DT>(rest, a, w);
    store_codes<DT>(out, whole * EPC, width, w);
  }
}

// Rows of any width: read twice, the second time from the caches.
template <int DT>
__global__ __launch_bounds__(kQuantBlock) void quant_wide_kernel(const unsigned char* x,
                                                                 long long stride_bytes, int width,
                                                                 int8_t* q, long long q_stride,
                                                                 float* scale) {
  constexpr int EPC = Fmt<DT>::EPC;
  const long long r = blockIdx.x;
  const unsigned char* row = x + r * stride_bytes;
  const int chunks = (width + EPC - 1) / EPC;
  uint32_t m = 0;
  for (int c = threadIdx.x; c < chunks; c += kQuantBlock)
    m = max(m, top_of<DT>(load_chunk_zero<DT>(row, (long long)c * EPC, width)));
  const RowScale a(row_top<kQuantBlock / kWave>(m));
  if (threadIdx.x == 0) scale[r] = a.out;
  for (int c = threadIdx.x; c < chunks; c += kQuantBlock) {
    uint32_t w[EPC / 4];
    codes_of<DT>(load_chunk_zero<DT>(row, (long long)c * EPC, width), a, w);
    store_codes<DT>(q + r * q_stride, c * EPC, width, w);
  }
}

template <int DT, int WPR, int NC, bool ONCE>
hipError_t launch_nc(const unsigned char* x, int rows, int width, long long stride_bytes,
                     int8_t* q, long long q_stride, float* scale, hipStream_t s) {
  constexpr int RPB = kQuantBlock / (WPR * kWave);
  hipLaunchKernelGGL((quant_kernel<DT, WPR, NC, ONCE>), dim3((rows + RPB - 1) / RPB),
                     dim3(kQuantBlock), 0, s, x, stride_bytes, rows, width, q, q_stride, scale);
  return hipGetLastError();
}

template <int DT, int WPR, bool ONCE>
hipError_t launch_wpr(const unsigned char* x, int rows, int width, long long stride_bytes,
                      int8_t* q, long long q_stride, float* scale, hipStream_t s) {
  // the rule below leaves two wavefronts two chunks a lane at least, and four as
  // many of a large input; fewer than four take three at most
  constexpr bool ONE = WPR == 1 || (WPR == 4 && !ONCE);
  const int per = (width / Fmt<DT>::EPC + WPR * kWave - 1) / (WPR * kWave);
  if constexpr (ONE)
    if (per <= 1)
      return launch_nc<DT, WPR, 1, ONCE>(x, rows, width, stride_bytes, q, q_stride, scale, s);
  if (per <= 2)
    return launch_nc<DT, WPR, 2, ONCE>(x, rows, width, stride_bytes, q, q_stride, scale, s);
  if constexpr (WPR < 4)
    return launch_nc<DT, WPR, 3, ONCE>(x, rows, width, stride_bytes, q, q_stride, scale, s);
  if (per <= 4)
    return launch_nc<DT, WPR, 4, ONCE>(x, rows, width, stride_bytes, q, q_stride, scale, s);
  return launch_nc<DT, WPR, 8, ONCE>(x, rows, width, stride_bytes, q, q_stride, scale, s);
}

// Wavefronts to a row. Many rows fill the card however they are cut, and fewer
// wavefronts to a row spend less on their largest value; past three chunks a
// lane the registers leave too few rows on their way. In us with 1, 2 and 4:
// bf16 126953 x 1024 66 79 118, 84635 x 1536 64 72 91, 16384 x 2048 21 21 23,
// 50781 x 2560 68 65 75, 31738 x 4096 64 62 62. Few rows are bound by the time of
// one: 2048 x 1024 4.4 4.3 4.6, 2048 x 2048 6.2 5.5 5.2, 300 x 4096 7.3 4.9 4.3.
template <int DT, bool ONCE>
hipError_t launch_once(const unsigned char* x, int rows, int width, long long stride_bytes,
                       int8_t* q, long long q_stride, float* scale, hipStream_t s) {
  const int whole = width / Fmt<DT>::EPC;
  if (whole <= (rows >= 4096 ? 3 : 2) * kWave)
    return launch_wpr<DT, 1, ONCE>(x, rows, width, stride_bytes, q, q_stride, scale, s);
  if (rows >= 4096 && whole <= 6 * kWave)
    return launch_wpr<DT, 2, ONCE>(x, rows, width, stride_bytes, q, q_stride, scale, s);
  return launch_wpr<DT, 4, ONCE>(x, rows, width, stride_bytes, q, q_stride, scale, s);
}

template <int DT>
hipError_t launch_dt(const unsigned char* x, int rows, int width, long long stride_bytes,
                     int8_t* q, long long q_stride, float* scale, hipStream_t s) {
  const int whole = width / Fmt<DT>::EPC;
  if (whole < 1 || whole > 8 * kQuantBlock) {
    hipLaunchKernelGGL((quant_wide_kernel<DT>), dim3(rows), dim3(kQuantBlock), 0, s, x,
                       stride_bytes, width, q, q_stride, scale);
    return hipGetLastError();
  }
  return (long long)rows * width * Fmt<DT>::ESZ > kQuantOnceBytes
             ? launch_once<DT, true>(x, rows, width, stride_bytes, q, q_stride, scale, s)
             : launch_once<DT, false>(x, rows, width, stride_bytes, q, q_stride, scale, s);
}

}  // namespace

hipError_t launch_quantize(const void* x, int dtype, int rows, int width, long long stride_bytes,
                           int8_t* q, long long q_stride, float* scale, hipStream_t s) {
  const unsigned char* p = static_cast<const unsigned char*>(x);
  return dtype == 0 ? launch_dt<0>(p, rows, width, stride_bytes, q, q_stride, scale, s)
                    : launch_dt<1>(p, rows, width, stride_bytes, q, q_stride, scale, s);
}

}  // namespace tsr
