// The RMS norm of rows with the residual's addition, as 8-bit codes
// (norm_quantize_rows): what int8_logits takes, from what a block leaves.
//
//   h = x + residual, rounded once to their type;  t_i = h_i w_i;  m = max |t|
//   code_i = 127 t_i / m to the nearest whole number, ties to even, exactly;
//   scale = m / (127 sqrt(mean(h^2) + eps)).
//
// The row's factor 1 / sqrt(...) is common to all of n_i = t_i / sqrt(...) and to
// their largest, so it cancels in the codes: they need the products alone, and the
// sum of squares and the largest product are formed in one pass over the row, which
// stays in registers until its codes are written.
//
// Exactness. Products are formed in float32, off by 2^-24 at most, and so is the
// quotient q = t (127 / m), by 2^-22 of itself or 2^-15 at most. A chunk with a q that
// near to a half, one in some hundred, goes through 64 bits, where products of float32
// values have no error. Two float32 products order as the exact ones do unless they are
// equal, so m is the largest exact one among those equal to the largest float32 one.
// The sum of squares is formed in 64 bits: no square of a finite value overflows.
//
// Bound by memory where there are many rows: x and the residual are read once, their sum
// and the codes written once. Measured: 16384 x 4096 bf16 with a residual and float32
// weights 75 to 77 us (6.2 TB/s, vector pipes 83 % busy), 333 x 5003 fp32 7.6 us,
// 1 x 4096 3.3 us, a launch's and a row's latencies.
#include "kernels.hpp"
#include "scores.hpp"
#include "wide_mem.hpp"

namespace tsr {
namespace {

constexpr int kNormBlock = 256;

// Whether v is above b m / 127 (a value on it: whether `odd`): b is a border between two
// codes, a whole number and a half. `a` + `low` is 127 v without an error. Next to the
// border 127 v - b m is a multiple of the operands' last bits and small, so the fma gives
// it exactly; elsewhere its sign is plain.
__device__ __forceinline__ bool side_of(double v, double b, double m, bool odd) {
  const double a = 127.0 * v, low = fma(127.0, v, -a);
  const double d = fma(-b, m, a) + low;
  return d > 0.0 || (d == 0.0 && odd);
}

// 127 t / m to the nearest whole number, ties to even, as if the quotient were exact.
__device__ __forceinline__ double exact_code(double t, double m) {
  const double v = fabs(t), f = floor(127.0 * v / m);
  return copysign(fmin(side_of(v, f + 0.5, m, (int)f & 1) ? f + 1.0 : f, 127.0), t);
}

template <int DT>
__device__ __forceinline__ float stored(float v) {   // rounded to the rows' type
  if constexpr (DT == 0) return v;
  return (float)(__bf16)v;
}

// EPC weights from element i on; past the row's last one 0.
template <int EPC, int WT>
__device__ __forceinline__ void load_weights(const unsigned char* w, int i, int n, float* out) {
  if (!w) {
#pragma unroll
    for (int e = 0; e < EPC; ++e) out[e] = 1.0f;
  } else if (i + EPC <= n) {
    if constexpr (WT == 1 && EPC == 8) {
      unpack<1>(load16(w + (long long)i * 2), out);
    } else if constexpr (WT == 1) {
      const Bytes8 b = *reinterpret_cast<const Bytes8*>(w + (long long)i * 2);
      float v[8];
      unpack<1>(make_uint4(b.w[0], b.w[1], 0, 0), v);
#pragma unroll
      for (int e = 0; e < EPC; ++e) out[e] = v[e];
    } else {
#pragma unroll
      for (int e = 0; e < EPC; e += 4) unpack<0>(load16(w + ((long long)i + e) * 4), out + e);
    }
  } else {
#pragma unroll
    for (int e = 0; e < EPC; ++e) out[e] = i + e < n ? load_elem<WT>(w, i + e) : 0.0f;
  }
}

template <int DT>
__device__ __forceinline__ uint4 add_chunks(uint4 x, uint4 r) {
  float a[Fmt<DT>::EPC], b[Fmt<DT>::EPC];
  unpack<DT>(x, a);
  unpack<DT>(r, b);
#pragma unroll
  for (int e = 0; e < Fmt<DT>::EPC; ++e) a[e] += b[e];
  return pack<DT>(a);
}

template <int DT>
__device__ __forceinline__ void store_sum(unsigned char* row, int i0, int width, uint4 h) {
  constexpr int EPC = Fmt<DT>::EPC, ESZ = Fmt<DT>::ESZ;
  const uint32_t w[4] = {h.x, h.y, h.z, h.w};
  if (i0 + EPC <= width) {
    store_words<4>(row + (long long)i0 * ESZ, w);
  } else {
#pragma unroll
    for (int e = 0; e < EPC; ++e) {
      if (i0 + e >= width) continue;
      if constexpr (DT == 0)
        *reinterpret_cast<uint32_t*>(row + (long long)(i0 + e) * 4) = w[e];
      else
        *reinterpret_cast<uint16_t*>(row + (long long)(i0 + e) * 2) =
            (uint16_t)(w[e / 2] >> (16 * (e % 2)));
    }
  }
}

// Whole numbers of [-127, 127] as bytes, four to a word.
template <int EPC>
__device__ __forceinline__ void store_codes(int8_t* row, int i0, int width, const float* q) {
  uint32_t w[EPC / 4];
#pragma unroll
  for (int e = 0; e < EPC; e += 4) {
    uint32_t b = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)   // code + 128 as an unsigned byte
      b = __builtin_amdgcn_cvt_pk_u8_f32(q[e + k] + 128.0f, k, b);
    w[e / 4] = b ^ 0x80808080u;
  }
  if (i0 + EPC <= width) {
    store_words<EPC / 4>(row + i0, w);
  } else {
#pragma unroll
    for (int e = 0; e < EPC; ++e)
      if (i0 + e < width) row[i0 + e] = (int8_t)(w[e / 4] >> (8 * (e % 4)));
  }
}

__device__ __forceinline__ double wave_max_f64(double x) {
  return wave_reduce(x, [](double a, double b) { return fmax(a, b); });
}

template <bool ONCE>
__device__ __forceinline__ uint4 load_chunk(const unsigned char* p) {
  return ONCE ? load16_once(p) : load16(p);
}

// A float that the compiler does not know: what is formed of it is formed where it is
// used and not kept from an earlier use.
__device__ __forceinline__ float opaque(float x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Rows in registers, NC chunks a lane; WPR wavefronts to a row, four in a workgroup. ONCE:
// read past the caches.
template <int DT, int WT, int WPR, int NC, bool ONCE>
__global__ __launch_bounds__(kNormBlock) void norm_kernel(NormArgs a) {
  constexpr int EPC = Fmt<DT>::EPC, T = WPR * kWave, RPB = kNormBlock / T;
  constexpr bool SHORT = DT == 1 && WT == 1;   // 16 bits of a product: exact in float32
  static_assert(WPR == 1 || RPB == 1, "one wavefront to a row, or the workgroup");
  __shared__ uint32_t tops[WPR];
  __shared__ double sums[WPR], mosts[WPR];
  __shared__ unsigned long long exact_most;
  const int part = __builtin_amdgcn_readfirstlane(threadIdx.x / T);
  const int t = threadIdx.x % T, wave = threadIdx.x / kWave;
  const int whole = a.width / EPC;
  const bool partial = whole * EPC < a.width && t == whole % T;
  const long long r = (long long)blockIdx.x * RPB + part, at = min(r, (long long)a.rows - 1);
  const bool live = r < a.rows;
  const unsigned char* x = a.x + at * a.x_stride;
  uint4 c[NC], rest{};
#pragma unroll
  for (int j = 0; j < NC; ++j)
    c[j] = load_chunk<ONCE>(x + (long long)min(j * T + t, whole - 1) * 16);
  if (partial) rest = load_chunk_zero<DT>(x, (long long)whole * EPC, a.width);
  float w[NC][EPC], wr[EPC];
#pragma unroll
  for (int e = 0; e < EPC; ++e) wr[e] = 0.0f;
  if (a.residual) {
    const unsigned char* res = a.residual + at * a.r_stride;
    uint4 d[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j)
      d[j] = load_chunk<ONCE>(res + (long long)min(j * T + t, whole - 1) * 16);
#pragma unroll
    for (int j = 0; j < NC; ++j)
      load_weights<EPC, WT>(a.weight, min(j * T + t, whole - 1) * EPC, a.width, w[j]);
#pragma unroll
    for (int j = 0; j < NC; ++j) c[j] = add_chunks<DT>(c[j], d[j]);
    if (partial)
      rest = add_chunks<DT>(rest, load_chunk_zero<DT>(res, (long long)whole * EPC, a.width));
  } else {
#pragma unroll
    for (int j = 0; j < NC; ++j)
      load_weights<EPC, WT>(a.weight, min(j * T + t, whole - 1) * EPC, a.width, w[j]);
  }
  if (partial) load_weights<EPC, WT>(a.weight, whole * EPC, a.width, wr);
  // threads past the last whole chunk have none
#pragma unroll
  for (int j = 0; j < NC; ++j)
    if (j * T + t >= whole) c[j] = make_uint4(0, 0, 0, 0);
  if (WPR > 1 && threadIdx.x == 0) exact_most = 0;
  if (a.out_h && live) {
    unsigned char* out = a.out_h + r * a.h_stride;
#pragma unroll
    for (int j = 0; j < NC; ++j)
      if (j * T + t < whole) store_sum<DT>(out, (j * T + t) * EPC, a.width, c[j]);
    if (partial) store_sum<DT>(out, whole * EPC, a.width, rest);
  }
  // f(h, weights, first element) for each chunk; past the last whole one the width
  const auto each = [&](auto&& f) {
    const Pass pass;
    float h[EPC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      pass.unpack<DT>(c[j], h);
      f(h, w[j], j * T + t < whole ? (j * T + t) * EPC : a.width);
      sched_fence();
    }
    if (partial) {
      pass.unpack<DT>(rest, h);
      f(h, wr, whole * EPC);
    }
  };
  uint32_t top = 0;
  double ss = 0.0;
  each([&](const float* h, const float* v, int) {
#pragma unroll
    for (int e = 0; e < EPC; ++e) {
      top = max(top, __float_as_uint(h[e] * v[e]) & 0x7FFFFFFFu);
      ss = fma((double)h[e], (double)h[e], ss);
    }
  });
  const uint32_t own = top;
  top = wave_max_u32(top);
  ss = wave_sum(ss);
  if constexpr (WPR > 1) {
    if (__lane_id() == 0) {
      tops[wave] = top;
      sums[wave] = ss;
    }
    __syncthreads();
    ss = 0.0;
#pragma unroll
    for (int v = 0; v < WPR; ++v) {
      top = max(top, tops[v]);
      ss += sums[v];
    }
  }
  const float most = __uint_as_float(top);
  double m = most;
  bool fine = true;
  int8_t* q = a.codes + r * a.q_stride;
  if (top >= 0x0D800000u && top <= 0x71800000u) {   // 2^-100 .. 2^100
    if constexpr (!SHORT) {   // the largest exact one of the products that are `most`
      double mine = 0.0;
      if (own == top)
        each([&](const float* h, const float* v, int) {
#pragma unroll
          for (int e = 0; e < EPC; ++e) {
            const float y = opaque(h[e]), z = opaque(v[e]);
            if (fabsf(y * z) == most) mine = fmax(mine, fabs((double)y * (double)z));
          }
        });
      if constexpr (WPR > 1) {
        if (own == top)
          atomicMax(&exact_most, (unsigned long long)__double_as_longlong(mine));
        __syncthreads();
        m = __longlong_as_double((long long)exact_most);
      } else {
        m = wave_max_f64(mine);
      }
    }
    const float inv = 127.0f / most;
    each([&](const float* h, const float* v, int i0) {
      if (!live || i0 >= a.width) return;
      float code[EPC], far = 0.0f;
#pragma unroll
      for (int e = 0; e < EPC; ++e) {
        const float y = h[e] * v[e] * inv;
        code[e] = rintf(y);
        far = fmaxf(far, fabsf(y - code[e]));
      }
      if (far >= 0.5f - 0x1p-14f) {
#pragma unroll
        for (int e = 0; e < EPC; ++e) {
          const float y = opaque(h[e]), z = opaque(v[e]);
          const double d = fabs((double)y * (double)z);
          const float f = floorf(fabsf(y * z * inv));
          const float up = side_of(d, (double)f + 0.5, m, (int)f & 1) ? 1.0f : 0.0f;
          code[e] = copysignf(fminf(f + up, 127.0f), y * z);
        }
      }
      store_codes<EPC>(q, i0, a.width, code);
    });
  } else {   // zeros, numbers near the ends of float32, NaN, infinities
    double mine = 0.0;
    each([&](const float* h, const float* v, int) {
#pragma unroll
      for (int e = 0; e < EPC; ++e) {
        const float y = opaque(h[e]), z = opaque(v[e]);
        const double d = fabs((double)y * (double)z);
        fine = fine && d < __builtin_huge_val() && fabsf(y) < kPosInf;
        mine = fmax(mine, d);
      }
    });
    fine = !__any(!fine);
    m = wave_max_f64(fine ? mine : 0.0);
    if constexpr (WPR > 1) {
      if (__lane_id() == 0) mosts[wave] = fine ? m : -1.0;
      __syncthreads();
#pragma unroll
      for (int v = 0; v < WPR; ++v) {
        fine = fine && mosts[v] >= 0.0;
        m = fmax(m, mosts[v]);
      }
      __syncthreads();
    }
    each([&](const float* h, const float* v, int i0) {
      if (!live || i0 >= a.width) return;
      float code[EPC];
#pragma unroll
      for (int e = 0; e < EPC; ++e) {
        const double d = (double)opaque(h[e]) * (double)opaque(v[e]);
        code[e] = fine && m > 0.0 ? (float)exact_code(d, m) : 0.0f;
      }
      store_codes<EPC>(q, i0, a.width, code);
    });
  }
  if (t == 0 && live)
    a.scale[r] = !fine      ? __uint_as_float(0x7FC00000u)
                 : m == 0.0 ? 0.0f
                            : (float)(m / (127.0 * sqrt(ss / a.width + a.eps)));
}

// Rows of any width: read twice, an element at a time and with a quotient in 64 bits for each, one
// workgroup to a row. 4096 x 12288 fp32 119 us, 4096 x 20480 bf16 241 us, 1 x 20480 bf16 52 us;
// in registers 4096 x 8192 fp32 takes 33 us and 4096 x 16384 bf16 63 us.
template <int DT, int WT>
__global__ __launch_bounds__(kNormBlock) void norm_wide_kernel(NormArgs a) {
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
  m = __longlong_as_double((long long)block_max_u64<kNormBlock>(
      (unsigned long long)__double_as_longlong(m), scratch));
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

// Inputs of more bytes than this are read past the caches, which could not keep them: 16384 x
// 4096 bf16 with a residual 75 us against 84. Smaller ones may be there still: 4096 x 4096
// 23 us read from them, 26 past them.
constexpr long long kNormOnceBytes = 192ll << 20;

template <int DT, int WT, int WPR, int NC>
hipError_t launch_nc(const NormArgs& a, hipStream_t s) {
  constexpr int RPB = kNormBlock / (WPR * kWave);
  const auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((a.rows + RPB - 1) / RPB), dim3(kNormBlock), 0, s, a);
    return hipGetLastError();
  };
  const long long bytes = (long long)a.rows * a.width * Fmt<DT>::ESZ * (a.residual ? 2 : 1);
  return bytes > kNormOnceBytes ? launch(norm_kernel<DT, WT, WPR, NC, true>)
                                : launch(norm_kernel<DT, WT, WPR, NC, false>);
}

template <int DT, int WT>
hipError_t launch_wt(const NormArgs& a, hipStream_t s) {
  const int whole = a.width / Fmt<DT>::EPC;
  if (whole < 1 || whole > 8 * kNormBlock) {
    hipLaunchKernelGGL((norm_wide_kernel<DT, WT>), dim3(a.rows), dim3(kNormBlock), 0, s, a);
    return hipGetLastError();
  }
  // Up to 128 chunks one wavefront to a row, which then has no barrier: 32768 x 1024 bf16
  // 41 us, with four 54; 1 x 1024 2.9 us and 2.5. Wider rows need four for their registers.
  if (whole <= kWave) return launch_nc<DT, WT, 1, 1>(a, s);
  if (whole <= 2 * kWave) return launch_nc<DT, WT, 1, 2>(a, s);
  if (whole <= kNormBlock) return launch_nc<DT, WT, 4, 1>(a, s);
  if (whole <= 2 * kNormBlock) return launch_nc<DT, WT, 4, 2>(a, s);
  if (whole <= 4 * kNormBlock) return launch_nc<DT, WT, 4, 4>(a, s);
  return launch_nc<DT, WT, 4, 8>(a, s);
}

}  // namespace

hipError_t launch_norm_quantize(const NormArgs& a, int dtype, int weight_dtype, hipStream_t s) {
  if (dtype == 0)
    return weight_dtype == 0 ? launch_wt<0, 0>(a, s) : launch_wt<0, 1>(a, s);
  return weight_dtype == 0 ? launch_wt<1, 0>(a, s) : launch_wt<1, 1>(a, s);
}

}  // namespace tsr
