// Distillation of a draft model from a teacher's top tokens (distill_topk): the
// loss of each row of logits and its gradient.
//
//   q_i = exp(t_i) of the entries; plain: over their sum; with a tail: q_r is what
//   they leave of 1, the teacher's mass of all other ids together
//   L = sum_i q_i (log q_i - log p_i) + q_r (log q_r - log p_r), p_r = 1 - sum_S p
//   dL/dz_j = (Q p_j - q_j) / T in S, p_j (Q - q_r / p_r) / T outside, Q = sum q + q_r
//
// p_r is summed over the ids outside S themselves, and their weights are taken against
// their own largest: as 1 - sum_S p it would be lost where S holds nearly everything.
#include "kernels.hpp"
#include "scores.hpp"
#include "wide_mem.hpp"

namespace tsr {
namespace {

constexpr int kDtBlock = 256;
constexpr int kDtTile = 32768;        // ids whose membership in S one pass of LDS holds
constexpr float kRestMin = 0x1p-20f;  // a remainder below this is rounding of the entries

// The entries of a row, one to a lane of a wavefront.
struct Entries {
  int id;          // -1: none, or a lane past the last
  bool first;      // no lower lane holds the same id
  double q, log_q; // the teacher's probability
  double same;     // sum of q over the lanes of this id
  double sum, rest;
  int status;
};

__device__ __forceinline__ Entries load_entries(const DistillArgs& a, long long r) {
  Entries e;
  const int lane = __lane_id();
  const bool in = lane < a.k;
  e.id = in ? a.ids[r * a.k + lane] : -1;
  const float t = in ? a.teacher[r * a.k + lane] : kNegInf;
  const bool real = e.id != -1;
  e.status = 0;
  const bool outside = real && (e.id < 0 || e.id >= a.V);
  if (__ballot(outside)) e.status = 3;
  else if (__ballot(real && !(t < kPosInf))) e.status = 1;
  const float top = wave_max(real ? t : kNegInf);   // drops NaN: those rows are marked
  if (!e.status && top == kNegInf) e.status = 2;
  if (outside) e.id = -1;
  // with a tail the values are log probabilities; without one any row constant cancels
  const double shift = a.tail || e.status ? 0.0 : (double)top;
  e.q = real && t > kNegInf ? exp((double)t - shift) : 0.0;
  e.log_q = (double)t - shift;
  e.sum = wave_sum(e.q);
  e.rest = 0.0;
  if (a.tail) {
    e.rest = 1.0 - e.sum;
    if (!(e.rest > (double)kRestMin)) e.rest = 0.0;
  } else {
    e.q /= e.sum;
    e.log_q -= log(e.sum);
    e.sum = 1.0;
  }
  e.first = e.id >= 0;
  e.same = 0.0;
  for (int l = 0; l < a.k; ++l) {
    const int other = (int)readlane_u32((uint32_t)e.id, l);
    const double q = readlane_f64(e.q, l);
    if (other != e.id) continue;
    e.same += q;
    if (l < lane) e.first = false;
  }
  return e;
}

template <int DT>
__global__ __launch_bounds__(kDtBlock) void distill_kernel(DistillArgs a) {
  __shared__ BlockScratch scratch;
  __shared__ uint32_t in_s[kDtTile / 32];
  const long long r = blockIdx.x;
  const unsigned char* row = a.logits + r * a.stride_bytes;
  unsigned char* out = a.grad ? a.grad + r * a.grad_stride_bytes : nullptr;
  const float weight = a.weight ? a.weight[r] : 1.0f;
  if (weight == 0.0f) {   // the row does not count: neither its logits nor its entries do
    if (out)
      for (int i = threadIdx.x; i < a.V; i += kDtBlock) store_elem<DT>(out, i, 0.0f);
    if (threadIdx.x == 0) {
      a.loss[r] = 0.0f;
      if (a.status) a.status[r] = 0;
    }
    return;
  }
  const Entries e = load_entries(a, r);   // each wavefront for itself
  // with a tail the entries' ids are left out of the sums and come back one by one
  const auto bits = [&](int t0) {
    __syncthreads();
    for (int i = threadIdx.x; i < kDtTile / 32; i += kDtBlock) in_s[i] = 0;
    __syncthreads();
    if (a.tail && threadIdx.x < kWave && e.id >= t0 && e.id - t0 < kDtTile)
      atomicOr(&in_s[(e.id - t0) / 32], 1u << ((e.id - t0) % 32));
    __syncthreads();
  };
  const auto left_out = [&](int i) { return in_s[i / 32] >> (i % 32) & 1; };
  const float z = e.id >= 0 ? load_elem<DT>(row, e.id) : kNegInf;
  const float Ms = wave_maxn(a.tail ? z : kNegInf);
  float Mr = kNegInf;
  for (int t0 = 0; t0 < a.V; t0 += kDtTile) {
    bits(t0);
    for (int i = threadIdx.x; i < min(a.V - t0, kDtTile); i += kDtBlock)
      if (!left_out(i)) Mr = fmaxn(Mr, load_elem<DT>(row, t0 + i));
  }
  Mr = block_maxn<kDtBlock>(Mr, scratch);
  const float M = fmaxn(Mr, Ms);
  const int status = e.status ? e.status : M == kNegInf ? 2 : !(M < kPosInf) ? 1 : 0;
  if (Mr == kNegInf) Mr = 0.0f;   // any number: all their weights are 0
  double Zr = 0.0;
  for (int t0 = 0; t0 < a.V; t0 += kDtTile) {
    bits(t0);
    for (int i = threadIdx.x; i < min(a.V - t0, kDtTile); i += kDtBlock)
      if (!left_out(i))
        Zr += (double)__builtin_amdgcn_exp2f(exponent(load_elem<DT>(row, t0 + i), Mr, a.c));
  }
  Zr = block_sum<kDtBlock>(Zr, scratch);
  const double ez = e.id >= 0 ? exp(((double)z - (double)M) * a.inv_t) : 0.0;
  const double log_f = ((double)Mr - (double)M) * a.inv_t;
  const double f = Zr > 0.0 ? exp(log_f) : 0.0;   // what a weight against Mr is against M
  const double Z = Zr * f + wave_sum(a.tail && e.first ? ez : 0.0);
  double term = 0.0;
  if (e.q > 0.0) term = e.q * (e.log_q - (((double)z - (double)M) * a.inv_t - log(Z)));
  double loss = wave_sum(term);
  if (e.rest > 0.0) loss += e.rest * (log(e.rest) - (log(Zr) + log_f - log(Z)));
  const float nan = __uint_as_float(0x7FC00000u);
  if (threadIdx.x == 0) {
    a.loss[r] = status ? nan : (float)(loss * weight);
    if (a.status) a.status[r] = status;
  }
  if (!out) return;
  const double each = weight * a.inv_t;
  const double whole = e.sum + e.rest;
  const GradRow p(Mr, a.c,
                  status ? (double)nan : Zr > 0.0 ? each * (whole * f / Z - e.rest / Zr) : 0.0,
                  0.0);
  for (int i = threadIdx.x; i < a.V; i += kDtBlock)
    store_elem<DT>(out, i, p.at(load_elem<DT>(row, i)));
  __syncthreads();
  if (threadIdx.x < kWave && !status && e.first)
    store_elem<DT>(out, e.id, (float)(each * (whole * ez / Z - e.same)));
}

}  // namespace

size_t distill_ws_bytes(int, int, int, int) { return 0; }

hipError_t launch_distill(const DistillArgs& a, int dtype, void*, hipStream_t s) {
  if (dtype == 0)
    hipLaunchKernelGGL((distill_kernel<0>), dim3(a.rows), dim3(kDtBlock), 0, s, a);
  else
    hipLaunchKernelGGL((distill_kernel<1>), dim3(a.rows), dim3(kDtBlock), 0, s, a);
  return hipGetLastError();
}

}  // namespace tsr
