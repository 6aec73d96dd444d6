// Log probabilities of given tokens, entropy and the likeliest alternatives of
// rows of logits (token_logprobs), and the gradient of the first two
// (token_logprobs_grad).
//
//   x_j = (z_j - M) / T, M = max z, Z = sum_j exp(x_j), log p_j = x_j - log Z
//   H = log Z - sum_j exp(x_j) x_j / Z   (both terms >= 0: nothing cancels)
//   dL/dz_j = (sum_i g_i [t_i = j] - p_j (sum_i g_i + gH (log p_j + H))) / T
#include "kernels.hpp"
#include "scores.hpp"
#include "wide_mem.hpp"

namespace tsr {
namespace {

constexpr int kLpBlock = 256;

// One workgroup to a row.
template <int DT>
__global__ __launch_bounds__(kLpBlock) void logprob_kernel(LogprobArgs a) {
  __shared__ BlockScratch scratch;
  const long long r = blockIdx.x;
  const unsigned char* row = a.logits + r * a.stride_bytes;
  float M = kNegInf;
  for (int i = threadIdx.x; i < a.V; i += kLpBlock) M = fmaxn(M, load_elem<DT>(row, i));
  M = block_maxn<kLpBlock>(M, scratch);
  const int status = M == kNegInf ? 2 : !(M < kPosInf) ? 1 : 0;
  double Z = 0.0, S = 0.0;
  if (!status) {
    for (int i = threadIdx.x; i < a.V; i += kLpBlock) {
      const float x = exponent(load_elem<DT>(row, i), M, a.c);
      const float e = __builtin_amdgcn_exp2f(x);
      Z += (double)e;
      S += (double)(e * x);
    }
    Z = block_sum<kLpBlock>(Z, scratch);
    S = block_sum<kLpBlock>(S, scratch);
  }
  int bad_token = 0;
  const float nan = __uint_as_float(0x7FC00000u);
  for (int i = threadIdx.x; i < a.n; i += kLpBlock) {
    const int t = a.tokens[r * a.n + i];
    float lp = 0.0f;
    if (t != -1) {
      const bool in = t >= 0 && t < a.V;
      bad_token |= !in;
      lp = in && !status ? log_prob(load_elem<DT>(row, t), M, Z, a.inv_t) : nan;
    }
    if (a.logprob) a.logprob[r * a.n + i] = lp;
  }
  bad_token = block_max<kLpBlock>(bad_token, scratch);
  if (threadIdx.x == 0) {
    if (a.entropy) a.entropy[r] = status ? nan : (float)((log(Z) - S / Z * kLn2));
    if (a.norm) {
      a.norm[2 * r] = status ? nan : M;
      a.norm[2 * r + 1] = status ? nan : (float)Z;
    }
    if (a.status) a.status[r] = status ? status : bad_token ? 3 : 0;
  }
  // the largest key below the last one, k times over
  unsigned long long last = ~0ull;
  for (int j = 0; j < a.k; ++j) {
    unsigned long long best = 0;
    if (!status && last) {
      for (int i = threadIdx.x; i < a.V; i += kLpBlock) {
        const float v = load_elem<DT>(row, i);
        const unsigned long long key = top_key(v, i);
        if (v > kNegInf && key < last && key > best) best = key;
      }
      best = block_max_u64<kLpBlock>(best, scratch);
    }
    last = best;
    if (threadIdx.x == 0) {
      const long long at = r * a.k + j;
      if (a.top_ids) a.top_ids[at] = best ? top_id(best) : -1;
      if (a.top_logprob)
        a.top_logprob[at] = best ? log_prob(top_value(best), M, Z, a.inv_t)
                                 : status ? nan : kNegInf;
    }
  }
}

template <int DT>
__global__ __launch_bounds__(kLpBlock) void logprob_grad_kernel(LogprobGradArgs a) {
  __shared__ BlockScratch scratch;
  const long long r = blockIdx.x;
  const unsigned char* row = a.logits + r * a.stride_bytes;
  unsigned char* out = a.out + r * a.out_stride_bytes;
  double G = 0.0;
  int any = 0;
  for (int i = threadIdx.x; i < a.n; i += kLpBlock) {
    const int t = a.tokens[r * a.n + i];
    if (t == -1) continue;
    const float g = a.g[r * a.n + i];
    any |= g != 0.0f;
    G += t >= 0 && t < a.V ? (double)g : __longlong_as_double(0x7FF8000000000000ll);
  }
  G = block_sum<kLpBlock>(G, scratch);
  const float ge = a.ge ? a.ge[r] : 0.0f;
  any = block_max<kLpBlock>(any, scratch) || ge != 0.0f || G != 0.0;
  if (!any) {   // nothing comes back to this row: its logits are not looked at
    for (int i = threadIdx.x; i < a.V; i += kLpBlock) store_elem<DT>(out, i, 0.0f);
    return;
  }
  GradRow p;
  p.M = a.norm[2 * r];
  const float Z = a.norm[2 * r + 1];
  p.c = a.c;
  p.A = -(float)G * a.inv_t / Z;
  p.B = 0.0f;
  if (ge != 0.0f) {
    const float H = a.entropy[r];
    p.A = (float)(-(G + (double)ge * ((double)H - log((double)Z))) * a.inv_t / Z);
    p.B = -ge * a.inv_t / Z * (float)kLn2;
  }
  for (int i = threadIdx.x; i < a.V; i += kLpBlock)
    store_elem<DT>(out, i, p.at(load_elem<DT>(row, i)));
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += kLpBlock) {
    const int t = a.tokens[r * a.n + i];
    if (t < 0 || t >= a.V) continue;
    float g = 0.0f;
    bool first = true;
    for (int k = 0; k < a.n; ++k) {
      if (a.tokens[r * a.n + k] != t) continue;
      if (k < i) first = false;
      g += a.g[r * a.n + k];
    }
    if (first) store_elem<DT>(out, t, fmaf(g, a.inv_t, p.at(load_elem<DT>(row, t))));
  }
}

}  // namespace

size_t logprobs_ws_bytes(int, int, int, int) { return 0; }

hipError_t launch_logprobs(const LogprobArgs& a, int dtype, void*, hipStream_t s) {
  if (dtype == 0)
    hipLaunchKernelGGL((logprob_kernel<0>), dim3(a.rows), dim3(kLpBlock), 0, s, a);
  else
    hipLaunchKernelGGL((logprob_kernel<1>), dim3(a.rows), dim3(kLpBlock), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_logprobs_grad(const LogprobGradArgs& a, int dtype, hipStream_t s) {
  if (dtype == 0)
    hipLaunchKernelGGL((logprob_grad_kernel<0>), dim3(a.rows), dim3(kLpBlock), 0, s, a);
  else
    hipLaunchKernelGGL((logprob_grad_kernel<1>), dim3(a.rows), dim3(kLpBlock), 0, s, a);
  return hipGetLastError();
}

}  // namespace tsr
