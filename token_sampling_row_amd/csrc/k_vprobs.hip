// Verification of drafted tokens from probabilities and given random numbers
// (verify_probs) [P2 39.4, eqs. 39.3-39.4; P3 "The Algorithm"].
#include "kernels.hpp"
#include "wide_mem.hpp"

namespace tsr {
namespace {

constexpr int kVpWaves = 16;
constexpr int kVpBlock = kVpWaves * kWave;
constexpr int kVpSteps = 1024;   // most steps a row is cut into

// What the K tests of one sequence decide.
struct VpCut {
  int status;    // TSR_ROW_*
  int kept;      // drafts kept
  int refused;   // whether draft `kept` was refused (else all were kept)
  int token;     // that draft's token
  int x;         // this lane's draft token
};

// The tests of sequence b, lane j < 32 taking draft j: kept iff u q(x) < p(x)
// (u < min(1, p / q) without the quotient; the product of two 24-bit factors
// is exact in 64 bits). Every wavefront that calls it gets the same answer.
template <int DT>
__device__ __forceinline__ VpCut vp_cut(const VprobsArgs& a, int b, int lane) {
  VpCut c{};
  const int len = a.lens ? a.lens[b] : a.K;
  const bool mine = lane < len && lane < a.K;
  c.x = mine ? a.tokens[(long long)b * a.K + lane] : 0;
  const bool out = mine && (c.x < 0 || c.x >= a.V);
  float p = 0.0f, q = 1.0f, u = 0.0f;
  if (mine && !out) {
    p = load_elem<DT>(a.target + b * a.t_seq + lane * a.t_row, c.x);
    if (a.draft) q = load_elem<DT>(a.draft + b * a.d_seq + lane * a.d_row, c.x);
    u = a.accept_u[(long long)b * a.K + lane];
  }
  const bool keep = mine && !out && (double)u * (double)q < (double)p;
  const unsigned long long refuse = __ballot(mine && !keep);
  const unsigned long long bad_x = __ballot(out);
  c.kept = refuse ? __ffsll((long long)refuse) - 1 : len;
  c.refused = refuse != 0;
  const bool seen = mine && lane <= c.kept;
  const unsigned long long bad_p =
      __ballot(seen && !(p >= 0.0f && p <= kFltMax && q >= 0.0f && q <= kFltMax));
  const float v = a.draw_u[b];
  const unsigned long long bad_u =
      __ballot((seen && !(u >= 0.0f && u < 1.0f)) || !(v >= 0.0f && v < 1.0f));
  c.token = (int)readlane_u32((uint32_t)c.x, c.kept & 31);
  c.status = (len < 0 || len > a.K) ? 4 : bad_x ? 3 : bad_p ? 1 : bad_u ? 4 : 0;
  return c;
}

// Weights of one chunk of the row that is drawn from, in 64 bits: the target's
// probabilities, less the draft's (SUB 1) or less the certain draft `x` (SUB
// 2). Returns their sum; NaN where a value read is no probability.
template <int DT, int SUB>
__device__ __forceinline__ double vp_weights(uint4 pr, uint4 qr, int e0, int x, double* w) {
  constexpr int EPC = Fmt<DT>::EPC;
  float p[EPC], q[EPC];
  unpack<DT>(pr, p);
  if constexpr (SUB == 1) unpack<DT>(qr, q);
  bool ok = true;
  double sum = 0.0;
#pragma unroll
  for (int e = 0; e < EPC; ++e) {
    ok = ok && p[e] >= 0.0f && p[e] <= kFltMax;
    double d = (double)p[e];
    if constexpr (SUB == 1) {
      ok = ok && q[e] >= 0.0f && q[e] <= kFltMax;
      d = fmax(d - (double)q[e], 0.0);
    }
    if constexpr (SUB == 2) d = e0 + e == x ? fmax(d - 1.0, 0.0) : d;
    w[e] = d;
    sum += d;
  }
  return ok ? sum : __builtin_nan("");
}

// Sums of the steps wave, wave + waves, ... of a row into `sums`; a step is
// `rep` times 64 chunks.
template <int DT, int SUB>
__device__ __forceinline__ void vp_sums(const unsigned char* prow, const unsigned char* qrow, int V,
                                        int x, int first, int stride, int steps, int rep,
                                        int lane, double* sums) {
  constexpr int EPC = Fmt<DT>::EPC;
  for (int s = first; s < steps; s += stride) {
    double sum = 0.0;
    for (int k = 0; k < rep; ++k) {
      const int e0 = ((s * rep + k) * kWave + lane) * EPC;
      const uint4 pr = load_chunk_zero<DT>(prow, e0, V);
      uint4 qr{};
      if constexpr (SUB == 1) qr = load_chunk_zero<DT>(qrow, e0, V);
      double w[EPC];
      sum += vp_weights<DT, SUB>(pr, qr, e0, x, w);
    }
    sum = wave_sum(sum);
    if (lane == 0) sums[s] = sum;
  }
}

// The step that holds aim = v * total: lane l holds steps 16 l .. 16 l + 15.
struct VpOwner {
  double total;
  int step;      // -1: the weights sum to nothing
  double base;   // total of the steps before it
};
__device__ __forceinline__ VpOwner vp_owner(const double* sums, int steps, float v, int lane) {
  constexpr int PER = kVpSteps / kWave;
  double mine = 0.0;
  for (int k = 0; k < PER; ++k) {
    const int s = lane * PER + k;
    if (s < steps) mine += sums[s];
  }
  const double incl = wave_incl_scan(mine);
  VpOwner o;
  o.total = readlane_f64(incl, kWave - 1);
  const double aim = (double)v * o.total;
  const unsigned long long over = __ballot(incl > aim);
  o.step = -1;
  o.base = 0.0;
  if (!over) return o;   // total 0 or NaN
  const int l = __ffsll((long long)over) - 1;
  double c = l > 0 ? readlane_f64(incl, l - 1) : 0.0;
  for (int k = 0; k < PER; ++k) {
    const int s = l * PER + k;
    if (s >= steps) break;
    const double w = sums[s];
    if (w > 0.0) {   // the last such step where rounding leaves none above aim
      o.step = s;
      o.base = c;
      if (c + w > aim) break;
    }
    c += w;
  }
  return o;
}

// The first id of the step whose running total exceeds aim; the last one with
// a weight where rounding leaves none.
template <int DT, int SUB>
__device__ __forceinline__ int vp_pick(const unsigned char* prow, const unsigned char* qrow, int V,
                                       int x, int step, int rep, double base, double aim,
                                       int lane) {
  constexpr int EPC = Fmt<DT>::EPC;
  int last = -1;
  for (int k = 0; k < rep; ++k) {
    const int e0 = ((step * rep + k) * kWave + lane) * EPC;
    const uint4 pr = load_chunk_zero<DT>(prow, e0, V);
    uint4 qr{};
    if constexpr (SUB == 1) qr = load_chunk_zero<DT>(qrow, e0, V);
    double w[EPC];
    const double sum = vp_weights<DT, SUB>(pr, qr, e0, x, w);
    const double incl = wave_incl_scan(sum);
    const double before = dpp_f64<kDppWaveShr1>(incl);   // lane 0: 0
    double c = base + before;
    int hit = -1, pos = -1;
#pragma unroll
    for (int e = 0; e < EPC; ++e) {
      c += w[e];
      if (w[e] > 0.0) {
        pos = e0 + e;
        if (hit < 0 && c > aim) hit = e0 + e;
      }
    }
    const unsigned long long hits = __ballot(hit >= 0);
    if (hits) return (int)readlane_u32((uint32_t)hit, __ffsll((long long)hits) - 1);
    last = max(last, wave_max(pos));
    base += readlane_f64(incl, kWave - 1);
  }
  return last;
}

// One workgroup per sequence.
template <int DT>
__global__ __launch_bounds__(kVpBlock) void vprobs_kernel(VprobsArgs a, int steps, int rep) {
  __shared__ double sums[kVpSteps];
  const int b = blockIdx.x, lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const VpCut c = vp_cut<DT>(a, b, lane);
  int status = c.status, token = -1;
  if (status == 0) {
    const unsigned char* prow = a.target + b * a.t_seq + c.kept * a.t_row;
    const unsigned char* qrow = a.draft ? a.draft + b * a.d_seq + c.kept * a.d_row : nullptr;
    const float v = a.draw_u[b];
    int sub = !c.refused ? 0 : a.draft ? 1 : 2;
    VpOwner o;
    for (;;) {
      if (sub == 0)
        vp_sums<DT, 0>(prow, qrow, a.V, c.token, wave, kVpWaves, steps, rep, lane, sums);
      else if (sub == 1)
        vp_sums<DT, 1>(prow, qrow, a.V, c.token, wave, kVpWaves, steps, rep, lane, sums);
      else
        vp_sums<DT, 2>(prow, qrow, a.V, c.token, wave, kVpWaves, steps, rep, lane, sums);
      __syncthreads();
      o = vp_owner(sums, steps, v, lane);
      if (sub == 0 || o.total != 0.0) break;
      sub = 0;           // nothing is left of the target: drawn from the target itself
      __syncthreads();   // every wavefront has read the sums
    }
    if (wave > 0) return;
    if (!(o.total >= 0.0)) {
      status = 1;
    } else if (o.step < 0) {
      status = 2;
    } else {
      const double aim = (double)v * o.total;
      token = sub == 0 ? vp_pick<DT, 0>(prow, qrow, a.V, c.token, o.step, rep, o.base, aim, lane)
              : sub == 1
                  ? vp_pick<DT, 1>(prow, qrow, a.V, c.token, o.step, rep, o.base, aim, lane)
                  : vp_pick<DT, 2>(prow, qrow, a.V, c.token, o.step, rep, o.base, aim, lane);
    }
  }
  if (wave > 0) return;
  if (lane <= a.K) {
    a.out_tokens[(long long)b * (a.K + 1) + lane] =
        status ? -1 : lane < c.kept ? c.x : lane == c.kept ? token : -1;
  }
  if (lane == 0) {
    a.out_accepted[b] = status ? 0 : c.kept;
    if (a.out_status) a.out_status[b] = status;
  }
}

template <int DT>
hipError_t launch_vprobs_dt(const VprobsArgs& a, hipStream_t s) {
  constexpr int SPAN = kWave * Fmt<DT>::EPC;
  const int spans = (a.V + SPAN - 1) / SPAN;
  const int rep = (spans + kVpSteps - 1) / kVpSteps;
  const int steps = (spans + rep - 1) / rep;
  hipLaunchKernelGGL((vprobs_kernel<DT>), dim3(a.rows), dim3(kVpBlock), 0, s, a, steps, rep);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_vprobs(const VprobsArgs& a, int dtype, hipStream_t s) {
  return dtype == 0 ? launch_vprobs_dt<0>(a, s) : launch_vprobs_dt<1>(a, s);
}

}  // namespace tsr
