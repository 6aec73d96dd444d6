// Verification of drafted tokens from probabilities and given random numbers
// (verify_probs) [P2 39.4, eqs. 39.3-39.4; P3 "The Algorithm"].
//
// Draft j is kept iff u q(x) < p(x); the row after the kept ones gives weights
// w = max(0, p - q) or p, and the token is the first whose running total exceeds
// v sum w. Only that row (and its draft's) is read, once for the sums of groups
// of spans, and one group of it again for the draw.
//
// Few rows are bound by three trips to memory, each waiting for the last (draft
// tokens, their probabilities, the row), and the draw's fourth: 1 x 32000 fp32
// 7.0 us, 64 x 32000 9.6 (12 MB). Many are bound by the rows' bytes: 128 x 128256
// fp32 19.6 us for the sums (92 MB, 4.7 TB/s) and 4.9 for the draw.
#include "kernels.hpp"
#include "wide_mem.hpp"

namespace tsr {
namespace {

// Wavefronts of the one-launch kernel: sixteen where a span's registers allow.
template <int DT> constexpr int kVpWaves = DT == 0 ? 16 : 8;
constexpr int kVpSliceWaves = 4;
constexpr int kVpSliceBlock = kVpSliceWaves * kWave;
// Batches of more bytes of target rows than this are read past the caches:
// 256 x 128256 fp32 39 us against 44, but 64 x 32000, which stays in them between
// the model and this call, 12 us against 10.
constexpr long long kVpOnceBytes = 48ll << 20;
constexpr int kVpGroup = 4;   // spans of a group; a wavefront has two groups' loads on their way
constexpr int kVpAlone = 32;  // groups that one workgroup sums as fast as several
template <int DT> constexpr int kVpUnit = kWave * Fmt<DT>::EPC * kVpGroup;   // ids of a group

// How many workgroups share a row's sums (1: the one-launch kernel, as fast up
// to 32 groups: 64 x 32000 fp32 9.6 us). A wavefront takes two groups at a time,
// or one where that leaves places empty (33 x 151935 bf16 11.4 us against 11.9,
// but 64 x 128256 bf16 15.7 against 14.5); 256 x 128256 fp32 with eight
// workgroups to a row 37 us, with four 39.
int vp_slices(int rows, int groups) {
  if (rows > kVpWsRows || groups <= kVpAlone) return 1;
  const int one = (groups + kVpSliceWaves - 1) / kVpSliceWaves;
  const int most = rows * one <= 768 ? one : (one + 1) / 2;
  const int want = (2048 + rows - 1) / rows;
  return want < most ? want : most;
}

// What the K tests of one sequence decide.
struct VpCut {
  int status;    // TSR_ROW_*
  int kept;      // drafts kept
  int refused;   // whether draft `kept` was refused (else all were kept)
  int token;     // that draft's token
  int x;         // this lane's draft token
  float v;       // the uniform of the draw
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
  const float u = mine ? a.accept_u[(long long)b * a.K + lane] : 0.0f;
  c.v = a.draw_u[b];
  float p = 0.0f, q = 1.0f;
  if (mine && !out) {
    p = load_elem<DT>(a.target + b * a.t_seq + lane * a.t_row, c.x);
    if (a.draft) q = load_elem<DT>(a.draft + b * a.d_seq + lane * a.d_row, c.x);
  }
  const bool keep = mine && !out && (double)u * (double)q < (double)p;
  const unsigned long long refuse = __ballot(mine && !keep);
  const unsigned long long bad_x = __ballot(out);
  c.kept = refuse ? __ffsll((long long)refuse) - 1 : len;
  c.refused = refuse != 0;
  const bool seen = mine && lane <= c.kept;
  const unsigned long long bad_p =
      __ballot(seen && !(p >= 0.0f && p <= kFltMax && q >= 0.0f && q <= kFltMax));
  const unsigned long long bad_u =
      __ballot((seen && !(u >= 0.0f && u < 1.0f)) || !(c.v >= 0.0f && c.v < 1.0f));
  c.token = (int)readlane_u32((uint32_t)c.x, c.kept & 31);
  c.status = (len < 0 || len > a.K) ? 4 : bad_x ? 3 : bad_p ? 1 : bad_u ? 4 : 0;
  return c;
}

// The row that is drawn from, cut into spans of 64 chunks (one a lane) and
// groups of kVpGroup x rep spans.
struct VpRow {
  const unsigned char* p;   // the target's row
  const unsigned char* q;   // the draft's, where it is taken off (SUB 1)
  int V;
  int x;                    // the token whose certain draft is taken off (SUB 2)
  int rep, groups;
  bool once;                // the rows of the batch outgrow the caches
};
template <int DT>
__device__ __forceinline__ VpRow vp_row(const VprobsArgs& a, int b, int kept, int x, int rep,
                                        int groups) {
  return VpRow{a.target + b * a.t_seq + kept * a.t_row,
               a.draft ? a.draft + b * a.d_seq + kept * a.d_row : nullptr, a.V, x, rep, groups,
               (long long)a.rows * a.V * Fmt<DT>::ESZ >= kVpOnceBytes};
}

// Weights of one chunk in 64 bits: the target's probabilities, less the draft's
// (SUB 1) or less the certain draft x (SUB 2). Returns their sum; NaN where a
// value read is no probability. The bits of a float in [0, largest] are at
// most 0x7F7FFFFF as an integer; a larger maximum is looked at again (it may be
// a negative zero).
template <int DT, int SUB>
__device__ __forceinline__ double vp_weights(uint4 pr, uint4 qr, int e0, int x, double* w) {
  constexpr int EPC = Fmt<DT>::EPC;
  float p[EPC], q[EPC];
  unpack<DT>(pr, p);
  if constexpr (SUB == 1) unpack<DT>(qr, q);
  uint32_t top = 0;
  double sum = 0.0;
#pragma unroll
  for (int e = 0; e < EPC; ++e) {
    top = max(top, __float_as_uint(p[e]));
    double d = (double)p[e];
    if constexpr (SUB == 1) {
      top = max(top, __float_as_uint(q[e]));
      d = fmax(d - (double)q[e], 0.0);
    }
    if constexpr (SUB == 2) d = e0 + e == x ? fmax(d - 1.0, 0.0) : d;
    w[e] = d;
    sum += d;
  }
  if (top > 0x7F7FFFFFu) {
#pragma unroll
    for (int e = 0; e < EPC; ++e) {
      const bool ok = p[e] >= 0.0f && p[e] <= kFltMax &&
                      (SUB != 1 || (q[e] >= 0.0f && q[e] <= kFltMax));
      if (!ok) sum = __builtin_nan("");
    }
  }
  return sum;
}

// kVpGroup spans from span s0 on: the chunks this lane has of them. All loads
// are on their way together; spans past the row's whole ones load the last of
// those again, and are then replaced by the partial one, loaded by itself, or by
// zeros.
template <int DT, int SUB>
struct VpGroup {
  uint4 p[kVpGroup], q[SUB == 1 ? kVpGroup : 1];
  __device__ __forceinline__ void load(const VpRow& r, int s0, int lane) {
    constexpr int EPC = Fmt<DT>::EPC, ESZ = Fmt<DT>::ESZ, SPAN = kWave * EPC;
    const int whole = r.V / SPAN;
    if (whole > 0 && r.once) {
#pragma unroll
      for (int i = 0; i < kVpGroup; ++i) {
        const long long at = (long long)min(s0 + i, whole - 1) * (SPAN * ESZ);
        p[i] = load16_once(r.p + at + lane * 16);
        if constexpr (SUB == 1) q[i] = load16_once(r.q + at + lane * 16);
      }
    } else if (whole > 0) {
#pragma unroll
      for (int i = 0; i < kVpGroup; ++i) {
        const long long at = (long long)min(s0 + i, whole - 1) * (SPAN * ESZ);
        p[i] = load16(r.p + at + lane * 16);
        if constexpr (SUB == 1) q[i] = load16(r.q + at + lane * 16);
      }
    }
    if (s0 + kVpGroup > whole) {   // the partial span, and nothing past it
      uint4 pe = make_uint4(0, 0, 0, 0), qe = pe;
      if (s0 <= whole) {
        pe = load_chunk_zero<DT>(r.p, whole * SPAN + lane * EPC, r.V);
        if constexpr (SUB == 1) qe = load_chunk_zero<DT>(r.q, whole * SPAN + lane * EPC, r.V);
      }
#pragma unroll
      for (int i = 0; i < kVpGroup; ++i) {
        if (s0 + i < whole) continue;
        const uint32_t keep = s0 + i == whole ? 0xFFFFFFFFu : 0u;
        p[i] = make_uint4(pe.x & keep, pe.y & keep, pe.z & keep, pe.w & keep);
        if constexpr (SUB == 1)
          q[i] = make_uint4(qe.x & keep, qe.y & keep, qe.z & keep, qe.w & keep);
      }
    }
  }
  __device__ __forceinline__ double weights(const VpRow& r, int s0, int i, int lane,
                                            double* w) const {
    constexpr int EPC = Fmt<DT>::EPC;
    return vp_weights<DT, SUB>(p[i], q[SUB == 1 ? i : 0], ((s0 + i) * kWave + lane) * EPC, r.x, w);
  }
};

// Sums of the groups first, first + stride, ... below `end` into `sums`.
template <int DT, int SUB>
__device__ __forceinline__ void vp_sums(const VpRow& r, int first, int stride, int end, int lane,
                                        double* sums) {
  for (int g = first; g < end; g += 2 * stride) {
    const bool two = g + stride < end;
    double sum[2] = {0.0, 0.0};
    for (int k = 0; k < r.rep; ++k) {
      const int s0 = (g * r.rep + k) * kVpGroup;
      const int s1 = ((g + stride) * r.rep + k) * kVpGroup;
      VpGroup<DT, SUB> v0, v1;
      v0.load(r, s0, lane);
      if (two) v1.load(r, s1, lane);
      double w[Fmt<DT>::EPC];
#pragma unroll
      for (int i = 0; i < kVpGroup; ++i) {
        sum[0] += v0.weights(r, s0, i, lane, w);
        sched_fence();   // one span's doubles at a time
      }
      if (two) {
#pragma unroll
        for (int i = 0; i < kVpGroup; ++i) {
          sum[1] += v1.weights(r, s1, i, lane, w);
          sched_fence();
        }
      }
    }
    const double a = wave_sum(sum[0]), b = wave_sum(sum[1]);
    if (lane == 0) {
      sums[g] = a;
      if (two) sums[g + stride] = b;
    }
  }
}
template <int DT>
__device__ __forceinline__ void vp_sums_of(const VpRow& r, int sub, int first, int stride, int end,
                                           int lane, double* sums) {
  if (sub == 0)
    vp_sums<DT, 0>(r, first, stride, end, lane, sums);
  else if (sub == 1)
    vp_sums<DT, 1>(r, first, stride, end, lane, sums);
  else
    vp_sums<DT, 2>(r, first, stride, end, lane, sums);
}

// The group that holds aim = v * total: lane l looks at `per` neighbouring ones.
struct VpOwner {
  double total;
  int group;     // -1: the weights sum to nothing, or not to a number
  double base;   // total of the groups before it
};
__device__ __forceinline__ VpOwner vp_owner(const double* sums, int groups, float v, int lane) {
  const int per = (groups + kWave - 1) / kWave;
  double mine = 0.0;
  for (int k = 0; k < per; ++k) {
    const int g = lane * per + k;
    if (g < groups) mine += sums[g];
  }
  const double incl = wave_incl_scan(mine);
  VpOwner o;
  o.total = readlane_f64(incl, kWave - 1);
  const double aim = (double)v * o.total;
  // the totals of different lanes are added in different orders, so one may pass
  // aim at a lane that adds nothing: only lanes with a weight are looked at
  const unsigned long long any = __ballot(mine > 0.0);
  const unsigned long long over = __ballot(mine > 0.0 && incl > aim);
  o.group = -1;
  o.base = 0.0;
  if (!any) return o;   // total 0 or NaN
  const int l = over ? __ffsll((long long)over) - 1 : 63 - __clzll((long long)any);
  double c = l > 0 ? readlane_f64(incl, l - 1) : 0.0;
  for (int k = 0; k < per; ++k) {
    const int g = l * per + k;
    if (g >= groups) break;
    const double w = sums[g];
    if (w > 0.0) {   // the last such group where rounding leaves none above aim
      o.group = g;
      o.base = c;
      if (c + w > aim) break;
    }
    c += w;
  }
  o.group = __builtin_amdgcn_readfirstlane(o.group);
  o.base = readlane_f64(o.base, 0);
  return o;
}

// The first id of the group whose running total exceeds aim; the last one with
// a weight where rounding leaves none.
template <int DT, int SUB>
__device__ __forceinline__ int vp_pick(const VpRow& r, const VpOwner& o, double aim, int lane) {
  constexpr int EPC = Fmt<DT>::EPC;
  double base = o.base;
  int found = -1;   // last id with a weight so far
  for (int k = 0; k < r.rep; ++k) {
    const int s0 = (o.group * r.rep + k) * kVpGroup;
    VpGroup<DT, SUB> v;
    v.load(r, s0, lane);
    // the first span that passes aim, else the last with a weight
    int span = -1;
    double before = base;
    uint4 pr{}, qr{};
#pragma unroll
    for (int i = 0; i < kVpGroup; ++i) {
      double w[EPC];
      const double sum = wave_sum(v.weights(r, s0, i, lane, w));
      const bool done = span >= 0 && base > aim;   // an earlier span passed it
      if (sum > 0.0 && !done) {
        span = s0 + i;
        before = base;
        pr = v.p[i];
        qr = v.q[SUB == 1 ? i : 0];
      }
      base = done ? base : base + sum;
      sched_fence();
    }
    if (span < 0) continue;
    const int e0 = (span * kWave + lane) * EPC;
    double w[EPC];
    const double sum = vp_weights<DT, SUB>(pr, qr, e0, r.x, w);
    const double incl = wave_incl_scan(sum);
    double c = before + dpp_f64<kDppWaveShr1>(incl);   // lane 0: nothing before it
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
    found = max(found, wave_max(pos));
    if (base > aim) break;   // by the spans' sums it was here
  }
  return found;
}

// The draw once the group sums are known (one wavefront). Returns the token,
// or -1 with a status.
template <int DT>
__device__ __forceinline__ int vp_draw(const VpRow& r, int sub, const VpOwner& o, float v, int lane,
                                       int* status) {
  if (!(o.total >= 0.0)) {
    *status = 1;
    return -1;
  }
  if (o.group < 0) {
    *status = 2;
    return -1;
  }
  const double aim = (double)v * o.total;
  return sub == 0   ? vp_pick<DT, 0>(r, o, aim, lane)
         : sub == 1 ? vp_pick<DT, 1>(r, o, aim, lane)
                    : vp_pick<DT, 2>(r, o, aim, lane);
}

__device__ __forceinline__ void vp_write(const VprobsArgs& a, int b, int status, int kept, int x,
                                         int token, int lane) {
  if (lane <= a.K)
    a.out_tokens[(long long)b * (a.K + 1) + lane] =
        status ? -1 : lane < kept ? x : lane == kept ? token : -1;
  if (lane == 0) {
    a.out_accepted[b] = status ? 0 : kept;
    if (a.out_status) a.out_status[b] = status;
  }
}

// One workgroup per sequence: tests, group sums in LDS, draw. Every wavefront
// makes the tests and finds the group for itself, so that only the sums wait for
// each other; 16 wavefronts keep a 128 KB row on its way at once.
template <int DT>
__global__ __launch_bounds__(kVpWaves<DT>* kWave) void vprobs_kernel(VprobsArgs a, int groups,
                                                                     int rep) {
  __shared__ double sums[kVpGroups];
  const int b = blockIdx.x, lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const VpCut c = vp_cut<DT>(a, b, lane);
  int status = c.status, token = -1;
  if (status == 0) {
    const VpRow r = vp_row<DT>(a, b, c.kept, c.token, rep, groups);
    int sub = !c.refused ? 0 : a.draft ? 1 : 2;
    VpOwner o;
    for (;;) {
      vp_sums_of<DT>(r, sub, wave, kVpWaves<DT>, groups, lane, sums);
      __syncthreads();
      o = vp_owner(sums, groups, c.v, lane);
      if (sub == 0 || o.total != 0.0) break;
      sub = 0;           // nothing is left of the target: drawn from the target itself
      __syncthreads();   // every wavefront has read the sums
    }
    if (wave > 0) return;
    token = vp_draw<DT>(r, sub, o, c.v, lane, &status);
  }
  if (wave > 0) return;
  vp_write(a, b, status, c.kept, c.x, token, lane);
}

// The same in two launches, for rows of many ids: `slices` workgroups to a
// sequence write group sums, then one workgroup draws. Each slice makes the
// tests for itself (two dependent loads); the first leaves what they decided
// for the draw. 33 x 151935 bf16: 6.8 us and 4.9, the second a launch, the sums'
// trip to memory and one group's.
template <int DT>
__global__ __launch_bounds__(kVpSliceBlock) void vprobs_slices_kernel(VprobsArgs a, int groups,
                                                                      int rep, int slices,
                                                                      VprobsWs ws) {
  const int b = blockIdx.y, slice = blockIdx.x, lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const VpCut c = vp_cut<DT>(a, b, lane);
  if (slice == 0 && threadIdx.x == 0)
    ws.cut[b] = make_int4(c.status, c.kept, c.refused, c.token);
  if (c.status != 0) return;
  const VpRow r = vp_row<DT>(a, b, c.kept, c.token, rep, groups);
  vp_sums_of<DT>(r, !c.refused ? 0 : a.draft ? 1 : 2, slice * kVpSliceWaves + wave,
                 slices * kVpSliceWaves, groups, lane, ws.sums + (long long)b * groups);
}

template <int DT>
__global__ __launch_bounds__(kVpSliceBlock) void vprobs_draw_kernel(VprobsArgs a, int groups,
                                                                    int rep, VprobsWs ws) {
  __shared__ double sums[kVpGroups];
  const int b = blockIdx.x, lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int4 cut = ws.cut[b];
  int status = cut.x, token = -1;
  const int x = lane < a.K ? a.tokens[(long long)b * a.K + lane] : 0;
  const float v = a.draw_u[b];
  for (int g = threadIdx.x; g < groups; g += kVpSliceBlock)
    sums[g] = ws.sums[(long long)b * groups + g];
  __syncthreads();
  if (status == 0) {
    const VpRow r = vp_row<DT>(a, b, cut.y, cut.w, rep, groups);
    int sub = !cut.z ? 0 : a.draft ? 1 : 2;
    VpOwner o = vp_owner(sums, groups, v, lane);
    if (sub != 0 && o.total == 0.0) {   // nothing is left of the target
      sub = 0;
      __syncthreads();
      vp_sums_of<DT>(r, 0, wave, kVpSliceWaves, groups, lane, sums);
      __syncthreads();
      o = vp_owner(sums, groups, v, lane);
    }
    if (wave > 0) return;
    token = vp_draw<DT>(r, sub, o, v, lane, &status);
  }
  if (wave > 0) return;
  vp_write(a, b, status, cut.y, x, token, lane);
}

// How a batch is cut.
struct VpPlan {
  int rep, groups, slices;
};
template <int DT>
VpPlan vp_plan(int rows, int vocab) {
  const int units = (vocab - 1) / kVpUnit<DT> + 1;
  VpPlan p;
  p.rep = (units + kVpGroups - 1) / kVpGroups;
  p.groups = (units + p.rep - 1) / p.rep;
  p.slices = vp_slices(rows, p.groups);
  return p;
}
size_t vp_bytes(int rows, int groups) {
  return (size_t)rows * (sizeof(int4) + (size_t)groups * sizeof(double));
}

template <int DT>
hipError_t launch_vprobs_dt(const VprobsArgs& a, void* block, hipStream_t s) {
  const VpPlan p = vp_plan<DT>(a.rows, a.V);
  if (p.slices > 1) {
    int4* cut = static_cast<int4*>(block);
    const VprobsWs ws{cut, reinterpret_cast<double*>(cut + a.rows)};
    hipLaunchKernelGGL((vprobs_slices_kernel<DT>), dim3(p.slices, a.rows), dim3(kVpSliceBlock), 0,
                       s, a, p.groups, p.rep, p.slices, ws);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((vprobs_draw_kernel<DT>), dim3(a.rows), dim3(kVpSliceBlock), 0, s, a,
                       p.groups, p.rep, ws);
  } else {
    hipLaunchKernelGGL((vprobs_kernel<DT>), dim3(a.rows), dim3(kVpWaves<DT> * kWave), 0, s, a,
                       p.groups, p.rep);
  }
  return hipGetLastError();
}

}  // namespace

size_t vprobs_ws_bytes(int dtype, int rows, int vocab) {
  const VpPlan p = dtype == 0 ? vp_plan<0>(rows, vocab) : vp_plan<1>(rows, vocab);
  return p.slices > 1 ? vp_bytes(rows, p.groups) : 0;
}

size_t vprobs_ws_most(int rows, int vocab) {
  // float32 rows have the most groups; fewer ids have no more of them
  const int groups = min((vocab - 1) / kVpUnit<0> + 1, kVpGroups);
  return groups <= kVpAlone ? 0 : vp_bytes(min(rows, kVpWsRows), groups);
}

hipError_t launch_vprobs(const VprobsArgs& a, int dtype, void* ws, hipStream_t s) {
  return dtype == 0 ? launch_vprobs_dt<0>(a, ws, s) : launch_vprobs_dt<1>(a, ws, s);
}

}  // namespace tsr
