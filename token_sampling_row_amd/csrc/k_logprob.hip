// Log probabilities of given tokens, entropy and the likeliest alternatives of
// rows of logits (token_logprobs), and the gradient of the first two
// (token_logprobs_grad).
//
//   x_j = (z_j - M) / T, M = max z, Z = sum_j exp(x_j), log p_j = x_j - log Z
//   H = log Z - sum_j exp(x_j) x_j / Z   (both terms >= 0: nothing cancels)
//   dL/dz_j = (sum_i g_i [t_i = j] - p_j (sum_i g_i + gH (log p_j + H))) / T
#include <algorithm>
#include <type_traits>

#include "grad_tile.hpp"

namespace tsr {
namespace {

constexpr int kLpBlock = 256;

// ------------------------------------------------------------ the likeliest ids
// Keys of ids that may be among the k largest, in a region of LDS for each wavefront.
template <int REGION>
struct Candidates {
  unsigned long long key[kSliceWaves][REGION];
  int n[kSliceWaves];
};
constexpr int kSliceRegion = 128;   // keys of a wavefront in a slice
constexpr int kJoinRegion = 512;    // and of one that joins slices

// put(rank, key) for each candidate that fewer than k exceed. Keys differ, so ranks do.
template <int REGION, class F>
__device__ __forceinline__ void rank_candidates(const Candidates<REGION>& c, int k, F&& put) {
  int n[kSliceWaves], total = 0;
#pragma unroll
  for (int w = 0; w < kSliceWaves; ++w) total += n[w] = c.n[w];
  for (int i = threadIdx.x; i < total; i += kSliceBlock) {
    int w = 0, at = i;
    while (at >= n[w]) at -= n[w++];
    const unsigned long long mine = c.key[w][at];
    int rank = 0;
#pragma unroll
    for (int v = 0; v < kSliceWaves; ++v)
#pragma unroll 4
      for (int q = 0; q < n[v]; ++q) rank += c.key[v][q] > mine;
    if (rank < k) put(rank, mine);
  }
}

// Chunks of a slice that hold candidates, a region for each wavefront.
constexpr int kHits = 64;
template <int DT>
struct Hits {
  uint4 chunk[kSliceWaves][kHits];
  int id[kSliceWaves][kHits];   // of the chunk's first element
  int n[kSliceWaves];
};

// The slice's candidates: its logits of at least `tau` (a key of values), of which there
// are k at least and few more: every wavefront has j = ceil(k / 4) threads whose largest
// logit is at least that. `cmax`: the largest of each chunk. A wavefront lists its chunks
// that hold any, and the workgroup then looks at their elements together: taken where
// they lie, each chunk would cost its wavefront eight tests for one or two that pass.
template <int DT, int NC>
__device__ __forceinline__ void gather(const Slice<DT, NC>& s, int V, const float* cmax,
                                       uint32_t tau, int k, Candidates<kSliceRegion>& c,
                                       Hits<DT>& hits, BlockScratch& scratch) {
  constexpr int EPC = Fmt<DT>::EPC;
  const int wave = threadIdx.x / kWave;
  const float least = key2f(tau);
  int n = 0;
  const auto list = [&](float most, uint4 chunk, int id) {
    const bool in = most >= least && most > kNegInf;
    const unsigned long long who = __ballot(in);
    if (who == 0) return;
    const int at = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32),
                                                 __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
    if (in && at < kHits) {
      hits.chunk[wave][at] = chunk;
      hits.id[wave][at] = id;
    }
    n += __popcll(who);
  };
#pragma unroll
  for (int j = 0; j < NC; ++j) list(cmax[j], s.c[j], s.chunk_id(j) * EPC);
  if (s.ragged) list(cmax[NC], s.rest, V / EPC * EPC);
  if (__lane_id() == 0) hits.n[wave] = n;
  __syncthreads();
  int count[kSliceWaves], total = 0, most = 0;
#pragma unroll
  for (int w = 0; w < kSliceWaves; ++w) {
    total += count[w] = hits.n[w];
    most = max(most, count[w]);
  }
  n = 0;
  if (most <= kHits) {
    for (int i0 = wave * kWave; i0 < total * EPC; i0 += kSliceBlock) {
      const int i = i0 + (int)__lane_id();
      int at = i / EPC, w = 0;
      const int e = i % EPC;
      while (w < kSliceWaves - 1 && at >= count[w]) at -= count[w++];
      bool in = i < total * EPC;
      float v = kNegInf;
      if (in) {
        if constexpr (DT == 0)
          v = reinterpret_cast<const float*>(&hits.chunk[w][at])[e];
        else
          v = __uint_as_float(
              (uint32_t) reinterpret_cast<const uint16_t*>(&hits.chunk[w][at])[e] << 16);
      }
      in = v >= least && v > kNegInf;
      const unsigned long long who = __ballot(in);
      const int to = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32),
                                                   __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
      if (in && to < kSliceRegion) c.key[wave][to] = top_key(v, hits.id[w][at] + e);
      n += __popcll(who);
    }
  } else {
    n = kSliceRegion + 1;
  }
  if (__lane_id() == 0) c.n[wave] = n;
  __syncthreads();
  most = 0;
#pragma unroll
  for (int w = 0; w < kSliceWaves; ++w) most = max(most, c.n[w]);
  if (most <= kSliceRegion) return;
  // Too many (equal logits, or the largest with few threads): one at a time. Each thread
  // keeps its largest key below those taken, and looks for its next when it is taken.
  __syncthreads();
  unsigned long long best = 0, last = ~0ull;
  int taken = 0;
  for (int i = 0; i < k; ++i) {
    if (best == 0 && last != 0) {
      s.each_again(V, [&](const float* v, int id) {
#pragma unroll
        for (int e = 0; e < EPC; ++e) {
          const unsigned long long key = top_key(v[e], id + e);
          if (v[e] > kNegInf && key < last && key > best) best = key;
        }
      });
      if (best == 0) last = 0;   // none is left with this thread
    }
    const unsigned long long top = block_max_u64<kSliceBlock>(best, scratch);
    if (top == 0) break;
    if (threadIdx.x == 0) c.key[0][i] = top;
    ++taken;
    if (best == top) {
      last = top;
      best = 0;
    }
  }
  if (threadIdx.x < kSliceWaves) c.n[threadIdx.x] = threadIdx.x == 0 ? taken : 0;
  __syncthreads();
}

// ------------------------------------------------------------ a row's outputs
__device__ __forceinline__ int row_status(float M) {
  return M == kNegInf ? 2 : !(M < kPosInf) ? 1 : 0;
}

// Everything of row r but its alternatives, by T threads. Every thread of the wavefronts
// that call this has the row's sums.
template <int DT, int T>
__device__ __forceinline__ void put_row(const LogprobArgs& a, long long r, const Sums& all,
                                        double logZ, int t) {
  const unsigned char* row = a.logits + r * a.stride_bytes;
  const int status = row_status(all.M);
  const float nan = __uint_as_float(0x7FC00000u);
  bool bad = false;
  for (int i = t; i < a.n; i += T) {
    const int id = a.tokens[r * a.n + i];
    float lp = 0.0f;
    if (id != -1) {
      const bool in = id >= 0 && id < a.V;
      bad |= !in;
      lp = in && !status ? log_prob(load_elem<DT>(row, id), all.M, logZ, a.inv_t) : nan;
    }
    a.logprob[r * a.n + i] = lp;
  }
  const bool any_bad = __any(bad);
  if (t == 0) {
    if (a.entropy) a.entropy[r] = status ? nan : (float)(logZ - all.S / all.Z * kLn2);
    if (a.norm) {
      a.norm[2 * r] = status ? nan : all.M;
      a.norm[2 * r + 1] = status ? nan : (float)all.Z;
    }
    if (a.status) a.status[r] = status ? status : any_bad ? 3 : 0;
  }
}

// The k alternatives from the candidates.
template <int REGION>
__device__ __forceinline__ void put_top(const LogprobArgs& a, long long r, const Sums& all,
                                        double logZ, const Candidates<REGION>& c) {
  const int status = row_status(all.M);
  int total = 0;
#pragma unroll
  for (int w = 0; w < kSliceWaves; ++w) total += c.n[w];
  if (status) total = 0;
  for (int i = total + threadIdx.x; i < a.k; i += kSliceBlock) {   // positions past the last
    a.top_ids[r * a.k + i] = -1;
    a.top_logprob[r * a.k + i] = status ? __uint_as_float(0x7FC00000u) : kNegInf;
  }
  if (status) return;
  rank_candidates(c, a.k, [&](int rank, unsigned long long key) {
    a.top_ids[r * a.k + rank] = top_id(key);
    a.top_logprob[r * a.k + rank] = log_prob(top_value(key), all.M, logZ, a.inv_t);
  });
}

// Workspace: each slice's sums, then each slice's k largest keys, largest first.
struct LpWs {
  Sums* sums;                  // [rows][slices]
  unsigned long long* keys;    // [rows][slices][k]
};

// One workgroup to a slice of a row; with one slice it is the whole row's.
template <int DT, int NC, bool TOP, bool ONCE>
__global__ __launch_bounds__(kSliceBlock) void logprob_slice_kernel(LogprobArgs a, Cut cut,
                                                                    LpWs ws) {
  __shared__ Sums each[kSliceWaves];
  __shared__ uint32_t bound[kSliceWaves];
  __shared__ typename std::conditional<TOP, Candidates<kSliceRegion>, int>::type cands;
  __shared__ typename std::conditional<TOP, Hits<DT>, int>::type hits;
  __shared__ typename std::conditional<TOP, BlockScratch, int>::type scratch;
  const int slice = blockIdx.x % cut.slices;
  const long long r = blockIdx.x / cut.slices;
  Slice<DT, NC> s;
  s.template load<ONCE>(a.logits + r * a.stride_bytes, a.V, slice, cut);
  float cmax[NC + 1];
  const float m = s.largest([&](int j, float most) { cmax[j] = most; });
  if constexpr (TOP) {   // bf16 values have 16 bits; of float32 ones as many do
    const uint32_t jth = jth_largest<16>(fkey(m), (a.k + kSliceWaves - 1) / kSliceWaves);
    if (__lane_id() == 0) bound[threadIdx.x / kWave] = jth;
  }
  float off;
  const Sums mine = s.template sums<true>(a.V, m, a.c, off);
  const Sums all = join_block<kSliceWaves>(mine, a.c, off, each);
  if constexpr (TOP) {
    uint32_t tau = bound[0];
#pragma unroll
    for (int w = 1; w < kSliceWaves; ++w) tau = min(tau, bound[w]);
    tau = max(tau, kKeyNegInf);   // cut short, a key of -inf is one of NaN
    if (all.M == all.M)
      gather(s, a.V, cmax, tau, a.k, cands, hits, scratch);
    else if (threadIdx.x < kSliceWaves)
      cands.n[threadIdx.x] = 0;
  }
  if (cut.slices == 1) {
    const double logZ = log(all.Z);
    if (threadIdx.x < kWave) put_row<DT, kWave>(a, r, all, logZ, threadIdx.x);
    if constexpr (TOP) {
      __syncthreads();
      put_top(a, r, all, logZ, cands);
    }
    return;
  }
  const long long at = r * cut.slices + slice;
  if (threadIdx.x == 0) ws.sums[at] = all;
  if constexpr (TOP) {
    __syncthreads();
    unsigned long long* keys = ws.keys + at * a.k;
    int total = 0;
#pragma unroll
    for (int w = 0; w < kSliceWaves; ++w) total += cands.n[w];
    for (int i = total + threadIdx.x; i < a.k; i += kSliceBlock) keys[i] = 0;
    rank_candidates(cands, a.k, [&](int rank, unsigned long long key) { keys[rank] = key; });
  }
}

// Without alternatives: one wavefront to a row.
template <int DT>
__global__ __launch_bounds__(kSliceBlock) void logprob_join_kernel(LogprobArgs a, int slices,
                                                                   LpWs ws) {
  const long long r = (long long)blockIdx.x * kSliceWaves + threadIdx.x / kWave;
  if (r >= a.rows) return;
  const Sums all = join_slices(ws.sums + r * slices, slices, a.c);
  put_row<DT, kWave>(a, r, all, log(all.Z), __lane_id());
}

// With alternatives: one workgroup to a row. Each slice's j = ceil(k / slices) largest
// are k ids together, so the smallest of the slices' j-th keys bounds the k largest.
template <int DT>
__global__ __launch_bounds__(kSliceBlock) void logprob_top_join_kernel(LogprobArgs a, int slices,
                                                                       LpWs ws) {
  __shared__ Candidates<kJoinRegion> cands;
  constexpr int EACH = kJoinRegion / kWave;   // keys to a thread
  const long long r = blockIdx.x;
  const int lane = __lane_id(), wave = threadIdx.x / kWave;
  const unsigned long long* keys = ws.keys + r * slices * a.k;
  const int j = (a.k + slices - 1) / slices;
  unsigned long long tau = ~0ull;
  if (lane < slices) tau = keys[lane * a.k + j - 1];
  unsigned long long mine[EACH];
  const int total = slices * a.k;
#pragma unroll
  for (int q = 0; q < EACH; ++q) {
    const int i = q * kSliceBlock + (int)threadIdx.x;
    mine[q] = i < total ? keys[i] : 0;
  }
  const Sums all = join_slices(ws.sums + r * slices, slices, a.c);
  const double logZ = log(all.Z);
  tau = wave_reduce(tau, [](unsigned long long x, unsigned long long y) { return x < y ? x : y; });
  int n = 0;
#pragma unroll
  for (int q = 0; q < EACH; ++q) {
    const bool in = mine[q] != 0 && mine[q] >= tau;
    const unsigned long long who = __ballot(in);
    if (in)
      cands.key[wave][n + __builtin_amdgcn_mbcnt_hi(
                              (uint32_t)(who >> 32),
                              __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0))] = mine[q];
    n += __popcll(who);
  }
  if (lane == 0) cands.n[wave] = n;
  if (wave == kSliceWaves - 1) put_row<DT, kWave>(a, r, all, logZ, lane);
  __syncthreads();
  put_top(a, r, all, logZ, cands);
}

// ------------------------------------------------------------ rows past the slices
// Alternatives of vocabularies whose slices have more than 2048 of them together (with 64
// alternatives over 524288 float32 or 1048576 bf16 ids): one workgroup to a row, which it
// reads once for each sum and each alternative.
template <int DT>
__global__ __launch_bounds__(kLpBlock) void logprob_wide_kernel(LogprobArgs a) {
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
  const double logZ = log(Z);
  int bad_token = 0;
  const float nan = __uint_as_float(0x7FC00000u);
  for (int i = threadIdx.x; i < a.n; i += kLpBlock) {
    const int t = a.tokens[r * a.n + i];
    float lp = 0.0f;
    if (t != -1) {
      const bool in = t >= 0 && t < a.V;
      bad_token |= !in;
      lp = in && !status ? log_prob(load_elem<DT>(row, t), M, logZ, a.inv_t) : nan;
    }
    a.logprob[r * a.n + i] = lp;
  }
  bad_token = block_max<kLpBlock>(bad_token, scratch);
  if (threadIdx.x == 0) {
    if (a.entropy) a.entropy[r] = status ? nan : (float)(logZ - S / Z * kLn2);
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
      a.top_ids[at] = best ? top_id(best) : -1;
      a.top_logprob[at] = best ? log_prob(top_value(best), M, logZ, a.inv_t)
                               : status ? nan : kNegInf;
    }
  }
}

// ------------------------------------------------------------ the gradient
// One workgroup to a tile of a row; every wavefront forms the row's factors for itself.
template <int DT, bool ONCE>
__global__ __launch_bounds__(kSliceBlock) void logprob_grad_kernel(LogprobGradArgs a, int tiles) {
  const int tile = blockIdx.x % tiles;
  const long long r = blockIdx.x / tiles;
  const unsigned char* row = a.logits + r * a.stride_bytes;
  unsigned char* out = a.out + r * a.out_stride_bytes;
  const int32_t* tokens = a.tokens + r * a.n;
  const float* gs = a.g + r * a.n;
  const int t0 = tile * kTileIds<DT>, t1 = min(a.V, t0 + kTileIds<DT>);
  double G = 0.0;
  bool any = false, here = false;   // something comes back to the row; a token lies in the tile
  for (int i = __lane_id(); i < a.n; i += kWave) {
    const int t = tokens[i];
    const float g = gs[i];
    if (t == -1) continue;
    const bool in = t >= 0 && t < a.V;
    any |= g != 0.0f || !in;
    here |= t >= t0 && t < t1;
    G += in ? (double)g : __longlong_as_double(0x7FF8000000000000ll);
  }
  const float ge = a.ge ? a.ge[r] : 0.0f;
  if (!__any(any) && ge == 0.0f) {   // the row's logits are not looked at
    zero_tile<DT>(out, a.V, tile);
    return;
  }
  G = wave_sum(G);
  const float Z = a.norm[2 * r + 1];
  const double each = (double)a.inv_t / (double)Z;
  double A = -G * each, B = 0.0;
  if (ge != 0.0f) {
    A -= each * (double)ge * ((double)a.entropy[r] - log((double)Z));
    B = -each * (double)ge * kLn2;
  }
  const GradRow p(a.norm[2 * r], a.c, A, B);
  put_tile<DT, ONCE>(row, out, a.V, tile, p);
  if (!__any(here)) return;   // the same for all of the workgroup
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += kSliceBlock) {
    const int t = tokens[i];
    if (t < t0 || t >= t1) continue;
    float g = 0.0f;
    bool first = true;
    for (int k = 0; k < a.n; ++k) {
      if (tokens[k] != t) continue;
      if (k < i) first = false;
      g += gs[k];
    }
    if (first) store_elem<DT>(out, t, fmaf(g, a.inv_t, p.at(load_elem<DT>(row, t))));
  }
}

}  // namespace

namespace {

constexpr int kKeysMost = kJoinRegion * kSliceWaves;   // of a row's slices together

// How rows are cut (slices 0: not at all, the wide kernel).
Cut lp_cut(int dtype, int rows, int vocab, int k) {
  const int whole = vocab / (dtype == 0 ? 4 : 8);
  int want = std::min({1024 / max(rows, 1), 64, (whole + kSliceBlock - 1) / kSliceBlock});   // TUNE
  if (k) want = min(want, kKeysMost / k);
  const Cut c = cut_of(whole, want);
  return k && c.slices * (long long)k > kKeysMost ? Cut{0, 0, 0} : c;
}

template <int DT, bool TOP, bool ONCE>
void launch_slices(const LogprobArgs& a, const Cut& cut, const LpWs& ws, hipStream_t s) {
  const dim3 grid((unsigned)a.rows * (unsigned)cut.slices), block(kSliceBlock);
  switch (cut.nc) {
    case 1: hipLaunchKernelGGL((logprob_slice_kernel<DT, 1, TOP, ONCE>), grid, block, 0, s, a, cut, ws); break;
    case 2: hipLaunchKernelGGL((logprob_slice_kernel<DT, 2, TOP, ONCE>), grid, block, 0, s, a, cut, ws); break;
    case 4: hipLaunchKernelGGL((logprob_slice_kernel<DT, 4, TOP, ONCE>), grid, block, 0, s, a, cut, ws); break;
    case 8: hipLaunchKernelGGL((logprob_slice_kernel<DT, 8, TOP, ONCE>), grid, block, 0, s, a, cut, ws); break;
    default: hipLaunchKernelGGL((logprob_slice_kernel<DT, 16, TOP, ONCE>), grid, block, 0, s, a, cut, ws);
  }
}

template <int DT>
hipError_t launch_dt(const LogprobArgs& all, void* workspace, hipStream_t s) {
  const Cut cut = lp_cut(DT, all.rows, all.V, all.k);
  if (cut.slices == 0) {
    hipLaunchKernelGGL((logprob_wide_kernel<DT>), dim3(all.rows), dim3(kLpBlock), 0, s, all);
    return hipGetLastError();
  }
  const int batch = batch_of(cut, all.rows);
  for (int r0 = 0; r0 < all.rows; r0 += batch) {
    LogprobArgs a = all;
    a.rows = min(batch, all.rows - r0);
    a.logits += (long long)r0 * a.stride_bytes;
    if (a.tokens) a.tokens += (long long)r0 * a.n, a.logprob += (long long)r0 * a.n;
    if (a.entropy) a.entropy += r0;
    if (a.k) a.top_ids += (long long)r0 * a.k, a.top_logprob += (long long)r0 * a.k;
    if (a.norm) a.norm += 2ll * r0;
    if (a.status) a.status += r0;
    LpWs ws{static_cast<Sums*>(workspace), nullptr};
    ws.keys = reinterpret_cast<unsigned long long*>(ws.sums + (long long)a.rows * cut.slices);
    if (a.k)
      launch_slices<DT, true, false>(a, cut, ws, s);
    else
      launch_slices<DT, false, false>(a, cut, ws, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (cut.slices == 1) continue;
    if (a.k)
      hipLaunchKernelGGL((logprob_top_join_kernel<DT>), dim3(a.rows), dim3(kSliceBlock), 0, s, a,
                         cut.slices, ws);
    else
      hipLaunchKernelGGL((logprob_join_kernel<DT>), dim3((a.rows + kSliceWaves - 1) / kSliceWaves),
                         dim3(kSliceBlock), 0, s, a, cut.slices, ws);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t logprobs_ws_bytes(int dtype, int rows, int vocab, int k) {
  const Cut cut = lp_cut(dtype, rows, vocab, k);
  if (cut.slices <= 1) return 0;
  return (size_t)batch_of(cut, rows) * cut.slices * (sizeof(Sums) + 8 * (size_t)k);
}

hipError_t launch_logprobs(const LogprobArgs& a, int dtype, void* ws, hipStream_t s) {
  return dtype == 0 ? launch_dt<0>(a, ws, s) : launch_dt<1>(a, ws, s);
}

namespace {

template <int DT>
hipError_t launch_grad(const LogprobGradArgs& all, hipStream_t s) {
  const int tiles = tiles_of<DT>(all.V);
  const int batch = max(1, (1 << 23) / tiles);   // workgroups of a launch: fewer than 2^24
  for (int r0 = 0; r0 < all.rows; r0 += batch) {
    LogprobGradArgs a = all;
    a.rows = min(batch, all.rows - r0);
    a.logits += (long long)r0 * a.stride_bytes;
    a.out += (long long)r0 * a.out_stride_bytes;
    if (a.n) a.tokens += (long long)r0 * a.n, a.g += (long long)r0 * a.n;
    a.norm += 2ll * r0;
    if (a.ge) a.ge += r0, a.entropy += r0;
    hipLaunchKernelGGL((logprob_grad_kernel<DT, false>), dim3(a.rows * tiles), dim3(kSliceBlock), 0,
                       s, a, tiles);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_logprobs_grad(const LogprobGradArgs& a, int dtype, hipStream_t s) {
  return dtype == 0 ? launch_grad<0>(a, s) : launch_grad<1>(a, s);
}

}  // namespace tsr
