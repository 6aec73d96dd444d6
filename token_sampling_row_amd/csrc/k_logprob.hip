// Log probabilities of given tokens, entropy and the likeliest alternatives of
// rows of logits (token_logprobs), and the gradient of the first two
// (token_logprobs_grad).
//
//   x_j = (z_j - M) / T, M = max z, Z = sum_j exp(x_j), log p_j = x_j - log Z
//   H = log Z - sum_j exp(x_j) x_j / Z   (both terms >= 0: nothing cancels)
//   dL/dz_j = (sum_i g_i [t_i = j] - p_j (sum_i g_i + gH (log p_j + H))) / T
//
// Bound by memory: a logit is read once, and the gradient writes as much again. Rows are
// cut into slices that registers hold, and the largest logit, the sums and the likeliest
// ids are all taken from there; a wavefront to a row joins the slices. Measured, bf16:
//   1024 x 151936   slices 49 us (6.3 TB/s), join 5. With 64 alternatives 61 to 66 and
//                   9: there the vector pipes are busy throughout (1490 instructions
//                   a wavefront, 128 of them exponentials at a quarter of the rate)
//   1 x 128256, 20 alternatives   5.6 us and 7.2: latencies of loads and exchanges
//   320 x 32000 fp32   11 us in one launch, from the caches
//   gradient, 1024 x 128256   80 us (6.6 TB/s), with the entropy's 85 (6.2), into the
//                   same memory again; 98 into other memory (5.4)
#include <algorithm>
#include <type_traits>

#include "grad_tile.hpp"

namespace tsr {
namespace {

constexpr int kLpBlock = 256;

// ------------------------------------------------------------ the likeliest ids
// Keys of ids that may be among the k largest of a slice, in any order: more than kKeys
// are not kept.
constexpr int kKeys = 256;
struct Candidates {
  unsigned long long key[kKeys];
  int n;
};
// Chunks of a slice that hold candidates, a region for each wavefront.
constexpr int kHits = 64;
template <int WAVES>
struct Hits {
  uint4 chunk[WAVES][kHits];
  int id[WAVES][kHits];   // of the chunk's first element
};

__device__ __forceinline__ int lanes_below(unsigned long long who) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32),
                                   __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
}

// put(rank, key) for each candidate that fewer than k exceed. Keys differ, so ranks do.
template <class F>
__device__ __forceinline__ void rank_candidates(const Candidates& c, int k, F&& put) {
  const int n = c.n;
  if ((int)threadIdx.x >= n) return;
  const unsigned long long mine = c.key[threadIdx.x];
  int rank = 0;
#pragma unroll 4
  for (int q = 0; q < n; ++q) rank += c.key[q] > mine;
  if (rank < k) put(rank, mine);
}

// The slice's candidates: its logits of at least `tau` (a key of values), of which there
// are k at least and few more: every wavefront has j = ceil(k / wavefronts) threads whose
// largest logit is at least that. `cmax`: the largest of each chunk. A wavefront lists its
// chunks that hold any, and looks at the elements of those alone: taken where they lie,
// each chunk would cost it eight tests for one or two that pass (1024 x 151936 with 64
// alternatives: slices 78 us against 98 when the workgroup looked at its lists together;
// each wavefront at its own 60.5 against 63.4). c.n is 0 before the call.
//
// Logits that are equal by the score, in their upper 16 bits with float32, are all candidates.
// Where they are too many the likeliest are taken one at a time, k passes: 1024 x 151936 bf16
// with 64 alternatives, all equal or finfo.min but for eight, 2.3 ms against 74 us (with -inf
// in that place 58); 512 x 128256 fp32 with 20, each 1000 more, 609 us against 50 (100 more 52).
template <int DT, int NC, int BLOCK>
__device__ __forceinline__ void gather(const Slice<DT, NC, BLOCK>& s, int V, const float* cmax,
                                       uint32_t tau, int k, Candidates& c,
                                       Hits<BLOCK / kWave>& hits, BlockScratch& scratch) {
  constexpr int EPC = Fmt<DT>::EPC;
  const int wave = threadIdx.x / kWave;
  uint4* chunks = hits.chunk[wave];
  int* ids = hits.id[wave];
  const float least = fmaxf(key2f(tau), -3.4028235e38f);   // -inf is none
  int n = 0;   // the same for the wavefront
  const auto list = [&](float most, uint4 chunk, int id) {
    const bool in = most >= least;
    const unsigned long long who = __ballot(in);
    const int next = n + (int)__popcll(who);
    if (next != n && next <= kHits && in) {
      const int at = n + lanes_below(who);
      chunks[at] = chunk;
      ids[at] = id;
    }
    n = next;
  };
#pragma unroll
  for (int j = 0; j < NC; ++j) list(cmax[j], s.c[j], s.chunk_id(j) * EPC);
  if (s.ragged) list(cmax[NC], s.rest, V / EPC * EPC);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (n <= kHits) {
    for (int i0 = 0; i0 < n * EPC; i0 += kWave) {
      const int i = i0 + (int)__lane_id(), at = i / EPC, e = i % EPC;
      float v = kNegInf;
      if (i < n * EPC) {
        if constexpr (DT == 0)
          v = reinterpret_cast<const float*>(&chunks[at])[e];
        else
          v = __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(&chunks[at])[e] << 16);
      }
      const bool in = v >= least;
      const unsigned long long who = __ballot(in);
      int first = 0;
      if (__lane_id() == 0) first = atomicAdd(&c.n, (int)__popcll(who));
      const int to = __builtin_amdgcn_readfirstlane(first) + lanes_below(who);
      if (in && to < kKeys) c.key[to] = top_key(v, ids[at] + e);
    }
  } else if (__lane_id() == 0) {
    atomicAdd(&c.n, kKeys + 1);
  }
  __syncthreads();
  if (c.n <= kKeys) return;
  __syncthreads();
  // Too many (equal logits, or the largest with few threads): one at a time. Each thread
  // keeps its largest key below those taken, and looks for its next when it is taken.
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
    const unsigned long long top = block_max_u64<BLOCK>(best, scratch);
    if (top == 0) break;
    if (threadIdx.x == 0) c.key[i] = top;
    ++taken;
    if (best == top) {
      last = top;
      best = 0;
    }
  }
  if (threadIdx.x == 0) c.n = taken;
  __syncthreads();
}

// ------------------------------------------------------------ a row's outputs
__device__ __forceinline__ int row_status(float M) {
  return M == kNegInf ? 2 : !(M < kPosInf) ? 1 : 0;
}

// The lane's first token of row r and its logit, loaded ahead of their use.
struct Given {
  int id;
  float z;
};
template <int DT>
__device__ __forceinline__ Given first_token(const LogprobArgs& a, long long r) {
  Given g{-1, 0.0f};
  if ((int)__lane_id() < a.n) {
    g.id = a.tokens[r * a.n + __lane_id()];
    if (g.id >= 0 && g.id < a.V) g.z = load_elem<DT>(a.logits + r * a.stride_bytes, g.id);
  }
  return g;
}

// Everything of row r but its alternatives, by one wavefront.
template <int DT>
__device__ __forceinline__ void put_row(const LogprobArgs& a, long long r, const Sums& all,
                                        double logZ, Given g) {
  const unsigned char* row = a.logits + r * a.stride_bytes;
  const int status = row_status(all.M), lane = __lane_id();
  const float nan = __uint_as_float(0x7FC00000u);
  bool bad = false;
  for (int i = lane; i < a.n; i += kWave) {
    if (i != lane) {
      g.id = a.tokens[r * a.n + i];
      if (g.id >= 0 && g.id < a.V) g.z = load_elem<DT>(row, g.id);
    }
    float lp = 0.0f;
    if (g.id != -1) {
      const bool in = g.id >= 0 && g.id < a.V;
      bad |= !in;
      lp = in && !status ? log_prob(g.z, all.M, logZ, a.inv_t) : nan;
    }
    a.logprob[r * a.n + i] = lp;
  }
  const bool any_bad = __any(bad);
  if (lane == 0) {
    if (a.entropy) a.entropy[r] = status ? nan : (float)(logZ - all.S / all.Z * kLn2);
    if (a.norm) {
      a.norm[2 * r] = status ? nan : all.M;
      a.norm[2 * r + 1] = status ? nan : (float)all.Z;
    }
    if (a.status) a.status[r] = status ? status : any_bad ? 3 : 0;
  }
}

// Position `i` of row r's alternatives (key 0: there is none).
__device__ __forceinline__ void put_top(const LogprobArgs& a, long long r, int i,
                                        unsigned long long key, const Sums& all, double logZ) {
  const float none = row_status(all.M) ? __uint_as_float(0x7FC00000u) : kNegInf;
  a.top_ids[r * a.k + i] = key ? top_id(key) : -1;
  a.top_logprob[r * a.k + i] = key ? log_prob(top_value(key), all.M, logZ, a.inv_t) : none;
}

// Workspace: each slice's sums, how many candidates it has, and the candidates' keys.
struct LpWs {
  Sums* sums;                  // [rows][slices]
  unsigned long long* keys;    // [rows][slices][cap], cap 64 or 128
  int2* count;                 // [rows][slices]: how many, and a bound that k of them reach
  int cap;
};

// One workgroup to a slice of a row; with one slice it is the whole row's.
template <int DT, int NC, int BLOCK, bool TOP, bool ONCE>
__global__ __launch_bounds__(BLOCK) void logprob_slice_kernel(LogprobArgs a, Cut cut, LpWs ws) {
  constexpr int WAVES = BLOCK / kWave;
  __shared__ Sums each[WAVES];
  __shared__ uint32_t bound[WAVES];
  __shared__ typename std::conditional<TOP, Candidates, int>::type cands;
  __shared__ typename std::conditional<TOP, Hits<WAVES>, int>::type hits;
  __shared__ typename std::conditional<TOP, BlockScratch, int>::type scratch;
  const int slice = blockIdx.x % cut.slices;
  const long long r = blockIdx.x / cut.slices;
  Slice<DT, NC, BLOCK> s;
  s.template load<ONCE>(a.logits + r * a.stride_bytes, a.V, slice, cut);
  Given given;
  if (cut.slices == 1 && threadIdx.x < kWave) given = first_token<DT>(a, r);
  float cmax[NC + 1];
  const float m = s.largest([&](int j, float most) { cmax[j] = most; });
  if constexpr (TOP) {   // bf16 values have 16 bits; of float32 ones as many do
    const uint32_t jth = jth_largest<16>(fkey(m), (a.k + WAVES - 1) / WAVES);
    if (__lane_id() == 0) bound[threadIdx.x / kWave] = jth;
    if (threadIdx.x == 0) cands.n = 0;
  }
  float off;
  const Sums mine = s.template sums<true>(a.V, m, a.c, off);
  const Sums all = join_block<WAVES>(mine, a.c, off, each);
  uint32_t tau = 0;
  if constexpr (TOP) {
    tau = bound[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) tau = min(tau, bound[w]);
    tau = max(tau, kKeyNegInf);   // cut short, a key of -inf is one of NaN
    if (row_status(all.M) == 0) gather(s, a.V, cmax, tau, a.k, cands, hits, scratch);
  }
  if (cut.slices == 1) {
    if constexpr (TOP) {
      for (int i = cands.n + (int)threadIdx.x; i < a.k; i += BLOCK)
        put_top(a, r, i, 0, all, 0.0);   // past the last
      if ((int)threadIdx.x >= max(cands.n, kWave)) return;
    } else if (threadIdx.x >= kWave) {
      return;
    }
    const double logZ = log(all.Z);   // not by wavefronts that have nothing to put
    if (threadIdx.x < kWave) put_row<DT>(a, r, all, logZ, given);
    if constexpr (TOP)
      rank_candidates(cands, a.k, [&](int rank, unsigned long long key) {
        put_top(a, r, rank, key, all, logZ);
      });
    return;
  }
  const long long at = r * cut.slices + slice;
  if (threadIdx.x == 0) ws.sums[at] = all;
  if constexpr (TOP) {
    unsigned long long* keys = ws.keys + at * ws.cap;
    const int n = cands.n;
    if (threadIdx.x == 0) ws.count[at] = make_int2(n <= ws.cap ? n : a.k, (int)tau);
    if (n <= ws.cap) {
      if ((int)threadIdx.x < n) keys[threadIdx.x] = cands.key[threadIdx.x];
    } else {
      rank_candidates(cands, a.k, [&](int rank, unsigned long long key) { keys[rank] = key; });
    }
  }
}

// Without alternatives: one wavefront to a row.
template <int DT>
__global__ __launch_bounds__(kSliceBlock) void logprob_join_kernel(LogprobArgs a, int slices,
                                                                   LpWs ws) {
  const long long r = (long long)blockIdx.x * kSliceWaves + threadIdx.x / kWave;
  if (r >= a.rows) return;
  const Given given = first_token<DT>(a, r);
  const Sums all = join_slices(ws.sums + r * slices, slices, a.c);
  put_row<DT>(a, r, all, log(all.Z), given);
}

// With alternatives: one wavefront to a row, EACH of its slices' candidates to a lane. The
// k-th largest is found bit by bit, by counting those that are no smaller; what is left
// (k, and equal values at the end) goes to the lanes and is sorted.
template <int DT, int EACH>
__global__ __launch_bounds__(kSliceBlock) void logprob_top_join_kernel(LogprobArgs a, int slices,
                                                                       LpWs ws) {
  __shared__ unsigned long long kept[kSliceWaves][2 * kWave];
  const int lane = __lane_id(), wave = threadIdx.x / kWave;
  const long long r = (long long)blockIdx.x * kSliceWaves + wave;
  if (r >= a.rows) return;
  int2 count = make_int2(0, 0);
  if (lane < slices) count = ws.count[r * slices + lane];   // 32 at most
  const unsigned long long* keys = ws.keys + r * slices * ws.cap;
  const int slots = slices * ws.cap;
  unsigned long long key[EACH];
#pragma unroll
  for (int q = 0; q < EACH; ++q) key[q] = q * kWave < slots ? keys[q * kWave + lane] : 0;
  const Given given = first_token<DT>(a, r);
  const Sums all = join_slices(ws.sums + r * slices, slices, a.c);
  const bool fine = row_status(all.M) == 0;
  const int part = ws.cap / kWave;   // 1 or 2
  int total = 0;
#pragma unroll
  for (int q = 0; q < EACH; ++q) {   // places that hold no candidate
    const int slice = part == 1 ? q : q / 2, at = part == 1 ? 0 : q % 2 * kWave;
    const int n = slice < slices ? (int)readlane_u32((uint32_t)count.x, slice) - at : 0;
    if (lane >= n || !fine) key[q] = 0;
    total += min(max(n, 0), kWave);
  }
  const int need = fine ? min(a.k, total) : 0;
  const auto how_many = [&](unsigned long long least) {
    int n = 0;
#pragma unroll
    for (int q = 0; q < EACH; ++q) n += __popcll(__ballot(key[q] >= least));
    return n;
  };
  unsigned long long least = 1;   // every key, where there are no more than k
  if (total > need && fine) {
    // between the largest of the slices' bounds, which k reach, and the largest logit: the
    // bits that these share are the k-th largest's. Keys of bf16 values differ in their
    // upper 16 bits.
    const uint32_t from = max(wave_max_u32((uint32_t)count.y), 1u), to = fkey(all.M);
    constexpr int LAST = DT == 1 ? 16 : 0;
    int b = 31 - (int)__clz((int)(from ^ to));   // -1: they are equal
    uint32_t found = b >= 0 ? from >> b >> 1 << b << 1 : from;
    if (DT == 1) found &= 0xFFFF0000u;
#pragma unroll 1
    for (; b >= LAST; --b) {
      const uint32_t more = found | 1u << b;
      const int n = how_many((unsigned long long)more << 32);
      if (n >= need) found = more;
      if (n == need) break;
    }
    // bf16: what the search leaves out is set throughout in the keys of negative values, and 0
    // in the others'
    if (DT == 1 && !(found & 0x80000000u)) found |= 0xFFFFu;
    least = (unsigned long long)found << 32;
    if (how_many(least) > 2 * kWave) {   // so many equal values: the lower ids of them
#pragma unroll 1
      for (b = 31; b >= 0; --b) {
        const unsigned long long more = least | 1ull << b;
        if (how_many(more) >= need) least = more;
      }
    }
  }
  int n = 0;   // 128 at most, by the search
#pragma unroll
  for (int q = 0; q < EACH; ++q) {
    const bool in = key[q] >= least && key[q] != 0;
    const unsigned long long who = __ballot(in);
    const int to = n + lanes_below(who);
    if (in && to < 2 * kWave) kept[wave][to] = key[q];
    n += __popcll(who);
  }
  const double logZ = log(all.Z);
  put_row<DT>(a, r, all, logZ, given);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  unsigned long long sorted = wave_sort_desc<64>(lane < n ? kept[wave][lane] : 0ull);
  if (n > kWave) {
    // the larger of the i-th here and the 63 - i-th there: the 64 largest of both, in an
    // order that one merge sorts
    const unsigned long long more =
        wave_sort_desc<64>(lane < n - kWave ? kept[wave][kWave + lane] : 0ull);
    const unsigned long long turned =
        (unsigned long long)lane_mirror<64>((uint32_t)(more >> 32)) << 32 |
        lane_mirror<64>((uint32_t)more);
    sorted = turned > sorted ? turned : sorted;
    sorted = cx_layer<32, false>(sorted);
    sorted = cx_layer<16, false>(sorted);
    sorted = cx_layer<8, false>(sorted);
    sorted = cx_layer<4, false>(sorted);
    sorted = cx_layer<2, false>(sorted);
    sorted = cx_layer<1, false>(sorted);
  }
  if (lane < a.k) put_top(a, r, lane, sorted, all, logZ);
}

// ------------------------------------------------------------ rows past the slices
// Alternatives of vocabularies of more slices than their candidates' places hold (more
// than 40 alternatives: over 262144 float32 or 524288 bf16 ids; fewer: twice as many): one
// workgroup to a row, which it reads once for each sum and each alternative, an element at a
// time. Slow: 1 x 524301 bf16 with 64 alternatives 18.9 ms, 64 x 524301 38.6 ms (64 x 524288,
// in slices, 36 us), 64 x 1048589 with 20 26 ms, 64 x 524303 fp32 with 20 13.6 ms.
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
// PAST: past the caches are 1 the logits read, 2 the gradient written as well.
template <int DT, int PAST>
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
  const double each = a.inv_t / (double)Z;
  double A = -G * each, B = 0.0;
  if (ge != 0.0f) {
    A -= each * (double)ge * ((double)a.entropy[r] - log((double)Z));
    B = -each * (double)ge * kLn2;
  }
  const GradRow p(a.norm[2 * r], a.c, A, B);
  put_tile<DT, PAST >= 1, PAST == 2>(row, out, a.V, tile, p);
  if (!__any(here)) return;   // the same for all of the workgroup
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += kSliceBlock) {
    const int t = tokens[i];
    if (t < t0 || t >= t1) continue;
    double g = 0.0;   // gradients of one id may cancel
    bool first = true;
    for (int k = 0; k < a.n; ++k) {
      if (tokens[k] != t) continue;
      if (k < i) first = false;
      g += (double)gs[k];
    }
    if (first)
      store_elem<DT>(out, t, (float)fma(g, a.inv_t, (double)p.at(load_elem<DT>(row, t))));
  }
}

}  // namespace

namespace {

constexpr int kSlotsMost = 2048;   // places for candidates of a row's slices: 32 a lane

// Places for a slice's candidates: some half more than k come as a rule.
int cap_of(int k) { return k == 0 ? 0 : k <= 40 ? kWave : 2 * kWave; }

constexpr int kRowBlock = 1024;   // threads of a workgroup that takes a whole row

// How rows are cut (slices 0: not at all, the wide kernel).
//  - Up to 1024 chunks: one workgroup of 256 threads and one launch. 1000 x 8192 bf16
//    7.8 us, in workgroups of 1024 threads 13.6; 1024 x 8192 with 20 alternatives 11.4.
//  - Few rows of up to 8192 chunks: one workgroup of 1024 threads, which saves the join.
//    1 x 32000 fp32, 20 alternatives 9.9 us against 11.8 in slices and their join; 64 rows
//    12.4 against 15.4; 256 x 32000 bf16 14.1 against 16.8, but 512 24 against 18. Without
//    alternatives 512 x 32000 fp32 14.3 against 16.3.
//  - Else slices: as many as give a thousand workgroups, at least what holds the row. 333 x
//    50001 fp32 with 5 alternatives 21.9 us, for two thousand 22.9, for four thousand 26.6
//    (each slice's candidates go to the join); without them 16.9, 15.8 and 15.8.
Cut lp_cut(int dtype, int rows, int vocab, int k) {
  const int whole = vocab / (dtype == 0 ? 4 : 8);
  if (whole <= 4 * kSliceBlock) return cut_of(whole, 1);
  if (whole <= 8 * kRowBlock && rows <= (k ? 256 : 512)) {
    Cut c{1, whole, 1, kRowBlock};
    while (c.nc * kRowBlock < whole) c.nc *= 2;
    return c;
  }
  int want = std::min({1024 / max(rows, 1), 64, (whole + kSliceBlock - 1) / kSliceBlock});
  if (k) want = min(want, 1024 / cap_of(k));
  const Cut c = cut_of(whole, want);
  return k && c.slices > kSlotsMost / cap_of(k) ? Cut{0, 0, 0} : c;
}

// Places in the workspace for a batch of rows.
size_t lp_bytes(const Cut& cut, int rows, int k) {
  return (size_t)rows * cut.slices *
         (sizeof(Sums) + (size_t)cap_of(k) * 8 + (k ? sizeof(int2) : 0));
}

// Candidates' places a lane: each step of the search counts all of them, so as few as hold the
// slices'. 1024 rows, 20 alternatives, kernel us: 4 slices 5.7 with 4 places, 6.2 with 6; 5
// slices 6.0 with 6, 6.8 with 8; 8 slices 6.4 with 8, 7.0 with 10; 16 slices 8.4 with 16, 12.1
// with 32 (64 rows 7.3, 10.7); 5 slices of 128 places 8.4 with 10, 8.8 with 16.
template <int DT>
void launch_top_join(const LogprobArgs& a, int slices, const LpWs& ws, hipStream_t s) {
  const dim3 grid((a.rows + kSliceWaves - 1) / kSliceWaves), block(kSliceBlock);
  const auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, s, a, slices, ws);
  };
  const int each = slices * ws.cap / kWave;
  if (each <= 4) return launch(logprob_top_join_kernel<DT, 4>);
  if (each <= 6) return launch(logprob_top_join_kernel<DT, 6>);
  if (each <= 8) return launch(logprob_top_join_kernel<DT, 8>);
  if (each <= 10) return launch(logprob_top_join_kernel<DT, 10>);
  if (each <= 16) return launch(logprob_top_join_kernel<DT, 16>);
  launch(logprob_top_join_kernel<DT, 32>);
}

template <int DT, bool TOP, bool ONCE>
void launch_slices(const LogprobArgs& a, const Cut& cut, const LpWs& ws, hipStream_t s) {
  const auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)a.rows * (unsigned)cut.slices), dim3(cut.block), 0, s,
                       a, cut, ws);
  };
  if (cut.block == kRowBlock) {
    if (cut.nc == 2) return launch(logprob_slice_kernel<DT, 2, kRowBlock, TOP, false>);
    if (cut.nc == 4) return launch(logprob_slice_kernel<DT, 4, kRowBlock, TOP, false>);
    return launch(logprob_slice_kernel<DT, 8, kRowBlock, TOP, false>);   // 67 MB at most
  }
  if (cut.nc == 1) return launch(logprob_slice_kernel<DT, 1, kSliceBlock, TOP, false>);
  if (cut.nc == 2) return launch(logprob_slice_kernel<DT, 2, kSliceBlock, TOP, false>);
  if (cut.nc == 4) return launch(logprob_slice_kernel<DT, 4, kSliceBlock, TOP, ONCE>);
  if (cut.nc == 8) return launch(logprob_slice_kernel<DT, 8, kSliceBlock, TOP, ONCE>);
  launch(logprob_slice_kernel<DT, 16, kSliceBlock, TOP, ONCE>);
}

// Batches of more bytes than this are read past the caches, which could not keep them: 512 x
// 128256 fp32 with 20 alternatives 51 us against 56, 1024 x 151936 bf16 with 64 76 against
// 78. Smaller ones may be there still, from the product that wrote them.
constexpr long long kOnceBytes = 128ll << 20;

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
    LpWs ws;
    const long long slots = (long long)a.rows * cut.slices;
    ws.cap = cap_of(a.k);
    ws.sums = static_cast<Sums*>(workspace);
    ws.keys = reinterpret_cast<unsigned long long*>(ws.sums + slots);
    ws.count = reinterpret_cast<int2*>(ws.keys + slots * ws.cap);
    const bool once = (long long)all.rows * all.V * Fmt<DT>::ESZ > kOnceBytes;
    if (a.k)
      once ? launch_slices<DT, true, true>(a, cut, ws, s)
           : launch_slices<DT, true, false>(a, cut, ws, s);
    else
      once ? launch_slices<DT, false, true>(a, cut, ws, s)
           : launch_slices<DT, false, false>(a, cut, ws, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (cut.slices == 1) continue;
    if (a.k)
      launch_top_join<DT>(a, cut.slices, ws, s);
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
  return lp_bytes(cut, batch_of(cut, rows), k);
}

hipError_t launch_logprobs(const LogprobArgs& a, int dtype, void* ws, hipStream_t s) {
  return dtype == 0 ? launch_dt<0>(a, ws, s) : launch_dt<1>(a, ws, s);
}

namespace {

template <int DT>
hipError_t launch_grad(const LogprobGradArgs& all, hipStream_t s) {
  const int tiles = tiles_of<DT>(all.V);
  const int batch = max(1, (1 << 23) / tiles);   // workgroups of a launch: fewer than 2^24
  // Logits that the caches could not keep beside the gradient are read past them: 1024 x
  // 128256 bf16 80 us against 101 (6.6 TB/s), but 256 x 128256 26 against 22.
  const long long bytes = (long long)all.rows * all.V * Fmt<DT>::ESZ;
  for (int r0 = 0; r0 < all.rows; r0 += batch) {
    LogprobGradArgs a = all;
    a.rows = min(batch, all.rows - r0);
    a.logits += (long long)r0 * a.stride_bytes;
    a.out += (long long)r0 * a.out_stride_bytes;
    if (a.n) a.tokens += (long long)r0 * a.n, a.g += (long long)r0 * a.n;
    a.norm += 2ll * r0;
    if (a.ge) a.ge += r0, a.entropy += r0;
    const auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(a.rows * tiles), dim3(kSliceBlock), 0, s, a, tiles);
    };
    if (bytes > kGradOnceBytes)
      launch(logprob_grad_kernel<DT, 2>);
    else if (bytes > kOnceBytes)
      launch(logprob_grad_kernel<DT, 1>);
    else
      launch(logprob_grad_kernel<DT, 0>);
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
