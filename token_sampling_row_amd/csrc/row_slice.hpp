// A row of logits cut into slices, one to a workgroup, each held in registers: read
// once, its sums taken against each thread's own largest logit (no exchange before the
// exponentials) and joined afterwards.
//
// A thread's weights: rc = fl(m c) for its largest m, x = fma(z, c, -rc), e = 2^x.
// x is the exponent (z - m) c but for rc - m c, the same for all of the thread's
// elements and known exactly (one fma): it goes into the factor that joins the
// thread to the others. That is one fma an element where (z - m) c takes two
// roundings and two instructions.
//
// Slices are of 16 chunks a thread at most (64 registers): 256 threads hold 32768 bf16
// logits, and a row of 151936 is five slices (token_logprobs of 1024 with 64 alternatives
// 73 us; in slices of 8 chunks a thread 88, most of it the selection's). Wider workgroups
// hold whole rows where that saves a second read (distill_topk) or a second launch
// (token_logprobs of few rows).
#pragma once

#include "kernels.hpp"
#include "scores.hpp"
#include "wide_mem.hpp"

namespace tsr {

constexpr int kSliceBlock = 256;
constexpr int kSliceWaves = kSliceBlock / kWave;

// How a row is cut: `slices` workgroups of up to `per` whole chunks each, `nc` to a
// thread (the elements behind the last whole chunk go with the last slice).
struct Cut {
  int slices, per, nc;
  int block = kSliceBlock;   // threads of a workgroup
};

// Weights against a largest logit M: their sum, and that of weight times exponent.
struct Sums {
  float M;
  double Z, S;
};

// What joins sums against m to others against M: 2^d with d = (m - M) c + off. -inf has
// no weight; NaN stays.
__device__ __forceinline__ void rebase(Sums& a, float M, float c, float off) {
  const float d = a.M == M ? off : fmaxf(fmaf(a.M - M, c, off), -2000.0f);
  const double f = (double)__builtin_amdgcn_exp2f(d);
  a.S = f * fma(a.Z, (double)d, a.S);
  a.Z *= f;
  a.M = M;
}

// The workgroup's sums from its threads'; `each` has a place for every wavefront.
template <int WAVES>
__device__ __forceinline__ Sums join_block(Sums a, float c, float off, Sums* each) {
  rebase(a, wave_maxn(a.M), c, off);
  a.Z = wave_sum(a.Z);
  a.S = wave_sum(a.S);
  if (__lane_id() == 0) each[threadIdx.x / kWave] = a;
  __syncthreads();
  if constexpr (WAVES > 4) {   // a lane for each: together they would take 100 registers
    Sums one{kNegInf, 0.0, 0.0};
    if ((int)__lane_id() < WAVES) one = each[__lane_id()];
    rebase(one, reduce_w<16>(one.M, [](float x, float y) { return fmaxn(x, y); }), c, 0.0f);
    one.Z = sum_w<16>(one.Z);
    one.S = sum_w<16>(one.S);
    return one;
  }
  float M = each[0].M;
#pragma unroll
  for (int w = 1; w < WAVES; ++w) M = fmaxn(M, each[w].M);
  Sums all{M, 0.0, 0.0};
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    Sums one = each[w];
    rebase(one, M, c, 0.0f);
    all.Z += one.Z;
    all.S += one.S;
  }
  return all;
}

// The sums of a row from its slices', by each wavefront for itself.
__device__ __forceinline__ Sums join_slices(const Sums* sums, int slices, float c) {
  Sums one{kNegInf, 0.0, 0.0};
  for (int i = __lane_id(); i < slices; i += kWave) {
    Sums next = sums[i];
    const float M = fmaxn(one.M, next.M);
    rebase(one, M, c, 0.0f);
    rebase(next, M, c, 0.0f);
    one.Z += next.Z;
    one.S += next.S;
  }
  rebase(one, wave_maxn(one.M), c, 0.0f);
  one.Z = wave_sum(one.Z);
  one.S = wave_sum(one.S);
  return one;
}

constexpr int kMaxSliceChunks = 16 * kSliceBlock;   // of the largest slice, 16 a thread

// A cut of rows of `whole` chunks into `slices` or as many as hold them.
inline Cut cut_of(int whole, int slices) {
  Cut c{slices, 0, 1};
  const int least = (whole + kMaxSliceChunks - 1) / kMaxSliceChunks;
  c.slices = least > slices ? least : slices < 1 ? 1 : slices;
  c.per = (whole + c.slices - 1) / c.slices;
  while (c.nc * kSliceBlock < c.per) c.nc *= 2;
  return c;
}
// Rows whose slices are in the workspace at a time.
inline int batch_of(const Cut& c, int rows) {
  const int most = c.slices > 64 ? (1 << 19) / c.slices : 1 << 13;
  return rows < most ? rows : most;
}

template <int DT>
__device__ __forceinline__ float max_of(const float* v) {
  if constexpr (DT == 0) return fmaxn(fmax3n(v[0], v[1], v[2]), v[3]);
  return fmaxn(fmax3n(fmax3n(v[0], v[1], v[2]), v[3], v[4]), fmax3n(v[5], v[6], v[7]));
}

template <int DT, int NC, int BLOCK = kSliceBlock>
struct Slice {
  static constexpr int EPC = Fmt<DT>::EPC;
  const unsigned char* row;
  uint4 c[NC];
  uint4 rest;   // the elements behind the last whole chunk, with one thread of the last slice
  int lo, hi;   // the slice's whole chunks
  bool ragged;

  __device__ __forceinline__ int chunk_id(int j) const {
    return lo + j * BLOCK + (int)threadIdx.x;
  }

  // Whether any thread has a j-th chunk (the same for all of them).
  __device__ __forceinline__ bool has(int j) const { return j * BLOCK < hi - lo; }

  // Loads are addressed from a uniform base; threads past the slice's last chunk repeat
  // it, and `largest` puts -inf in its place.
  template <bool ONCE>
  __device__ __forceinline__ void load(const unsigned char* at, int V, int slice, const Cut& cut) {
    row = at;
    const int whole = V / EPC;
    lo = slice * cut.per;
    hi = min(lo + cut.per, whole);
    ragged = slice == cut.slices - 1 && whole * EPC < V;
    const unsigned char* base =
        whole > 0 ? row + (long long)min(lo, whole - 1) * 16
                  : reinterpret_cast<const unsigned char*>(&g_neg_inf_chunk[DT]);
    const uint32_t last = (uint32_t)max(hi - lo - 1, 0);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const unsigned char* p = base + min((uint32_t)(j * BLOCK) + threadIdx.x, last) * 16u;
      c[j] = ONCE ? load16_once(p) : load16(p);
    }
    rest = neg_inf_chunk<DT>();
    if (ragged && threadIdx.x == BLOCK - 1) rest = load_chunk_slow<DT>(row, whole, V);
  }

  // f(values, number of the first) for each chunk of the thread
  template <class F>
  __device__ __forceinline__ void each(int V, F&& f) const {
    const Pass pass;
    float v[EPC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      if (!has(j)) continue;
      pass.unpack<DT>(c[j], v);
      f(v, chunk_id(j) * EPC);
      sched_fence();
    }
    if (ragged) {
      pass.unpack<DT>(rest, v);
      f(v, V / EPC * EPC);
    }
  }

  // The same for passes that are seldom taken: the chunks read again, one at a time.
  template <class F>
  __device__ __forceinline__ void each_again(int V, F&& f) const {
    float v[EPC];
#pragma unroll 1
    for (int i = lo + (int)threadIdx.x; i < hi; i += BLOCK) {
      tsr::unpack<DT>(load16(row + (long long)i * 16), v);
      f(v, i * EPC);
    }
    if (ragged) {
      tsr::unpack<DT>(rest, v);
      f(v, V / EPC * EPC);
    }
  }

  // Leaves the ids of a row's entries (one to a lane of every wavefront, -1: none) out of
  // the slice: their logits become -inf. Eight bits a chunk, a thread's together. Each
  // wavefront lists those of its own chunks: no barrier before the sums (with one they
  // start when the slowest wavefront's ids have come: 1024 x 128256 115 us against 105).
  struct LeftOut {
    uint32_t word[BLOCK][(NC + 3) / 4];
  };
  __device__ __forceinline__ void leave_out(int V, int id, LeftOut& out) {
    constexpr int W = (NC + 3) / 4;
#pragma unroll
    for (int w = 0; w < W; ++w) out.word[threadIdx.x][w] = 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int q = id < 0 ? -1 : id / EPC - lo;
    if (q >= 0 && q < hi - lo && q % BLOCK / kWave == (int)threadIdx.x / kWave) {
      const int j = q / BLOCK;
      atomicOr(&out.word[q % BLOCK][j / 4], 1u << (8 * (j % 4) + id % EPC));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (ragged) {   // behind the last whole chunk: with every wavefront's own ids
      const int at = V / EPC * EPC;
      uint32_t bits = 0;
      unsigned long long who = __ballot(id >= at);
      while (who) {
        bits |= 1u << ((int)readlane_u32((uint32_t)id, __ffsll((long long)who) - 1) - at);
        who &= who - 1;
      }
      drop(rest, bits);
    }
    uint32_t word[W], any = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) any |= word[w] = out.word[threadIdx.x][w];
    if (!__any(any != 0)) return;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const uint32_t bits = word[j / 4] >> (8 * (j % 4)) & 255u;
      if (__any(bits != 0)) drop(c[j], bits);
    }
  }
  static __device__ __forceinline__ void drop(uint4& ch, uint32_t bits) {
    uint32_t w[4] = {ch.x, ch.y, ch.z, ch.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == 0) {
        w[i] = bits >> i & 1 ? 0xFF800000u : w[i];
      } else {
        w[i] = bits >> (2 * i) & 1 ? (w[i] & 0xFFFF0000u) | 0xFF80u : w[i];
        w[i] = bits >> (2 * i + 1) & 1 ? (w[i] & 0xFFFFu) | 0xFF800000u : w[i];
      }
    }
    ch = make_uint4(w[0], w[1], w[2], w[3]);
  }

  // The thread's largest logit, NaN where it holds one; of(j, largest of chunk j) for each
  // (j = NC: the elements behind the last whole chunk).
  template <class F>
  __device__ __forceinline__ float largest(F&& of) {
    const Pass pass;
    float v[EPC], m = kNegInf;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      if (!has(j)) {
        of(j, kNegInf);
        continue;
      }
      if ((j + 1) * BLOCK > hi - lo) {   // the same for all threads
        const uint4 none = neg_inf_chunk<DT>();
        const bool in = chunk_id(j) < hi;
        c[j].x = in ? c[j].x : none.x;
        c[j].y = in ? c[j].y : none.y;
        c[j].z = in ? c[j].z : none.z;
        c[j].w = in ? c[j].w : none.w;
      }
      pass.unpack<DT>(c[j], v);
      const float most = max_of<DT>(v);
      of(j, most);
      m = fmaxn(m, most);
      sched_fence();
    }
    float most = kNegInf;
    if (ragged) {
      pass.unpack<DT>(rest, v);
      most = max_of<DT>(v);
    }
    of(NC, most);
    return fmaxn(m, most);
  }

  // The thread's sums against its largest logit m (S in units of log 2) and what its
  // exponents are short of. Sixteen products at most are added in float32. Exponents are
  // held above -2000, where weights are 0: a logit of -inf gives 0 in S and not NaN.
  template <bool WITH_S>
  __device__ __forceinline__ Sums sums(int V, float m, float c_log2, float& off) const {
    constexpr int GROUP = 16 / EPC;   // chunks whose products are added in float32
    const float ref = m > kNegInf ? m : 0.0f;
    const float rc = ref * c_log2;
    off = -fmaf(ref, c_log2, -rc);
    Sums a{m, 0.0, 0.0};
    float z = 0.0f, s = 0.0f;
    const auto add = [&](const float* v, auto&& x_of) {
#pragma unroll
      for (int e = 0; e < EPC; ++e) {
        const float x = x_of(v[e]);
        const float w = __builtin_amdgcn_exp2f(x);
        z += w;
        if constexpr (WITH_S) s = fmaf(w, x, s);
      }
    };
    const auto flush = [&] {
      a.Z += (double)z;
      if constexpr (WITH_S) a.S += (double)s;
      z = s = 0.0f;
    };
    if (fabsf(rc) <= 0x1p20f) {
      const auto x_of = [&](float v) {
        const float x = fmaf(v, c_log2, -rc);
        return WITH_S ? fmaxf(x, -2000.0f) : x;
      };
      const Pass pass;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        float v[EPC];
        if (has(j)) {
          pass.unpack<DT>(c[j], v);
          add(v, x_of);
        }
        if (j % GROUP == GROUP - 1) flush();
        sched_fence();
      }
      if (NC % GROUP) flush();
      if (ragged) {
        float v[EPC];
        pass.unpack<DT>(rest, v);
        add(v, x_of);
        flush();
      }
    } else {   // the rounding of m c is no small shift of the exponents
      off = 0.0f;
      each(V, [&](const float* v, int) {
        add(v, [&](float y) { return exponent(y, ref, c_log2); });
        flush();
      });
    }
    return a;
  }
};

// The j-th largest of a wavefront's keys, or less: its first BITS bits and zeros.
template <int BITS>
__device__ __forceinline__ uint32_t jth_largest(uint32_t key, int j) {
  uint32_t found = 0;
#pragma unroll
  for (int b = 31; b > 31 - BITS; --b) {
    const uint32_t more = found | 1u << b;
    if (__popcll(__ballot(key >= more)) >= j) found = more;
  }
  return found;
}

}  // namespace tsr
