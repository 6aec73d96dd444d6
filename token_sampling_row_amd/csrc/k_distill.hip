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
//
// Bound by memory: a logit is read once and its gradient written once where a workgroup's
// registers hold the row, which is all that the row kernel moves. Wider rows, and few of
// them, go through slices, and the gradient reads the logits again, from the caches where
// they are no more than those hold. Measured, bf16, kernel and TB/s of the logits and the
// gradient together:
//   1024 x 151936, 64 entries, tail   124 to 129 us (5.0 to 4.8): a row takes its compute
//                   unit's registers whole, so a row's stores and the next one's loads
//                   overlap only as far as wavefronts end
//   1024 x 128256, tail 105 us (5.0), without 100; 256 x 128256, 20 entries 24 us (5.5)
//   33 x 8191 fp32  7 us: one row's latencies
//   512 x 128256 fp32   slices 47 us, join 8, gradient 76
#include <algorithm>

#include "grad_tile.hpp"

namespace tsr {
namespace {

constexpr float kRestMin = 0x1p-20f;  // a remainder below this is rounding of the entries

// The entries of a row, one to a lane of a wavefront.
struct Entries {
  int id;              // -1: none, or a lane past the last
  bool first;          // no lower lane holds the same id
  double q, log_q;     // the teacher's probability
  double same;         // sum of q over the lanes of this id
  double sum, rest;
  int status;
  float z;             // its logit
};

__device__ __forceinline__ int raw_id(const DistillArgs& a, long long r) {
  const int lane = __lane_id();
  return lane < a.k ? a.ids[r * a.k + lane] : -1;
}
__device__ __forceinline__ float teacher_of(const DistillArgs& a, long long r) {
  const int lane = __lane_id();
  return lane < a.k ? a.teacher[r * a.k + lane] : kNegInf;
}
// -1 for what is no id of the vocabulary
__device__ __forceinline__ int valid_id(const DistillArgs& a, int id) {
  return id >= 0 && id < a.V ? id : -1;
}

__device__ __forceinline__ Entries entries_of(const DistillArgs& a, int id, float t) {
  Entries e;
  const int lane = __lane_id();
  e.id = id;
  const bool real = id != -1;
  e.status = 0;
  const bool outside = real && valid_id(a, id) < 0;
  if (__any(outside)) e.status = 3;
  else if (__any(real && !(t < kPosInf))) e.status = 1;
  const float top = wave_max(real ? t : kNegInf);   // drops NaN: those rows are marked
  if (!e.status && top == kNegInf) e.status = 2;
  if (outside) e.id = -1;
  // with a tail the values are log probabilities; without one any row constant cancels
  const double shift = a.tail || e.status ? 0.0 : (double)top;
  e.q = real && t > kNegInf ? exp_small((double)t - shift) : 0.0;
  e.log_q = (double)t - shift;
  e.sum = wave_sum(e.q);
  e.rest = 0.0;
  if (a.tail) {
    e.rest = 1.0 - e.sum;
    if (!(e.rest > (double)kRestMin)) e.rest = 0.0;
  } else {
    e.q /= e.sum;
    e.log_q -= log_small(e.sum);
    e.sum = 1.0;
  }
  e.first = e.id >= 0;
  e.same = e.q;
  bool twice = false;
  for (int l = 0; l < a.k; ++l)
    twice |= (int)readlane_u32((uint32_t)e.id, l) == e.id && l != lane;
  if (__any(twice && e.first)) {   // an id that comes again: one order for all of its lanes
    e.same = 0.0;
    for (int l = 0; l < a.k; ++l) {
      const bool is = (int)readlane_u32((uint32_t)e.id, l) == e.id;
      const double q = readlane_f64(e.q, l);
      if (is) e.same += q;
      if (is && l < lane) e.first = false;
    }
  }
  return e;
}

// A row's sums with its entries': M and Z of all ids, and of the ids outside S (of all,
// without a tail) against their own largest, Mr and Zr.
struct RowSums {
  float M, Mr;
  double Z, Zr;
  int status;
};

// By one wavefront.
__device__ __forceinline__ RowSums row_sums(const DistillArgs& a, const Entries& e,
                                            const Sums& other) {
  RowSums s;
  s.Mr = other.M;
  s.Zr = other.Z;
  s.M = fmaxn(other.M, a.tail ? wave_maxn(e.id >= 0 ? e.z : kNegInf) : kNegInf);
  s.status = e.status ? e.status : s.M == kNegInf ? 2 : !(s.M < kPosInf) ? 1 : 0;
  s.Z = other.Z;
  if (a.tail) {   // what a weight against Mr is against M
    const float f = other.M > kNegInf ? __builtin_amdgcn_exp2f(exponent(other.M, s.M, a.c)) : 0.0f;
    const float ez = __builtin_amdgcn_exp2f(exponent(e.z, s.M, a.c));
    s.Z = other.Z * (double)f + wave_sum(e.first ? (double)ez : 0.0);
  }
  return s;
}

// What the gradient of a row takes: e_j A for weights against M, and an entry's own value.
struct RowGrad {
  float M;
  double A;
  float entry;
};
__device__ __forceinline__ RowGrad row_grad_of(const DistillArgs& a, float weight,
                                               const Entries& e, const RowSums& s) {
  const double each = (double)weight * a.inv_t, whole = e.sum + e.rest;
  const double f = a.tail ? (double)__builtin_amdgcn_exp2f(exponent(s.Mr, s.M, a.c)) : 1.0;
  const double ez = e.id >= 0 ? (double)__builtin_amdgcn_exp2f(exponent(e.z, s.M, a.c)) : 0.0;
  const float nan = __uint_as_float(0x7FC00000u);
  RowGrad g;
  // without an id outside S there is no weight to multiply: any M and a factor of 0
  g.M = s.Mr == kNegInf ? 0.0f : s.Mr;
  g.A = s.status ? (double)nan : s.Zr > 0.0 ? each * (whole * f / s.Z - e.rest / s.Zr) : 0.0;
  g.entry = s.status ? nan : (float)(each * (whole * ez / s.Z - e.same));
  return g;
}

// Loss and status of row r.
__device__ __forceinline__ void put_loss(const DistillArgs& a, long long r, float weight,
                                         const Entries& e, const RowSums& s) {
  const double logZ = log_small(s.Z);
  double term = 0.0;
  if (e.q > 0.0) term = e.q * (e.log_q - (((double)e.z - (double)s.M) * a.inv_t - logZ));
  double loss = wave_sum(term);
  if (e.rest > 0.0) {   // +inf where the draft gives the other ids nothing
    const double log_pr = s.Mr > kNegInf
                              ? log_small(s.Zr) + ((double)s.Mr - (double)s.M) * a.inv_t - logZ
                              : -__builtin_huge_val();
    loss += e.rest * (log_small(e.rest) - log_pr);
  }
  if (__lane_id() == 0) {
    a.loss[r] = s.status ? __uint_as_float(0x7FC00000u) : (float)(loss * weight);
    if (a.status) a.status[r] = s.status;
  }
}

// A row that does not count.
__device__ __forceinline__ void put_nothing(const DistillArgs& a, long long r) {
  a.loss[r] = 0.0f;
  if (a.status) a.status[r] = 0;
}

// ------------------------------------------------------------ a row in one workgroup
// Read once: the gradient is formed from the registers that the sums were. PAST: past the
// caches are 1 the logits read, 2 the gradient written as well.
template <int DT, int NC, int BLOCK, int PAST>
__global__ __launch_bounds__(BLOCK) void distill_row_kernel(DistillArgs a) {
  constexpr int EPC = Fmt<DT>::EPC;
  __shared__ Sums each[BLOCK / kWave];
  __shared__ typename Slice<DT, NC, BLOCK>::LeftOut left_out;
  __shared__ Entries entries[kWave];   // kept here between the two uses: registers are short
  __shared__ float own[kWave];         // the entries' gradients
  __shared__ struct {
    RowSums sums;
    float M;
    double A;
  } row_grad;
  const long long r = blockIdx.x;
  unsigned char* out = a.grad ? a.grad + r * a.grad_stride_bytes : nullptr;
  const int whole = a.V / EPC;
  const float weight = a.weight ? a.weight[r] : 1.0f;
  if (weight == 0.0f) {   // the row does not count: neither its logits nor its entries do
    if (out) {
      for (int i = threadIdx.x; i < whole; i += BLOCK)
        store16<false>(out + (long long)i * 16, make_uint4(0, 0, 0, 0));
      if ((int)threadIdx.x < a.V - whole * EPC)
        store_elem<DT>(out, whole * EPC + (int)threadIdx.x, 0.0f);
    }
    if (threadIdx.x == 0) put_nothing(a, r);
    return;
  }
  const int id = raw_id(a, r);
  const float t = teacher_of(a, r);
  const unsigned char* row = a.logits + r * a.stride_bytes;
  Slice<DT, NC, BLOCK> s;
  s.template load<PAST != 0>(row, a.V, 0, Cut{1, whole, NC});
  float z = kNegInf;
  if (threadIdx.x < kWave) {   // the row is on its way
    if (valid_id(a, id) >= 0) z = load_elem<DT>(row, id);
    entries[threadIdx.x] = entries_of(a, id, t);
  }
  if (a.tail) s.leave_out(a.V, valid_id(a, id), left_out);
  float off;
  const float m = s.largest([](int, float) {});
  const Sums mine = s.template sums<false>(a.V, m, a.c, off);
  if (threadIdx.x < kWave) entries[threadIdx.x].z = z;   // it came last
  const Sums other = join_block<BLOCK / kWave>(mine, a.c, off, each);
  if (!out) {
    if (threadIdx.x < kWave) {
      const Entries& e = entries[threadIdx.x];
      put_loss(a, r, weight, e, row_sums(a, e, other));
    }
    return;
  }
  if (threadIdx.x < kWave) {
    const Entries& e = entries[threadIdx.x];
    const RowSums sums = row_sums(a, e, other);
    const RowGrad g = row_grad_of(a, weight, e, sums);
    own[threadIdx.x] = g.entry;
    if (threadIdx.x == 0) {
      row_grad.sums = sums;
      row_grad.M = g.M;
      row_grad.A = g.A;
    }
  }
  __syncthreads();
  const GradRow p(row_grad.M, a.c, row_grad.A, 0.0);
  const Pass pass;
  const auto put = [&](auto&& of) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      if (!s.has(j)) continue;
      float v[EPC];
      pass.unpack<DT>(s.c[j], v);
#pragma unroll
      for (int i = 0; i < EPC; ++i) v[i] = of(v[i]);
      unsigned char* base = out + j * BLOCK * 16;   // uniform
      if (j * BLOCK + (int)threadIdx.x < whole)
        store16<PAST == 2>(base + threadIdx.x * 16u, pack<DT>(v));
      sched_fence();
    }
  };
  if (p.plain)
    put([&](float x) { return p.of<true, true>(x); });
  else
    put([&](float x) { return p.of<false, false>(x); });
  if ((int)threadIdx.x < a.V - whole * EPC)
    store_elem<DT>(out, whole * EPC + (int)threadIdx.x,
                   p.at(load_elem<DT>(row, whole * EPC + (int)threadIdx.x)));
  // the loss, while the others store
  if (threadIdx.x < kWave) put_loss(a, r, weight, entries[threadIdx.x], row_grad.sums);
  __syncthreads();   // the entries' own values over what was put there
  if (threadIdx.x < kWave && entries[threadIdx.x].first)
    store_elem<DT>(out, entries[threadIdx.x].id, own[threadIdx.x]);
}

// ------------------------------------------------------------ wider rows
// Workspace: the sums of each slice, what the gradient takes of each row, and each
// entry's gradient (k to a row).
struct DtRow {
  double A;
  float M;
  float weight;
};
struct DtWs {
  Sums* sums;      // [rows][slices]
  DtRow* rows;     // [rows]
  float* entry;    // [rows][k]
};

template <int DT, int NC>
__global__ __launch_bounds__(kSliceBlock) void distill_slice_kernel(DistillArgs a, Cut cut,
                                                                    DtWs ws) {
  __shared__ Sums each[kSliceWaves];
  __shared__ typename Slice<DT, NC>::LeftOut left_out;
  const int slice = blockIdx.x % cut.slices;
  const long long r = blockIdx.x / cut.slices;
  if (a.weight && a.weight[r] == 0.0f) return;
  const int id = a.tail ? valid_id(a, raw_id(a, r)) : -1;
  Slice<DT, NC> s;
  s.template load<false>(a.logits + r * a.stride_bytes, a.V, slice, cut);
  if (a.tail) s.leave_out(a.V, id, left_out);
  float off;
  const float m = s.largest([](int, float) {});
  const Sums mine = s.template sums<false>(a.V, m, a.c, off);
  const Sums all = join_block<kSliceWaves>(mine, a.c, off, each);
  if (threadIdx.x == 0) ws.sums[r * cut.slices + slice] = all;
}

// Row r's entries and the sums of its slices, by one wavefront.
template <int DT>
__device__ __forceinline__ RowSums join_row(const DistillArgs& a, long long r, const Sums* sums,
                                            int slices, Entries& e) {
  const int id = raw_id(a, r);
  const float t = teacher_of(a, r);
  const float z =
      valid_id(a, id) >= 0 ? load_elem<DT>(a.logits + r * a.stride_bytes, id) : kNegInf;
  const Sums other = join_slices(sums, slices, a.c);
  e = entries_of(a, id, t);
  e.z = z;
  return row_sums(a, e, other);
}

// One wavefront to a row.
template <int DT>
__global__ __launch_bounds__(kSliceBlock) void distill_join_kernel(DistillArgs a, int slices,
                                                                   DtWs ws) {
  const long long r = (long long)blockIdx.x * kSliceWaves + threadIdx.x / kWave;
  if (r >= a.rows) return;
  const int lane = __lane_id();
  const float weight = a.weight ? a.weight[r] : 1.0f;
  if (weight == 0.0f) {
    if (lane == 0) {
      put_nothing(a, r);
      ws.rows[r].weight = 0.0f;
    }
    return;
  }
  Entries e;
  const RowSums sums = join_row<DT>(a, r, ws.sums + r * slices, slices, e);
  put_loss(a, r, weight, e, sums);
  const RowGrad g = row_grad_of(a, weight, e, sums);
  if (lane == 0) ws.rows[r] = DtRow{g.A, g.M, weight};
  if (lane < a.k) ws.entry[r * a.k + lane] = g.entry;
}

// One workgroup to a tile of a row, the last rows first: they are what the caches still
// hold of the pass before. ONCE: written past the caches. JOIN: with the row's join in each
// of its tiles (where there are few, that takes less than a launch of its own).
template <int DT, bool ONCE, bool JOIN>
__global__ __launch_bounds__(kSliceBlock) void distill_grad_kernel(DistillArgs a, int tiles,
                                                                   int slices, DtWs ws) {
  __shared__ DtRow joined;
  const int tile = blockIdx.x % tiles, lane = __lane_id();
  const long long r = a.rows - 1 - (long long)(blockIdx.x / tiles);
  unsigned char* out = a.grad + r * a.grad_stride_bytes;
  float own = 0.0f;   // the entry's gradient, in the first wavefront
  DtRow d;
  if constexpr (JOIN) {
    d.weight = a.weight ? a.weight[r] : 1.0f;
    if (d.weight != 0.0f) {
      if (threadIdx.x < kWave) {
        Entries e;
        const RowSums sums = join_row<DT>(a, r, ws.sums + r * slices, slices, e);
        const RowGrad g = row_grad_of(a, d.weight, e, sums);
        own = g.entry;
        if (lane == 0) joined = DtRow{g.A, g.M, d.weight};
        if (tile == 0) put_loss(a, r, d.weight, e, sums);
      }
      __syncthreads();
      d = joined;
    } else if (tile == 0 && threadIdx.x == 0) {
      put_nothing(a, r);
    }
  } else {
    d = ws.rows[r];
    if (lane < a.k && d.weight != 0.0f) own = ws.entry[r * a.k + lane];
  }
  if (d.weight == 0.0f) {
    zero_tile<DT>(out, a.V, tile);
    return;
  }
  const int id = valid_id(a, raw_id(a, r));
  const unsigned char* row = a.logits + r * a.stride_bytes;
  put_tile<DT, false, ONCE>(row, out, a.V, tile, GradRow(d.M, a.c, d.A, 0.0));
  const bool here = id >= 0 && id / kTileIds<DT> == tile;
  if (!__any(here)) return;   // the same for all of the workgroup
  __syncthreads();
  // an id that comes twice has the same value with each
  if (threadIdx.x < kWave && here) store_elem<DT>(out, id, own);
}

// Rows of up to this many chunks take one workgroup each, and are read once.
constexpr int kHalfBlock = 512, kRowBlock = 1024;
constexpr int kRowChunks = 20 * kRowBlock;

// How rows are cut; one slice: not at all (us, calls back to back).
//  - Up to 4096 chunks: one workgroup of 256 threads and one launch. 1 x 8192 bf16 9.5, in
//    slices and tiles 12.5; 64 x 8192 9.7 against 18.5, 64 x 32000 11.3 against 12.0.
//  - Up to 20480 chunks from 128 rows on: one workgroup of 512 or 1024 threads. 128 x 128256
//    bf16 20.8 against 22.4 in slices, 256 rows 24.7 against 39.5; but 64 rows 19.4 against
//    15.2 and 1 row 16.5 against 11.9.
//  - Else slices: as many as give a thousand workgroups, at least what holds the row.
Cut dt_cut(int dtype, int rows, int vocab) {
  const int whole = vocab / (dtype == 0 ? 4 : 8);
  if (whole <= kMaxSliceChunks) return cut_of(whole, 1);
  if (whole <= kRowChunks && rows >= 128) {
    const int block = whole <= 16 * kHalfBlock ? kHalfBlock : kRowBlock;
    return Cut{1, whole, (whole + block - 1) / block, block};
  }
  const int want = std::min({1024 / max(rows, 1), 64, (whole + kSliceBlock - 1) / kSliceBlock});
  return cut_of(whole, want);
}

// Batches of more bytes than this, logits and gradient together, are read past the caches,
// which could not keep them: 1024 x 128256 bf16 105 us against 128, 1022 x 64000 50 against
// 58. (Slices are read from the caches again, and it is their gradient that is written
// past them: 512 x 128256 fp32 128 us against 157, with a reader of the gradient behind it
// 207 against 220.)
constexpr long long kOnceBytes = 192ll << 20;

// Chunks a thread, as few as hold the row: those past it are skipped, but take registers. Kernel
// us, 1024 rows bf16: 96000 ids 74.0 with 12, 76.3 with 16; 128256 ids 93.9 with 16, 95.8 with
// 20; 48000 ids, 512 threads, 35.1 with 12 and with 16.
// Without a gradient rows are read through the caches: 1024 x 151936 65 us a call (4.8 TB/s), with
// a tail 71.
template <int DT, int PAST>
void launch_rows(const DistillArgs& a, const Cut& cut, hipStream_t s) {
  const auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(a.rows), dim3(cut.block), 0, s, a);
  };
  if (cut.block == kSliceBlock) {
    if (cut.nc == 1) return launch(distill_row_kernel<DT, 1, kSliceBlock, 0>);
    if (cut.nc == 2) return launch(distill_row_kernel<DT, 2, kSliceBlock, 0>);
    if (cut.nc == 4) return launch(distill_row_kernel<DT, 4, kSliceBlock, 0>);
    if (cut.nc == 8) return launch(distill_row_kernel<DT, 8, kSliceBlock, PAST>);
    return launch(distill_row_kernel<DT, 16, kSliceBlock, PAST>);
  }
  if (cut.block == kHalfBlock) {
    if (cut.nc <= 12) return launch(distill_row_kernel<DT, 12, kHalfBlock, PAST>);
    return launch(distill_row_kernel<DT, 16, kHalfBlock, PAST>);
  }
  if (cut.nc <= 12) return launch(distill_row_kernel<DT, 12, kRowBlock, PAST>);
  if (cut.nc <= 16) return launch(distill_row_kernel<DT, 16, kRowBlock, PAST>);
  launch(distill_row_kernel<DT, 20, kRowBlock, PAST>);
}

template <int DT>
void launch_slices(const DistillArgs& a, const Cut& cut, const DtWs& ws, hipStream_t s) {
  const dim3 grid((unsigned)a.rows * (unsigned)cut.slices), block(kSliceBlock);
  switch (cut.nc) {
    case 1: hipLaunchKernelGGL((distill_slice_kernel<DT, 1>), grid, block, 0, s, a, cut, ws); break;
    case 2: hipLaunchKernelGGL((distill_slice_kernel<DT, 2>), grid, block, 0, s, a, cut, ws); break;
    case 4: hipLaunchKernelGGL((distill_slice_kernel<DT, 4>), grid, block, 0, s, a, cut, ws); break;
    case 8: hipLaunchKernelGGL((distill_slice_kernel<DT, 8>), grid, block, 0, s, a, cut, ws); break;
    default: hipLaunchKernelGGL((distill_slice_kernel<DT, 16>), grid, block, 0, s, a, cut, ws);
  }
}

// Batches of up to this many tiles join their rows in each.
constexpr int kJoinTiles = 4096;

// Rows whose slices and tiles a batch holds: 2^23 workgroups of a launch at most.
int dt_batch(const Cut& cut, int rows, int tiles) {
  return std::min(batch_of(cut, rows), max(1, (1 << 23) / tiles));
}

template <int DT>
hipError_t launch_dt(const DistillArgs& all, void* workspace, hipStream_t s) {
  const Cut cut = dt_cut(DT, all.rows, all.V);
  const long long bytes = 2ll * all.rows * all.V * Fmt<DT>::ESZ;
  if (cut.slices == 1) {
    if (all.grad && bytes > 2 * kGradOnceBytes)
      launch_rows<DT, 2>(all, cut, s);
    else if (all.grad && bytes > kOnceBytes)
      launch_rows<DT, 1>(all, cut, s);
    else
      launch_rows<DT, 0>(all, cut, s);
    return hipGetLastError();
  }
  const int tiles = tiles_of<DT>(all.V), batch = dt_batch(cut, all.rows, tiles);
  for (int r0 = 0; r0 < all.rows; r0 += batch) {
    DistillArgs a = all;
    a.rows = min(batch, all.rows - r0);
    a.logits += (long long)r0 * a.stride_bytes;
    a.ids += (long long)r0 * a.k;
    a.teacher += (long long)r0 * a.k;
    if (a.weight) a.weight += r0;
    a.loss += r0;
    if (a.grad) a.grad += (long long)r0 * a.grad_stride_bytes;
    if (a.status) a.status += r0;
    DtWs ws;
    ws.sums = static_cast<Sums*>(workspace);
    ws.rows = reinterpret_cast<DtRow*>(ws.sums + (long long)a.rows * cut.slices);
    ws.entry = reinterpret_cast<float*>(ws.rows + a.rows);
    launch_slices<DT>(a, cut, ws, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 block(kSliceBlock);
    const bool join = a.grad && (long long)a.rows * tiles <= kJoinTiles;
    if (!join) {
      hipLaunchKernelGGL((distill_join_kernel<DT>),
                         dim3((a.rows + kSliceWaves - 1) / kSliceWaves), block, 0, s, a, cut.slices,
                         ws);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
      if (!a.grad) continue;
    }
    const auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(a.rows * tiles), block, 0, s, a, tiles, cut.slices, ws);
    };
    if (join)
      launch(distill_grad_kernel<DT, false, true>);
    else if (bytes > kOnceBytes)
      launch(distill_grad_kernel<DT, true, false>);
    else
      launch(distill_grad_kernel<DT, false, false>);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t distill_ws_bytes(int dtype, int rows, int vocab, int) {
  const Cut cut = dt_cut(dtype, rows, vocab);
  if (cut.slices == 1) return 0;
  const int batch = dt_batch(cut, rows, dtype == 0 ? tiles_of<0>(vocab) : tiles_of<1>(vocab));
  return (size_t)batch * (cut.slices * sizeof(Sums) + sizeof(DtRow) + kMaxTop * sizeof(float));
}

hipError_t launch_distill(const DistillArgs& a, int dtype, void* ws, hipStream_t s) {
  return dtype == 0 ? launch_dt<0>(a, ws, s) : launch_dt<1>(a, ws, s);
}

}  // namespace tsr
