// The 8-bit output projection (int8_logits): out[r][n] = sum_k x[r][k] w[n][k]
// in 32-bit integers, times the row's and the channel's scale.
//
// Few rows are bound by the weight's bytes: 1 x 128256 x 4096 79 us, 6.7 TB/s of
// the 6.9 that reads reach here; 64 x 128256 104 us, 5.2 TB/s, its logits' 16 MB
// among them. Many are bound by the matrix pipes and by the LDS that feeds them:
// 1024 x 151936 x 4096 513 us, 2.49 P op/s (its two launches traced alone 500 and
// 31), the pipes busy two thirds of it (products of random codes alone reach 3.8,
// where the card's power holds its clock); a stage of a 256 x 256 tile takes 1536
// cycles of LDS reads and 512 of loads landing there beside 2048 of products.
// The weight is cut into runs of channels: every hidden row, or up to 320 of
// them, meets a run while it is in LDS. The tiles of one run share it through an
// L2; the hidden rows come to each of the eight anew with every round of tiles
// (909 MB fetched in the first launch of the 1024 rows, the weight 604 of them).
#pragma once

#include <cmath>
#include <type_traits>

#include "kernels.hpp"
#include "wide_mem.hpp"

namespace tsr {

typedef int v4i __attribute__((ext_vector_type(4)));

// 16 bytes per lane from byte at + k of a buffer to `p` + 16 lane in LDS. (The
// host pass of the compiler does not know the 16-byte form.) ONCE: bytes that
// no other workgroup reads are not kept in the caches.
template <bool ONCE>
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t buffer, int8_t* p, uint32_t at,
                                       int k) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer, (__attribute__((address_space(3))) void*)p, 16,
                                           (int)at, k, 0, ONCE ? 2 : 0);
#endif
}
// `bytes` bytes from p (0: every load of it is out of range, and reads nothing).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const int8_t* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(p), 0, (int)bytes, 0x00027000);
}
// Waits until at most N loads are on their way and every LDS access is done.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "count");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));
}

// Every wavefront of the workgroup, its LDS accesses done; stores and loads stay
// on their way.
__device__ __forceinline__ void meet() {
  wait_loads<63>();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  sched_fence();
}

// Tiles of BM hidden rows by BN channels. WM x WN wavefronts each hold MT x NT
// blocks of 16 x 16 sums.
//
// v_mfma_i32_16x16x64_i8: lane l gives row l % 16 of the first operand (here
// channels) and of the second (hidden rows), 16 bytes at (l / 16) * 16 of 64;
// it gets channels (l / 16) * 4 + 0..3 of hidden row l % 16. Block t of a
// wavefront takes channels (i / 4) * 4 NT + t * 4 + i % 4 (i < 16) of its
// 16 NT, so that a lane ends with 4 NT neighbouring channels of one row and
// four lanes write a whole line.
//
// A stage holds TK bytes of each of the tile's rows in LDS, as 16-byte chunks;
// chunk c of row r lies at place c ^ turn(r), so that the 16 lanes which read
// one chunk of 16 rows take every bank in turn.
template <int BM, int BN, int WM, int WN, int TK>
struct Tile {
  static constexpr int WAVES = WM * WN, THREADS = WAVES * kWave;
  static constexpr int MT = BM / (16 * WM), NT = BN / (16 * WN);
  static constexpr int CH = TK / 16, PR = 64 / CH;   // chunks of a row, rows of a 1 KiB piece
  static constexpr int XI = BM / PR / WAVES, WI = BN / PR / WAVES;   // pieces per wavefront
  static constexpr int H = TK / 64;                                  // products along a stage
  static_assert(TK == 128 || TK == 256, "turns");
  static_assert(XI * PR * WAVES == BM && WI * PR * WAVES == BN, "pieces");
  static_assert(MT * 16 * WM == BM && NT * 16 * WN == BN, "blocks");

  int m0, n0;               // the tile's first row and channel
  int lane, wave, wm, wn;   // wm, wn: this wavefront's place in the tile

  // Workgroups go round the eight XCDs: each XCD gets a run of tiles, the rows'
  // tiles of one run of channels next to each other (they share its L2).
  __device__ __forceinline__ bool place(int m_tiles, int tiles) {
    const int tile = (blockIdx.x & 7) * ((tiles + 7) / 8) + (blockIdx.x >> 3);
    m0 = (tile % m_tiles) * BM;
    n0 = (tile / m_tiles) * BN;
    lane = threadIdx.x & (kWave - 1);
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    wm = wave % WM;
    wn = wave / WM;
    return tile < tiles;
  }
  static __device__ __forceinline__ int turn(int r) { return r & (CH - 1); }
  // piece q of this wavefront: the row its lane brings, and which bytes of it
  __device__ __forceinline__ int row_of(int q, int pieces) const {
    return (wave * pieces + q) * PR + lane / CH;
  }
  __device__ __forceinline__ int byte_of(int r) const { return ((lane % CH) ^ turn(r)) * 16; }
  static __device__ __forceinline__ int channel_of(int r) {
    const int i = r & 15, t = (r % (16 * NT)) / 16;
    return r / (16 * NT) * (16 * NT) + (i >> 2) * (4 * NT) + t * 4 + (i & 3);
  }
  // byte offsets of the pieces from the tile's first row; rows past the last
  // one repeat it (their sums are not stored)
  template <class T>
  __device__ __forceinline__ void offsets(const Int8Args& a, T* xo, T* wo) const {
#pragma unroll
    for (int q = 0; q < XI; ++q) {
      const int r = row_of(q, XI);
      xo[q] = (T)min(r, a.rows - 1 - m0) * (T)a.x_stride + (T)byte_of(r);
    }
#pragma unroll
    for (int q = 0; q < WI; ++q) {
      const int r = row_of(q, WI);
      wo[q] = (T)min(channel_of(r), a.vocab - 1 - n0) * (T)a.w_stride + (T)byte_of(r);
    }
  }
  // a partial stage from byte k of the rows on, zero behind their end
  template <class T>
  __device__ __forceinline__ void fetch_partial(const Int8Args& a, const int8_t* xb,
                                                const int8_t* wb, const T* xo, const T* wo, int k,
                                                int8_t* xs, int8_t* ws) const {
    uint4 v[XI + WI];
#pragma unroll
    for (int q = 0; q < XI; ++q) {
      const int c = byte_of(row_of(q, XI));
      v[q] = load_bytes_zero(xb + (xo[q] - (T)c), k + c, a.width);
    }
#pragma unroll
    for (int q = 0; q < WI; ++q) {
      const int c = byte_of(row_of(q, WI));
      v[XI + q] = load_bytes_zero(wb + (wo[q] - (T)c), k + c, a.width);
    }
    place_pieces(v, v + XI, xs, ws);
  }
  __device__ __forceinline__ void place_pieces(const uint4* x, const uint4* w, int8_t* xs,
                                               int8_t* ws) const {
#pragma unroll
    for (int q = 0; q < XI; ++q)
      *reinterpret_cast<uint4*>(xs + (wave * XI + q) * 1024 + lane * 16) = x[q];
#pragma unroll
    for (int q = 0; q < WI; ++q)
      *reinterpret_cast<uint4*>(ws + (wave * WI + q) * 1024 + lane * 16) = w[q];
  }
  // operand q of the NT + MT that product h of a stage takes
  __device__ __forceinline__ void read(int q, const int8_t* xs, const int8_t* ws, int h, v4i* w,
                                       v4i* x) const {
    const int i = lane & 15;
    const int at = i * TK + (((h * 4 + (lane >> 4)) ^ turn(i)) * 16);
    if (q < NT)
      w[q < NT ? q : 0] = *reinterpret_cast<const v4i*>(ws + (wn * NT + q) * 16 * TK + at);
    else
      x[q < NT ? 0 : q - NT] =
          *reinterpret_cast<const v4i*>(xs + (wm * MT + q - NT) * 16 * TK + at);
  }
  static __device__ __forceinline__ void clear(v4i (*acc)[MT]) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int u = 0; u < MT; ++u) acc[t][u] = v4i{0, 0, 0, 0};
  }
  static __device__ __forceinline__ void multiply_row(v4i (*acc)[MT], int u, const v4i* w,
                                                      const v4i* x) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
      acc[t][u] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[t], x[u], acc[t][u], 0, 0, 0);
  }
  __device__ __forceinline__ void multiply_stage(v4i (*acc)[MT], const int8_t* xs,
                                                 const int8_t* ws) const {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      v4i w[NT], x[MT];
#pragma unroll
      for (int q = 0; q < NT + MT; ++q) read(q, xs, ws, h, w, x);
#pragma unroll
      for (int u = 0; u < MT; ++u) multiply_row(acc, u, w, x);
      sched_fence();
    }
  }
  // What the sums of this lane are multiplied with and added to. Read before the
  // products where registers allow, for a tile's end waits for it otherwise.
  static constexpr bool EARLY = MT * NT <= 24;
  struct Scales {
    float w[4 * NT], b[4 * NT], x[MT];
  };
  __device__ __forceinline__ void load_scales(const Int8Args& a, Scales* s) const {
    const int c0 = n0 + wn * (16 * NT) + (lane >> 4) * (4 * NT);
#pragma unroll
    for (int e = 0; e < 4 * NT; ++e) {
      const int c = min(c0 + e, a.vocab - 1);
      s->w[e] = a.w_scale[c];
      s->b[e] = a.bias ? a.bias[c] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < MT; ++u)
      s->x[u] = a.x_scale[min(m0 + (wm * MT + u) * 16 + (lane & 15), a.rows - 1)];
  }
  // The sum rounded to float32, times the row's scale, then times the channel's
  // and plus the bias in one rounding; float32 holds far more than the codes do.
  //
  // The results pass through LDS (`even` and `odd` in turn, each as large as a
  // stage of the larger operand), so that a row's run of channels leaves in whole
  // lines: from the sums' own lanes, in pieces of 16 to 64 bytes, 64 x 128256 took
  // 110 us (105 so) and 1000 x 50001, whose rows end inside lines, 247 (221).
  // Chunk c of LDS row r lies at place c ^ (r & 7).
  template <int DT>
  __device__ __forceinline__ void store(const Int8Args& a, const v4i (*acc)[MT], Scales& s,
                                        int8_t* even, int8_t* odd) const {
    constexpr int ESZ = Fmt<DT>::ESZ, EPC = Fmt<DT>::EPC, ROW = BN * ESZ, CB = ROW / 16;
    constexpr int FIT = (BM > BN ? BM : BN) * TK / (16 * WM * ROW);
    constexpr int UP = FIT < MT ? FIT : MT;   // blocks of rows a pass
    constexpr int RP = 16 * WM * UP;          // rows a pass
    static_assert(UP >= 1 && CB >= 8, "a pass fits a stage");
    const int i = lane & 15, cw = wn * (16 * NT) + (lane >> 4) * (4 * NT);
    if constexpr (!EARLY) load_scales(a, &s);
    const bool whole_lines =
        (((uintptr_t)a.out | (uintptr_t)a.out_stride_bytes) & 127) == 0;
    meet();   // every wavefront has read its last stage
#pragma unroll
    for (int p = 0; p < MT; p += UP) {
      int8_t* buf = (p / UP) % 2 ? odd : even;
#pragma unroll
      for (int u = 0; u < UP && p + u < MT; ++u) {
        const int lr = (wm * UP + u) * 16 + i;
        uint32_t w[4 * NT * ESZ / 4];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = fmaf((float)acc[t][p + u][e] * s.x[p + u], s.w[t * 4 + e], s.b[t * 4 + e]);
          if constexpr (DT == 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[t * 4 + e] = __float_as_uint(v[e]);
          } else {
            w[t * 2] = bf16_pair(v[0], v[1]);
            w[t * 2 + 1] = bf16_pair(v[2], v[3]);
          }
        }
        constexpr int N = 4 * NT * ESZ < 16 ? 2 : 4;   // words a write
#pragma unroll
        for (int k = 0; k < 4 * NT * ESZ / 4; k += N) {
          const int at = cw * ESZ + k * 4;
          int8_t* o = buf + lr * ROW + ((at / 16) ^ (lr & 7)) * 16 + at % 16;
          if constexpr (N == 4)
            *reinterpret_cast<uint4*>(o) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
          else
            *reinterpret_cast<uint2*>(o) = make_uint2(w[k], w[k + 1]);
        }
      }
      meet();
#pragma unroll
      for (int q = 0; q < (RP * CB + THREADS - 1) / THREADS; ++q) {
        const int n = q * THREADS + threadIdx.x;
        if (RP * CB % THREADS != 0 && n >= RP * CB) break;
        const int lr = n / CB, c = n % CB;
        const int u = p + lr / 16 % UP;
        const int r = m0 + (lr / (16 * UP) * MT + u) * 16 + lr % 16;
        if (u >= MT || r >= a.rows) continue;
        const uint4 v = *reinterpret_cast<const uint4*>(buf + lr * ROW + (c ^ (lr & 7)) * 16);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        const int e0 = n0 + c * EPC;
        unsigned char* o = a.out + (long long)r * a.out_stride_bytes + (long long)e0 * ESZ;
        if (e0 + EPC <= a.vocab) {
          // whole lines of many rows' logits leave the caches before they are read:
          // 256 x 128256 150 us kept in them, 139 not, 1024 x 151936 519 and 511 (24
          // rows 84 and 90; lines that two tiles share, 256 x 50001 x 4095: 122 and
          // 180). With the sampler behind, which reads them: 128 x 128256 159 and
          // 154, 256 x 128256 183 and 174, 1024 x 128256 506 and 508, but 256 x
          // 32000 65 and 66, 320 x 32000 fp32 79 and 82.
          if (BM >= 128 && whole_lines)
            store16_once(o, v);
          else
            store_words<4>(o, w);
        } else {
#pragma unroll
          for (int e = 0; e < EPC; ++e) {
            if (e0 + e >= a.vocab) break;
            if constexpr (DT == 0)
              reinterpret_cast<uint32_t*>(o)[e] = w[e];
            else
              reinterpret_cast<uint16_t*>(o)[e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
          }
        }
      }
    }
  }
};

// Operands whose rows start at 4-byte words: loads go straight to LDS, XR stages
// of the hidden rows and WR of the weight deep. The hidden rows are in the caches,
// the weight comes from memory: where LDS does not hold three stages of both, it
// holds two and three (1024 x 131072 x 4096 in 256 x 256: two and two 463 us, two
// and three 432; with the weight in the caches 413, without loads 294). The loads
// for later lie between the products, so that a wavefront's matrix pipe does not
// wait while they are issued.
template <int DT, int BM, int BN, int WM, int WN, int TK, int XR, int WR, bool ONCE>
__global__ __launch_bounds__(WM* WN* kWave, 1) void int8_ring_kernel(Int8Args a, int m_tiles,
                                                                     int tiles) {
  using T = Tile<BM, BN, WM, WN, TK>;
  constexpr int MT = T::MT, NT = T::NT, XI = T::XI, WI = T::WI, H = T::H, DMAS = XI + WI;
  constexpr int AHEAD = WR - XR, TURN = AHEAD == 0 ? XR : XR * WR;   // stages of a turn of both
  static_assert(XR >= 2 && XR <= 4 && (AHEAD == 0 || (XR == 2 && WR == 3)), "ring");
  static_assert((TURN * H) % 2 == 0, "ring");
  // one object per operand and stage: only so are loads into one stage known
  // not to meet reads of another
  __shared__ __attribute__((aligned(1024))) int8_t x0[BM * TK];
  __shared__ __attribute__((aligned(1024))) int8_t w0[BN * TK];
  __shared__ __attribute__((aligned(1024))) int8_t x1[BM * TK];
  __shared__ __attribute__((aligned(1024))) int8_t w1[BN * TK];
  __shared__ __attribute__((aligned(1024))) int8_t x2[XR > 2 ? BM * TK : 16];
  __shared__ __attribute__((aligned(1024))) int8_t w2[WR > 2 ? BN * TK : 16];
  __shared__ __attribute__((aligned(1024))) int8_t x3[XR > 3 ? BM * TK : 16];
  __shared__ __attribute__((aligned(1024))) int8_t w3[WR > 3 ? BN * TK : 16];
  auto x_of = [&](int b) { return b % XR == 0 ? x0 : b % XR == 1 ? x1 : b % XR == 2 ? x2 : x3; };
  auto w_of = [&](int b) { return b % WR == 0 ? w0 : b % WR == 1 ? w1 : b % WR == 2 ? w2 : w3; };
  T t;
  if (!t.place(m_tiles, tiles)) return;
  typename T::Scales scales;
  if constexpr (T::EARLY) t.load_scales(a, &scales);
  const int8_t* xb = a.x + (long long)t.m0 * a.x_stride;
  const int8_t* wb = a.w + (long long)t.n0 * a.w_stride;
  // the tile's bytes end with the last byte of its last row
  const uint32_t xn = (uint32_t)(min(BM, a.rows - t.m0) - 1) * (uint32_t)a.x_stride + a.width;
  const uint32_t wn = (uint32_t)(min(BN, a.vocab - t.n0) - 1) * (uint32_t)a.w_stride + a.width;
  uint32_t xo[XI], wo[WI];
  t.offsets(a, xo, wo);
  v4i acc[NT][MT];
  T::clear(acc);

  const int stages = a.width / TK;
  // piece q of the hidden rows' stage b and of the weight's stage b + AHEAD; past
  // the last stage it reads nothing, and is counted by the waits all the same
  auto fetch_piece = [&](int q, int b, int8_t* xs, int8_t* ws) {
    const int k = q < XI ? b : b + AHEAD;
    const bool in = k < stages;
    if (q < XI)
      to_lds<false>(buffer_of(xb, in ? xn : 0), xs + (t.wave * XI + q) * 1024,
                    xo[q < XI ? q : 0], in ? k * TK : 0);
    else
      to_lds<ONCE>(buffer_of(wb, in ? wn : 0), ws + (t.wave * WI + q - XI) * 1024,
                   wo[q < XI ? 0 : q - XI], in ? k * TK : 0);
  };
  auto fetch = [&](int q0, int b, int8_t* xs, int8_t* ws) {
#pragma unroll
    for (int q = q0; q < DMAS; ++q) fetch_piece(q, b, xs, ws);
  };
  if constexpr (AHEAD > 0) fetch(XI, -1, nullptr, w0);   // the weight's first stage
  fetch(0, 0, x0, w_of(AHEAD));
  if constexpr (XR > 2) fetch(0, 1, x1, w1);
  if constexpr (XR > 3) fetch(0, 2, x2, w2);
  int8_t* const xl = x_of(XR - 1);
  int8_t* const wl = w_of(WR - 1);
  if (stages * TK < a.width) {
    // a partial stage goes through registers, beside the first whole ones' loads
    t.fetch_partial(a, xb, wb, xo, wo, stages * TK, xl, wl);
    __syncthreads();
    t.multiply_stage(acc, xl, wl);
    __syncthreads();
  }
  if (stages > 0) {
    fetch(0, XR - 1, xl, wl);
    constexpr int LATER = AHEAD > 0 ? WI : 0;   // the weight's last pieces are for later
    wait_loads<DMAS*(XR - 1) + LATER>();
    __builtin_amdgcn_s_barrier();
    sched_fence();
    v4i wv[2][NT], xv[2][MT];
#pragma unroll
    for (int q = 0; q < NT + MT; ++q) t.read(q, x0, w0, 0, wv[0], xv[0]);
    // Stage b = J of a turn of the rings. Its last product meets the next stage,
    // which has landed for every wavefront behind the barrier; so has everyone's
    // reading of this one, whose places take the stages b + XR and b + WR.
    auto stage = [&](auto j, auto more, int b) {
      constexpr int J = decltype(j)::value, F = J * H;
      constexpr bool MORE = decltype(more)::value;
      constexpr bool LAST = !MORE && J + 1 == XR;   // no stage follows
      int8_t *xs = x_of(J), *ws = w_of(J), *xnext = x_of(J + 1), *wnext = w_of(J + 1);
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const bool to_next = h + 1 == H;
        if (to_next && !LAST) {
          wait_loads<DMAS*(MORE ? XR - 2 : J + 2 < XR ? XR - 2 - J : 0) + LATER>();
          __builtin_amdgcn_s_barrier();
          sched_fence();
        }
#pragma unroll
        for (int u = 0; u < MT; ++u) {
          if (!to_next || !LAST) {
#pragma unroll
            for (int q = u * (NT + MT) / MT; q < (u + 1) * (NT + MT) / MT; ++q) {
              if (to_next)
                t.read(q, xnext, wnext, 0, wv[(F + h + 1) & 1], xv[(F + h + 1) & 1]);
              else
                t.read(q, xs, ws, h + 1, wv[(F + h + 1) & 1], xv[(F + h + 1) & 1]);
            }
          }
          if (MORE && to_next) {
#pragma unroll
            for (int q = u * DMAS / MT; q < (u + 1) * DMAS / MT; ++q)
              fetch_piece(q, b + XR, xs, ws);
          }
          T::multiply_row(acc, u, wv[(F + h) & 1], xv[(F + h) & 1]);
          sched_fence();
        }
      }
    };
    constexpr std::integral_constant<int, 0> j0{};
    constexpr std::integral_constant<int, 1> j1{};
    constexpr std::integral_constant<int, 2> j2{};
    constexpr std::integral_constant<int, 3> j3{};
    constexpr std::integral_constant<int, 4> j4{};
    constexpr std::integral_constant<int, 5> j5{};
    constexpr std::true_type more{};
    constexpr std::false_type no_more{};
    int b = 0;
    if constexpr (AHEAD > 0) {   // every stage as if more followed
      for (; b + TURN <= stages; b += TURN) {
        stage(j0, more, b);
        stage(j1, more, b + 1);
        stage(j2, more, b + 2);
        stage(j3, more, b + 3);
        stage(j4, more, b + 4);
        stage(j5, more, b + 5);
      }
      if (b < stages) stage(j0, more, b);
      if (b + 1 < stages) stage(j1, more, b + 1);
      if (b + 2 < stages) stage(j2, more, b + 2);
      if (b + 3 < stages) stage(j3, more, b + 3);
      if (b + 4 < stages) stage(j4, more, b + 4);
    } else {
      for (; b + XR < stages; b += XR) {
        stage(j0, more, b);
        stage(j1, more, b + 1);
        if constexpr (XR > 2) stage(j2, more, b + 2);
        if constexpr (XR > 3) stage(j3, more, b + 3);
      }
      // the last turn, of 1 to XR stages
      stage(j0, no_more, b);
      if (b + 1 < stages) {
        stage(j1, no_more, b + 1);
        if constexpr (XR > 2) {
          if (b + 2 < stages) {
            stage(j2, no_more, b + 2);
            if constexpr (XR > 3) {
              if (b + 3 < stages) stage(j3, no_more, b + 3);
            }
          }
        }
      }
    }
  }
  wait_loads<0>();   // LDS takes no more loads: the results pass through it
  t.template store<DT>(a, acc, scales, BM > BN ? x0 : w0, BM > BN ? x1 : w1);
}

// Operands at any byte: loads into registers, put into LDS once the stage
// before them is multiplied. A 16-byte load that does not start at a 4-byte word
// runs at a third of the rate (2.0 against 5.0 TB/s from the caches), so a lane
// loads the four words from the one that holds its first byte on, takes the
// fifth from the next lane (the last lane of a row loads it), and shifts.
template <int DT, int BM, int BN, int WM, int WN, int TK>
__global__ __launch_bounds__(WM* WN* kWave) void int8_tile_kernel(Int8Args a, int m_tiles,
                                                                  int tiles) {
  using T = Tile<BM, BN, WM, WN, TK>;
  constexpr int XI = T::XI, WI = T::WI, N = XI + WI;
  __shared__ __attribute__((aligned(1024))) int8_t x0[BM * TK];
  __shared__ __attribute__((aligned(1024))) int8_t x1[BM * TK];
  __shared__ __attribute__((aligned(1024))) int8_t w0[BN * TK];
  __shared__ __attribute__((aligned(1024))) int8_t w1[BN * TK];
  T t;
  if (!t.place(m_tiles, tiles)) return;
  typename T::Scales scales;
  if constexpr (T::EARLY) t.load_scales(a, &scales);
  const int8_t* xb = a.x + (long long)t.m0 * a.x_stride;
  const int8_t* wb = a.w + (long long)t.n0 * a.w_stride;
  uint32_t off[N];
  t.offsets(a, off, off + XI);
  v4i acc[T::NT][T::MT];
  T::clear(acc);
  const int stages = a.width / TK;
  if (stages * TK < a.width) {   // a partial stage first
    t.fetch_partial(a, xb, wb, off, off + XI, stages * TK, x1, w1);
    __syncthreads();
    t.multiply_stage(acc, x1, w1);
  }

  // from here on lane c of a row's lanes brings chunk c
  const int c = t.lane % T::CH;
  const bool last = c == T::CH - 1;
  int at[N];       // where it goes in LDS
  uint32_t skew = 0;   // bytes of the first word before the chunk, 2 bits a piece
  static_assert(N <= 16, "pieces");
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const int r = q < XI ? t.row_of(q, XI) : t.row_of(q - XI, WI);
    off[q] = off[q] - t.byte_of(r) + c * 16;
    at[q] = r * TK + (c ^ T::turn(r)) * 16;
    const uint32_t s = ((uint32_t)(uintptr_t)(q < XI ? xb : wb) + off[q]) & 3;
    skew |= s << (2 * q);
  }
  uint4 v[N];
  uint32_t fifth[N];
  auto fetch = [&](int b) {
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const uint32_t s = (skew >> (2 * q)) & 3;
      const int8_t* p = (q < XI ? xb : wb) + (long long)b * TK + ((long long)off[q] - s);
      const Words4 w = *reinterpret_cast<const Words4*>(p);
      v[q] = make_uint4(w.x, w.y, w.z, w.w);
      fifth[q] = 0;
      if (last && s != 0) fifth[q] = *reinterpret_cast<const uint32_t*>(p + 16);
    }
  };
  auto put = [&](int8_t* xs, int8_t* ws) {
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const uint32_t s = (skew >> (2 * q)) & 3;
      const uint32_t next = dpp_u32<0x101 /* row_shl:1: the next lane's */>(v[q].x);
      const uint32_t e = last ? fifth[q] : next;
      *reinterpret_cast<uint4*>((q < XI ? xs : ws) + at[q]) =
          make_uint4(__builtin_amdgcn_alignbyte(v[q].y, v[q].x, s),
                     __builtin_amdgcn_alignbyte(v[q].z, v[q].y, s),
                     __builtin_amdgcn_alignbyte(v[q].w, v[q].z, s),
                     __builtin_amdgcn_alignbyte(e, v[q].w, s));
    }
  };
  if (stages > 0) {
    fetch(0);
    put(x0, w0);
    __syncthreads();
    int b = 0;
    for (; b + 2 < stages; b += 2) {
      fetch(b + 1);
      t.multiply_stage(acc, x0, w0);
      put(x1, w1);
      __syncthreads();
      fetch(b + 2);
      t.multiply_stage(acc, x1, w1);
      put(x0, w0);
      __syncthreads();
    }
    const bool two = b + 1 < stages;
    if (two) fetch(b + 1);
    t.multiply_stage(acc, x0, w0);
    if (two) {
      put(x1, w1);
      __syncthreads();
      t.multiply_stage(acc, x1, w1);
    }
  }
  t.template store<DT>(a, acc, scales, BM > BN ? x0 : w0, BM > BN ? x1 : w1);
}

template <int BM, int BN>
void tiles_of(const Int8Args& a, int* m_tiles, int* tiles) {
  *m_tiles = (a.rows + BM - 1) / BM;
  *tiles = *m_tiles * ((a.vocab + BN - 1) / BN);
}

template <int DT, int BM, int BN, int WM, int WN, int TK, int XR, int WR, bool ONCE>
hipError_t launch_ring(const Int8Args& a, hipStream_t s) {
  int m_tiles, tiles;
  tiles_of<BM, BN>(a, &m_tiles, &tiles);
  hipLaunchKernelGGL((int8_ring_kernel<DT, BM, BN, WM, WN, TK, XR, WR, ONCE>),
                     dim3((tiles + 7) / 8 * 8), dim3(WM * WN * kWave), 0, s, a, m_tiles, tiles);
  return hipGetLastError();
}

template <int DT, int BM, int BN, int WM, int WN, int TK>
hipError_t launch_tile(const Int8Args& a, hipStream_t s) {
  int m_tiles, tiles;
  tiles_of<BM, BN>(a, &m_tiles, &tiles);
  hipLaunchKernelGGL((int8_tile_kernel<DT, BM, BN, WM, WN, TK>), dim3((tiles + 7) / 8 * 8),
                     dim3(WM * WN * kWave), 0, s, a, m_tiles, tiles);
  return hipGetLastError();
}

// Tile shapes for more than 64 rows: how many run at once (one or two to a
// compute unit), how long a full round of them takes in us at width 4096 with the
// weight in the caches, and which share of that a round of few takes. Shapes that
// run in pairs keep that share up to half the places. Measured (us a round, many
// rounds and one of few tiles): 256x256 54 38, 192x256 42 33, 320x128 38 31,
// 128x256 34 26, 128x128 39 20, one to a compute unit 21 17, 64x64 16 10.
struct TileCost {
  int bm, bn, at_once;
  double us, least;
};
constexpr TileCost kTileCost[] = {{256, 256, 256, 54.0, 0.70}, {192, 256, 256, 42.5, 0.79},
                                  {320, 128, 256, 38.0, 0.82}, {128, 256, 256, 34.0, 0.77},
                                  {128, 128, 512, 39.0, 0.52}, {128, 128, 256, 21.5, 0.80},
                                  {64, 64, 512, 16.2, 0.64}};
constexpr int kTileShapes = sizeof(kTileCost) / sizeof(kTileCost[0]);
constexpr double kWeightBytesPerUs = 4.8e6;   // as the tiles read it from memory

inline long long tiles_in(const TileCost& c, int rows, int vocab) {
  return (long long)((rows + c.bm - 1) / c.bm) * ((vocab + c.bn - 1) / c.bn);
}
// The rounds' time and the weight's, which hide each other but for where they
// are alike (their fourth powers added).
inline double tiles_us(const TileCost& c, int rows, int vocab, int width) {
  const long long tiles = tiles_in(c, rows, vocab), rest = tiles % c.at_once;
  double part = 0.0;
  if (rest > 0) {
    double more = (double)rest / c.at_once;
    if (c.at_once == 512) more = more > 0.5 ? 2.0 * more - 1.0 : 0.0;
    part = c.least + (1.0 - c.least) * more;
  }
  const double r = ((double)(tiles / c.at_once) + part) * c.us * width / 4096.0;
  const double m = (double)vocab * width / kWeightBytesPerUs;
  return sqrt(sqrt(r * r * r * r + m * m * m * m));
}
// The shape with the least time. Measured at width 4096 (us), the shapes in the
// table's order: 256 x 32000 49 46 43 39 49 51 71, 320 x 32000 53 47 44 65 65 60 82,
// 384 x 32000 54 47 78 67 67 68 93, 128 x 128256 127 116 163 113 115 119 156,
// 200 x 8960 41 35 34 28 22 19 22, 90 x 8192 38 33 31 26 20 17 11, 1024 x 131072
// 431 509 602 542 624 702 1036.
inline int pick_tile(int rows, int vocab, int width) {
  int best = 0;
  for (int i = 1; i < kTileShapes; ++i)
    if (tiles_us(kTileCost[i], rows, vocab, width) < tiles_us(kTileCost[best], rows, vocab, width))
      best = i;
  return best;
}
// The whole batch in one launch, or the channels that fill whole rounds of a
// large shape first and the others in the shape that suits them, where that
// saves more than a launch's 3 us. `first`: the channels of the first launch.
struct TilePlan {
  int shape, first;
};
inline TilePlan plan_tiles(int rows, int vocab, int width) {
  TilePlan p{pick_tile(rows, vocab, width), vocab};
  double least = tiles_us(kTileCost[p.shape], rows, vocab, width);
  for (int i = 0; i < kTileShapes; ++i) {
    const TileCost& c = kTileCost[i];
    const long long full = tiles_in(c, rows, vocab) / c.at_once;
    const long long first = full * c.at_once / ((rows + c.bm - 1) / c.bm) * c.bn;
    if (first <= 0 || first >= vocab) continue;
    const int rest = vocab - (int)first;
    const double us =
        tiles_us(c, rows, (int)first, width) +
        tiles_us(kTileCost[pick_tile(rows, rest, width)], rows, rest, width) + 3.0;
    if (us < least) {
      p = TilePlan{i, (int)first};
      least = us;
    }
  }
  return p;
}

// ONCE where the weight's lines are whole (a line that two loads share would be
// read twice) and it is too large to be in the caches from the call before:
// 1 x 128256 x 4096 78 us against 93, with its rows 4100 apart 92 against 84,
// 60 x 8192 x 4096 18 against 15; hidden rows 4100 apart, at words only, 5 x 128256
// 79 against 92, 256 x 128256 132 against 140. Small tiles that share a weight leave it in the
// caches for each other (1024 x 131072 x 4096 in 128 x 128 656 us past them, 624
// in them; in 256 x 256 431 and 453).
constexpr long long kInt8OnceBytes = 48ll << 20;

template <int DT, bool ONCE>
hipError_t launch_shape(const Int8Args& a, int shape, hipStream_t s) {
  switch (shape) {
    case 0: return launch_ring<DT, 256, 256, 2, 4, 128, 2, 3, ONCE>(a, s);
    case 1: return launch_ring<DT, 192, 256, 2, 4, 128, 2, 3, ONCE>(a, s);
    case 2: return launch_ring<DT, 320, 128, 4, 2, 128, 2, 3, ONCE>(a, s);
    case 3: return launch_ring<DT, 128, 256, 2, 4, 128, 3, 3, ONCE>(a, s);
    case 4:
      if (ONCE && a.rows <= 128) return launch_ring<DT, 128, 128, 2, 2, 128, 2, 3, ONCE>(a, s);
      return launch_ring<DT, 128, 128, 2, 2, 128, 2, 3, false>(a, s);
    case 5: return launch_ring<DT, 128, 128, 2, 4, 128, 4, 4, false>(a, s);
    default: return launch_ring<DT, 64, 64, 2, 2, 128, 4, 4, false>(a, s);
  }
}
template <int DT, bool ONCE>
hipError_t launch_direct(const Int8Args& a, hipStream_t s) {
  if (a.rows <= 16) return launch_ring<DT, 16, 64, 1, 4, 256, 4, 4, ONCE>(a, s);
  if (a.rows <= 32) return launch_ring<DT, 32, 64, 1, 4, 128, 4, 4, ONCE>(a, s);
  if (a.rows <= 64) {
    // all tiles at once, two to a compute unit, where those of half the channels
    // are no more (us, 64 x 64 and 64 x 128): 50 x 8192 x 4096 10 15, 50 x 16000 16 20,
    // 50 x 32000 29 30, but 50 x 50000 46 43
    if (a.vocab <= 512 * 64) return launch_ring<DT, 64, 64, 2, 2, 128, 4, 4, ONCE>(a, s);
    return launch_ring<DT, 64, 128, 1, 4, 128, 3, 3, ONCE>(a, s);
  }
  const TilePlan p = plan_tiles(a.rows, a.vocab, a.width);
  Int8Args part = a;
  part.vocab = p.first;
  const hipError_t e = launch_shape<DT, ONCE>(part, p.shape, s);
  if (e != hipSuccess || p.first == a.vocab) return e;
  part.vocab = a.vocab - p.first;
  part.w += (long long)p.first * a.w_stride;
  part.w_scale += p.first;
  if (a.bias) part.bias += p.first;
  part.out += (long long)p.first * Fmt<DT>::ESZ;
  return launch_shape<DT, ONCE>(part, pick_tile(a.rows, part.vocab, a.width), s);
}

template <int DT>
hipError_t launch_int8_dt(const Int8Args& a, hipStream_t s) {
  const bool x_words = a.x_stride % 4 == 0 && (uintptr_t)a.x % 4 == 0;
  auto w_multiple = [&](int n) { return a.w_stride % n == 0 && (uintptr_t)a.w % n == 0; };
  if (x_words && w_multiple(4)) {
    const bool once = w_multiple(128) && (long long)a.vocab * a.width >= kInt8OnceBytes;
    return once ? launch_direct<DT, true>(a, s) : launch_direct<DT, false>(a, s);
  }
  // measured at width 4095 (us): 1 x 128256 93 (64 rows a tile 109), 30 x 128256 115
  // (123, 128x128 127), 64 x 128256 136 (128x128 141), 256 x 50001 118 (256x128 127,
  // 128x256 134, 256x256 217)
  if (a.rows <= 16) return launch_tile<DT, 16, 64, 1, 4, 256>(a, s);
  if (a.rows <= 32) return launch_tile<DT, 32, 64, 1, 4, 256>(a, s);
  if (a.rows <= 64) return launch_tile<DT, 64, 64, 1, 4, 256>(a, s);
  // up to three tiles of 64 x 64 to a compute unit (us, 64 x 64 and 128 x 128):
  // 90 x 24000 x 4095 45 48, 250 x 8000 31 41, 128 x 12000 36 47; past them 100 x
  // 28000 63 51, 90 x 32000 61 51, 128 x 128256 238 156
  if ((long long)((a.rows + 63) / 64) * ((a.vocab + 63) / 64) <= 768)
    return launch_tile<DT, 64, 64, 1, 4, 128>(a, s);
  return launch_tile<DT, 128, 128, 1, 4, 128>(a, s);
}

}  // namespace tsr
