// A row's gradient p (A + B x), written in tiles (token_logprobs_grad, distill_topk).
//
// Bound by memory: each logit is read once and each element written once. No
// loop and no state from one tile to the next. Tiles of 4 chunks a thread: 1024 x 128256
// bf16 with the entropy's gradient, reading past the caches, 87 us (525 MB at 6.0 TB/s;
// without it 80, 6.6), of 2 chunks 95 and of 8 87; 64 x 32000 fp32 6.1 us, 5.5 and 6.4.
#pragma once

#include "row_slice.hpp"

namespace tsr {

constexpr int kTileChunks = 4;   // 16-byte chunks a thread
template <int DT>
constexpr int kTileIds = kSliceBlock * kTileChunks * Fmt<DT>::EPC;

// Gradients of more bytes than the 256 MiB of the last cache are written past it: they could
// not stay, and what they push out costs more. token_logprobs_grad, gradients to memory of
// their own (to the same memory again; and read whole afterwards), us: 1024 x 151936 bf16 105
// against 116 (105, 112; 270, 287), 2048 x 128256 175 against 193 (175, 191; 444, 470).
// Smaller ones gain alone and lose as soon as they are read: 1024 x 128256 90 against 97 (90,
// 85; 230, 188). distill_topk, 1024 x 151936: 124 against 131, 2048 x 128256 196 against 204.
constexpr long long kGradOnceBytes = 256ll << 20;

template <bool ONCE>
__device__ __forceinline__ void store16(void* p, uint4 v) {
  if constexpr (ONCE) {
    store16_once(p, v);
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    store_words<4>(p, w);
  }
}

// Ids [tile * kTileIds, ...) of a row of V. READ_ONCE, WRITE_ONCE: past the caches.
template <int DT, bool READ_ONCE, bool WRITE_ONCE>
__device__ __forceinline__ void put_tile(const unsigned char* row, unsigned char* out, int V,
                                         int tile, const GradRow& g) {
  constexpr int EPC = Fmt<DT>::EPC;
  const int whole = V / EPC;
  const int first = tile * kSliceBlock * kTileChunks + (int)threadIdx.x;
  uint4 c[kTileChunks];
#pragma unroll
  for (int j = 0; j < kTileChunks; ++j) {   // chunks past the last whole one repeat it
    const unsigned char* p = row + (long long)min(first + j * kSliceBlock, whole - 1) * 16;
    c[j] = whole == 0 ? make_uint4(0, 0, 0, 0) : READ_ONCE ? load16_once(p) : load16(p);
  }
  const auto all = [&](auto&& of) {
#pragma unroll
    for (int j = 0; j < kTileChunks; ++j) {
      float v[EPC];
      unpack<DT>(c[j], v);
#pragma unroll
      for (int e = 0; e < EPC; ++e) v[e] = of(v[e]);
      const int i = first + j * kSliceBlock;
      if (i < whole) store16<WRITE_ONCE>(out + (long long)i * 16, pack<DT>(v));
    }
  };
  if (g.plain)
    all([&](float z) { return g.of<true, true>(z); });
  else if (g.B != 0.0f)
    all([&](float z) { return g.of<true, false>(z); });
  else
    all([&](float z) { return g.of<false, false>(z); });
  // the elements behind the last whole chunk, with the tile that they lie in
  const int at = whole * EPC;
  if (at < V && at / kTileIds<DT> == tile && (int)threadIdx.x < V - at)
    store_elem<DT>(out, at + (int)threadIdx.x, g.at(load_elem<DT>(row, at + (int)threadIdx.x)));
}

template <int DT>
__device__ __forceinline__ void zero_tile(unsigned char* out, int V, int tile) {
  constexpr int EPC = Fmt<DT>::EPC;
  const int whole = V / EPC;
#pragma unroll
  for (int j = 0; j < kTileChunks; ++j) {
    const int i = (tile * kTileChunks + j) * kSliceBlock + (int)threadIdx.x;
    if (i < whole) store16<false>(out + (long long)i * 16, make_uint4(0, 0, 0, 0));
  }
  const int at = whole * EPC;
  if (at < V && at / kTileIds<DT> == tile && (int)threadIdx.x < V - at)
    store_elem<DT>(out, at + (int)threadIdx.x, 0.0f);
}

template <int DT>
int tiles_of(int V) {
  return (int)(((long long)V + kTileIds<DT> - 1) / kTileIds<DT>);
}

}  // namespace tsr
