// Wide loads and stores at any byte alignment (the unaligned access mode the
// HSA runtime sets), never outside the row they are given.
#pragma once

#include "device_common.hpp"

namespace tsr {

struct __attribute__((packed, aligned(1))) Bytes16 { uint32_t w[4]; };
struct __attribute__((packed, aligned(1))) Bytes8 { uint32_t w[2]; };
struct __attribute__((packed, aligned(1))) Bytes4 { uint32_t w[1]; };

__device__ __forceinline__ uint4 load16(const void* p) {
  const Bytes16 b = *static_cast<const Bytes16*>(p);
  return make_uint4(b.w[0], b.w[1], b.w[2], b.w[3]);
}

// Four words at a word boundary.
typedef uint32_t Words4 __attribute__((ext_vector_type(4), aligned(4)));

template <int N>
__device__ __forceinline__ void store_words(void* p, const uint32_t* w) {
  static_assert(N == 1 || N == 2 || N == 4, "words");
  if constexpr (N == 1) {
    *static_cast<Bytes4*>(p) = Bytes4{{w[0]}};
  } else if constexpr (N == 2) {
    *static_cast<Bytes8*>(p) = Bytes8{{w[0], w[1]}};
  } else {
    *static_cast<Bytes16*>(p) = Bytes16{{w[0], w[1], w[2], w[3]}};
  }
}

// 16 bytes, at any byte, that are not kept in the caches.
typedef uint32_t Any4 __attribute__((ext_vector_type(4), aligned(1)));
__device__ __forceinline__ uint4 load16_once(const void* p) {
  const Any4 v = __builtin_nontemporal_load(static_cast<const Any4*>(p));
  return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ void store16_once(void* p, uint4 v) {
  const Any4 w = {v.x, v.y, v.z, v.w};
  __builtin_nontemporal_store(w, static_cast<Any4*>(p));
}

// Elements [e0, e0 + EPC) of a row of n elements; those at or past n read as 0.
template <int DT>
__device__ __forceinline__ uint4 load_chunk_zero(const unsigned char* row, long long e0,
                                                 long long n) {
  constexpr int EPC = Fmt<DT>::EPC, ESZ = Fmt<DT>::ESZ;
  if (e0 + EPC <= n) return load16(row + e0 * ESZ);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < EPC; ++e) {
    if (e0 + e < n) {
      if constexpr (DT == 0)
        w[e] = *reinterpret_cast<const uint32_t*>(row + (e0 + e) * 4);
      else
        w[e / 2] |= (uint32_t) * reinterpret_cast<const uint16_t*>(row + (e0 + e) * 2)
                    << (16 * (e % 2));
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Bytes [k, k + 16) of a row of n bytes; those at or past n read as 0. Without
// a branch where n >= 16: the last 16 bytes of the row at most, shifted down by
// those before k.
__device__ __forceinline__ uint4 load_bytes_zero(const int8_t* row, int k, int n) {
  if (n < 16) {
    uint64_t lo = 0, hi = 0;
#pragma unroll 1
    for (int e = k; e < n; ++e) {
      const uint64_t byte = (uint8_t)row[e];
      if (e - k < 8)
        lo |= byte << (8 * (e - k));
      else
        hi |= byte << (8 * (e - k - 8));
    }
    return make_uint4((uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32));
  }
  const int at = min(k, n - 16);
  const uint4 v = load16(row + at);
  const int s = min(k - at, 16) * 8;   // 0 .. 128 bits
  uint64_t lo = v.x | (uint64_t)v.y << 32, hi = v.z | (uint64_t)v.w << 32;
  lo = s >= 64 ? hi : lo;
  hi = s >= 64 ? 0 : hi;
  const int r = s & 63;
  lo = r ? lo >> r | hi << (64 - r) : lo;
  hi >>= r;
  if (s >= 128) lo = 0;
  return make_uint4((uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32));
}

// Two floats as bfloat16, each to nearest even; the first in the low half.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)a) |
         ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)b) << 16);
}

}  // namespace tsr
