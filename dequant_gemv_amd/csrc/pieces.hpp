// Pieces of rows of any length: 16 or 32 bytes loaded and stored by one thread
// whatever element they start at.  With !Loose every row is a whole number of
// pieces, aligned to their size.  Otherwise rows of 16-bit elements start at any
// even address and rows of fp32 at any multiple of four: pieces are read as the
// dwords around them and shifted into place, and stored as whole dwords with a
// 16-bit store at either end where they start or end in the middle of one.  (8192
// rows of 4095 fp16 copied in 75 us by single elements, 23 like this; aligned
// ones of 4096 take 21.)
#pragma once
#include "device.hpp"
#include "rows.hpp"

namespace qgemv {

typedef unsigned u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// N elements as their bits: 8 of any type, or 4 of fp32.
template <typename T, int N = 8>
struct Bits {
  static_assert(N == 8 || (N == 4 && sizeof(T) == 4), "elements of a piece");
  static constexpr int kWords = N * (int)sizeof(T) / 4;
  unsigned w[kWords];
};

// Elements [e, e + count) of p, an array of `total` elements whose start is 16-byte
// aligned; the rest of the N are zero.  (A partial piece is loaded whole where the
// array goes on, so that a wave's lanes take one path.)
template <typename T, bool Loose, int N = 8>
__device__ __forceinline__ Bits<T, N> load_bits(const T* p, int64_t e, int count, int64_t total) {
  Bits<T, N> b;
  if constexpr (!Loose) {
    const u32x4* const src = reinterpret_cast<const u32x4*>(p + e);
#pragma unroll
    for (int i = 0; i < Bits<T, N>::kWords / 4; ++i) {
      const u32x4 v = src[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) b.w[4 * i + j] = v[j];
    }
    return b;
  }
  if (count < N && e + N > total) {  // the end of the array
#pragma unroll
    for (int i = 0; i < Bits<T, N>::kWords; ++i) b.w[i] = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < count) {
        if constexpr (sizeof(T) == 4)
          b.w[i] = __builtin_bit_cast(unsigned, p[e + i]);
        else
          b.w[i / 2] |= (unsigned)reinterpret_cast<const uint16_t*>(p)[e + i] << (16 * (i % 2));
      }
    return b;
  }
  if constexpr (sizeof(T) == 4) {
    const u32x4_a4* const src = reinterpret_cast<const u32x4_a4*>(p + e);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4_a4 v = src[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) b.w[4 * i + j] = 4 * i + j < count ? v[j] : 0u;
    }
  } else {
    // the dwords that hold the 16 bytes; where the piece starts in the middle of
    // one, its last element is the first half of a fifth, whose other half may be past the array
    const unsigned* const src = reinterpret_cast<const unsigned*>(p) + (e >> 1);
    const u32x4_a4 v = *reinterpret_cast<const u32x4_a4*>(src);
    const unsigned odd = (unsigned)e & 1u;
    const unsigned last = odd ? (unsigned)reinterpret_cast<const uint16_t*>(p)[e + 7] : 0u;
    b.w[0] = __builtin_amdgcn_alignbyte(v[1], v[0], 2u * odd);
    b.w[1] = __builtin_amdgcn_alignbyte(v[2], v[1], 2u * odd);
    b.w[2] = __builtin_amdgcn_alignbyte(v[3], v[2], 2u * odd);
    b.w[3] = __builtin_amdgcn_alignbyte(last, v[3], 2u * odd);
    if (count < N)
#pragma unroll
      for (int i = 0; i < 4; ++i) b.w[i] = 2 * i + 1 < count ? b.w[i] : 2 * i < count ? b.w[i] & 0xFFFFu : 0u;
  }
  return b;
}

template <typename T, bool Loose, int N = 8>
__device__ __forceinline__ void store_bits(T* p, int64_t e, int count, const Bits<T, N>& b) {
  if constexpr (!Loose) {
    u32x4* const dst = reinterpret_cast<u32x4*>(p + e);
#pragma unroll
    for (int i = 0; i < Bits<T, N>::kWords / 4; ++i) dst[i] = u32x4{b.w[4 * i], b.w[4 * i + 1], b.w[4 * i + 2], b.w[4 * i + 3]};
  } else if constexpr (sizeof(T) == 4) {
    if (count == N) {
      u32x4_a4* const dst = reinterpret_cast<u32x4_a4*>(p + e);
#pragma unroll
      for (int i = 0; i < N / 4; ++i) dst[i] = u32x4_a4{b.w[4 * i], b.w[4 * i + 1], b.w[4 * i + 2], b.w[4 * i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < N - 1; ++i)
        if (i < count) p[e + i] = __builtin_bit_cast(T, b.w[i]);
    }
  } else {
    // whole dwords, from the first one's start: element 0, or 1 after a 16-bit store
    const unsigned odd = (unsigned)e & 1u;
    uint16_t* const dst = reinterpret_cast<uint16_t*>(p) + e;
    const unsigned w[4] = {__builtin_amdgcn_alignbyte(b.w[1], b.w[0], 2u * odd), __builtin_amdgcn_alignbyte(b.w[2], b.w[1], 2u * odd),
                           __builtin_amdgcn_alignbyte(b.w[3], b.w[2], 2u * odd), b.w[3] >> (16u * odd)};
    const int rest = count - (int)odd;
    if (odd) dst[0] = (uint16_t)b.w[0];
    unsigned* const to = reinterpret_cast<unsigned*>(dst + odd);
    if (rest == 8) {
      *reinterpret_cast<u32x4_a4*>(to) = u32x4_a4{w[0], w[1], w[2], w[3]};
    } else if (rest == 7) {
      __builtin_memcpy(to, w, 12);  // (a vector of three has the size of four, and a store of it may have too)
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (2 * i + 1 < rest) to[i] = w[i];
    }
    if (rest & 1) dst[count - 1] = (uint16_t)(rest == 1 ? w[0] : rest == 3 ? w[1] : rest == 5 ? w[2] : w[3]);
  }
}

template <typename T, int N>
__device__ __forceinline__ void from_bits(const Bits<T, N>& b, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (sizeof(T) == 4)
      v[i] = __builtin_bit_cast(float, b.w[i]);
    else
      v[i] = (float)__builtin_bit_cast(T, (unsigned short)(b.w[i / 2] >> (16 * (i % 2))));
  }
}

template <typename T, int N>
__device__ __forceinline__ Bits<T, N> to_bits(const float (&v)[N]) {
  Bits<T, N> b;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N; ++i) b.w[i] = __builtin_bit_cast(unsigned, v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) b.w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
  }
  return b;
}

}  // namespace qgemv
