// What the kernels that read a plan (include/qroute.h) share: finding a
// workgroup's tile of rows, matrix-core operands of 16 x 16 tiles and stores of
// outputs.
#pragma once
#include "device.hpp"
#include "epilogue.hpp"
#include "prefill_tile.hpp"
#include "route_grid.hpp"

namespace qgemv {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// x rows that are not there: beyond every x descriptor's range (at most 2^30
// bytes), also when an offset of up to 2^31 is added.
constexpr uint32_t kDeadRow = 0x40000000u;

struct RoutedTile {
  int e;
  int first;  // sorted position of the tile's first row
  int rows;   // at most bt; 0: no such tile
};

// Tile `index` of the weight sets' rows, cut into tiles of bt rows each: every
// wave scans the counts, 64 weight sets at a time.  With Rest the slots that
// name no weight set follow as weight set e_count.  Offsets are clamped into
// [0, n], so no tile reaches past the slots whatever they hold.
template <bool Rest = false>
__device__ __forceinline__ RoutedTile find_tile(const int32_t* offsets, int e_count, int n, int bt, int index) {
  const int lane = threadIdx.x & 63;
  const int sets = e_count + (Rest ? 1 : 0);
  int carry = 0;
  for (int e0 = 0; e0 < sets; e0 += 64) {
    const int e = e0 + lane;
    int first = 0, rows = 0;
    if (e < sets) {
      first = min(max(offsets[e], 0), n);
      const int end = Rest && e == e_count ? n : offsets[e + 1];
      rows = min(max(end, first), n) - first;
    }
    const int tiles = (rows + bt - 1) / bt;
    int incl = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
    const uint64_t reach = __ballot(carry + incl > index);
    if (reach) {
      const int src = __ffsll((unsigned long long)reach) - 1;
      const int at = index - carry - (__shfl(incl, src) - __shfl(tiles, src));  // tile within the weight set
      RoutedTile t;
      t.e = __builtin_amdgcn_readfirstlane(e0 + src);
      t.first = __builtin_amdgcn_readfirstlane(__shfl(first, src) + at * bt);
      t.rows = __builtin_amdgcn_readfirstlane(min(bt, __shfl(rows, src) - at * bt));
      return t;
    }
    carry += __shfl(incl, 63);
  }
  return RoutedTile{0, 0, 0};
}

// Workgroup b of n as its place in a walk that gives each of the eight XCDs (b %
// 8) a contiguous part: neighbours in the walk share an L2.
__device__ __forceinline__ int xcd_walk(int b, int n) {
  const int x = b % 8, each = n / 8, more = n % 8;
  return x * each + min(x, more) + b / 8;
}

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16_bf(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

__device__ __forceinline__ void store_y(void* y, int dtype, int64_t at, float v) {
  if (dtype == kF32)
    static_cast<float*>(y)[at] = v;
  else if (dtype == kF16)
    static_cast<_Float16*>(y)[at] = (_Float16)pin_f32(v);
  else
    static_cast<__bf16*>(y)[at] = (__bf16)pin_f32(v);
}

}  // namespace qgemv
