// The grids of the routed launches (include/qroute.h).  Plain host code, shared by the
// launchers, by the C ABI's argument validation and by its tests: HIP takes
// fewer than 2^32 work items in a dimension of a launch.
#pragma once
#include <stdint.h>

#include <algorithm>

#include "prefill_plan.hpp"

namespace qgemv {

constexpr int64_t kMaxWorkItems = (int64_t(1) << 32) - 1;

// Tiles of bt rows that n slots over e weight sets can make at most.
inline int64_t max_tiles(int64_t n, int64_t e, int64_t bt) {
  const int64_t used = n < e ? n : e;
  return used + (n - used) / bt;
}

// ---- row movers ---------------------------------------------------------------

constexpr int kRouteMoveThreads = 256;

// Pieces of 8 elements of a row of c, one a thread; rows that are not whole pieces are
// cut where the output's address is a multiple of the piece, which can make one more.
inline int64_t route_row_pieces(int64_t c) { return (c + 7) / 8 + (c % 8 != 0 ? 1 : 0); }

inline int64_t route_move_workgroups(int64_t rows, int64_t c) {
  return (rows * route_row_pieces(c) + kRouteMoveThreads - 1) / kRouteMoveThreads;
}

// Most that rows * (c + 16) may be: rows * pieces(c) <= rows * (c + 15) / 8 is then below
// 2^32, also rounded up to whole workgroups (c < 2^24 + 1: from 2048 rows on
// rows / 8 is 256 or more, with fewer it is 2^32 - 2^21 at most).
constexpr int64_t kRouteMaxElems = int64_t(1) << 35;

// Waves of the combine's gradient per token: one for rows of at most 1024 elements, and
// where four would be too many work items.
inline int route_grad_waves(int64_t t, int64_t c) {
  return c <= 1024 || t * kRouteMoveThreads > kMaxWorkItems ? 1 : 4;
}
inline int64_t route_grad_workgroups(int64_t t, int64_t c) {
  const int64_t tokens = 4 / route_grad_waves(t, c);  // a workgroup's
  return (t + tokens - 1) / tokens;
}

// ---- routed products ------------------------------------------------------------

// Routed products on packed matrices of format `fmt`.
enum RouteFmt : int { kRouteQ4k = 0, kRouteNvfp4 = 1, kRouteTq1 = 2 };

constexpr int kQ4kBT = 64;   // tokens of a workgroup of the many-row Q4_K kernel
constexpr int kQ4kBN = 256;  // its weight rows
constexpr int kQ4kWaves = 8;

enum RoutedKernel : int { kRoutedRows, kRoutedQ4k, kRoutedTile };

struct RoutedPlan {
  RoutedKernel kernel;
  int rw, kw;      // kRoutedRows: 16 rw weight rows a workgroup, K in kw parts
  int bt, nb;      // kRoutedTile: bt tokens x 128 nb weight rows
  int threads;     // of a workgroup
  int64_t groups;  // workgroups along the weight rows
  int64_t tiles;   // of tokens, at most
};

// The launch of n > 0 slots over e weight sets of m > 0 rows.
inline RoutedPlan routed_plan(int fmt, int64_t n, int64_t e, int64_t m) {
  const bool q4k = fmt == kRouteQ4k;
  const int64_t used = n < e ? n : e;
  const int64_t rows = n / used;  // of a weight set, on average
  // tiles of bt tokens to expect: each weight set's last one is half full on average
  const auto tiles = [&](int64_t bt) {
    return used == 1 ? (n + bt - 1) / bt : std::max<int64_t>(used, n / bt + used / 2);
  };
  // What a kernel takes for 256 of K, in 1/100 us, by its workgroups: of 16 tokens
  // x 64 weight rows (K in parts while they are few, see below), 64 x 128 and 256 x 256
  // (128 x 256 where weight sets have no more tokens).  Fitted to Q4_K through these three;
  // at 31 sizes of each, NVFP4 and TQ1_0 come within 12% of the best of the three but for one
  // (TQ1_0, 256 rows of each of two sets of 4096 x 14336: 228 us, 171 by the first).  Us by
  // the three, NVFP4 / TQ1_0, 8 sets of 14336 x 4096: 34 rows each 135, 131, 151 / 122, 137,
  // 161; 48 rows 171, 135, 153 / 152, 139, 161; 64 rows 217, 182, 159 / 191, 200, 185; 128
  // rows 386, 293, 233 / 346, 298, 224.  Few weight rows leave large tiles a few CUs: one set
  // of 512 x 13568, 400 rows: 29, 121, 313 / 32, 140, 386.  The average hides a popular
  // set: 1024 tokens over 64 sets of 1024 x 4096, one with seven tenths of them, take 74 us
  // against 46 for an even spread (Q4_K; NVFP4 56 and 54, TQ1_0 46 and 43).
  const int64_t few = tiles(16) * ((m + 63) / 64), mid = tiles(64) * ((m + 127) / 128);
  const int64_t big = tiles(256) * ((m + 255) / 256);
  const int64_t cost_few = few <= 128 ? 35 : few <= 256 ? 50 : 20 + 50 * few / 256;
  const int64_t cost_mid = 150 + 185 * std::max<int64_t>(mid, 256) / 256;
  const int64_t cost_big = (big + 255) / 256 * (rows <= 128 ? 530 : 760);
  // Q4_K's own, 64 x 256, one workgroup a CU (8 sets of 14336 x 4096, us by the first kernel
  // and by this one: 12 rows each 76, 84; 16 rows 94, 82; 32 rows 140, 95; one set of 4096 x
  // 4096: 256 rows 37, 46; 512 rows 66, 48; of 512 x 13568, 1600 rows: 108, 133).
  const int64_t cost_q4k = (tiles(kQ4kBT) * ((m + kQ4kBN - 1) / kQ4kBN) + 255) / 256 * 270;
  RoutedPlan p{};
  // Up to 32 rows a weight set the other formats' few-row kernel does better than the
  // estimate, which is Q4_K's (8 sets of 14336 x 4096, 28 rows each: TQ1_0 91 us, 137 by
  // tiles, NVFP4 119 and 132; 32 sets of 4096 x 4096, 32 rows each: 128, 141; 149, 138).
  if (q4k ? cost_few <= cost_q4k : rows <= 32 || (cost_few <= cost_mid && cost_few <= cost_big)) {
    p.kernel = kRoutedRows;
    // Workgroups of 64 rows and all of K where that gives more than a CU's one
    // (three fit a CU).  With fewer, a workgroup's walk through K is what takes
    // the time: 64 rows with K in two parts, or 32 with K in four, while these
    // make at most one workgroup a CU (Q4_K, one token, two weight sets: 14336 x
    // 4096 15.3 / 19.1 / 28.6 us in this order, 8192 x 4096 12.0 / 10.8 / 15.5,
    // 4096 x 4096 11.6 / 11.1 / 9.3, 4096 x 14336 30.6 / 28.4 / 17.7).
    // (TQ1_0, whose decoding takes longer than its few bytes, in two parts while the workgroups
    // are at most two a CU: 74 slots over 8 weight sets, us with two parts and with one: 4096 x
    // 2048 13.5, 13.2; x 4096 20.5, 20.8; x 8192 32.2, 34.9; x 14336 50.6, 53.7; 2560 x 8192 30.9,
    // 33.6; 4608 x 8192 45.3, 43.7; 8192 x 4096 34.4, 30.0; 8192 x 14336 110.7, 107.5)
    p.rw = few <= 128 ? 2 : 4;
    p.kw = few <= 128 ? 4 : few <= (fmt == kRouteTq1 ? 512 : 256) ? 2 : 1;
    p.threads = 64 * p.rw * p.kw;
    p.groups = (m + 16 * p.rw - 1) / (16 * p.rw);
    p.tiles = max_tiles(n, e, 16);
  } else if (q4k) {
    p.kernel = kRoutedQ4k;
    p.threads = 64 * kQ4kWaves;
    p.groups = (m + kQ4kBN - 1) / kQ4kBN;
    p.tiles = max_tiles(n, e, kQ4kBT);
  } else {
    p.kernel = kRoutedTile;
    p.bt = cost_mid <= cost_big ? 64 : 256;
    p.nb = cost_mid <= cost_big ? 1 : 2;
    p.threads = 512;
    p.groups = (m + kPfBN * p.nb - 1) / (kPfBN * p.nb);
    p.tiles = max_tiles(n, e, p.bt);
  }
  return p;
}

inline int64_t routed_work_items(const RoutedPlan& p) { return p.groups * p.tiles * p.threads; }

}  // namespace qgemv
