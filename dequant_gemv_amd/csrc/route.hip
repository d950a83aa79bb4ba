// The plan of a routed step (slots sorted by the weight set they name) and the
// movement of rows into that order, back with weights applied, and its
// gradient (include/qroute.h), for gfx950.
#include "device.hpp"
#include "epilogue.hpp"
#include "launch_route.hpp"
#include "pieces.hpp"

namespace qgemv {

// ---- the plan ---------------------------------------------------------------
//
// A stable counting sort: position = offsets[key] + number of earlier slots
// with the same key, where a slot that names no weight set has key E.  A
// workgroup takes kSortWaves contiguous runs of 64 * kSortItems slots, one a
// wave.  Within a batch of 64 slots a lane's rank is the number of lower lanes
// with its key, found with one ballot per key bit; the run's count per key is
// kept in LDS, one array a wave, so no atomic is needed and the order is that
// of the slots.  Up to one workgroup's slots are sorted in one launch;
// more take two: the counts of every workgroup go to the workspace and each slot's
// rank in its workgroup to position; then each workgroup adds up the counts
// before it and writes its own slots.  Bound by the launches and their chains of
// latencies, not by bytes (128 slots over 64 keys 4.3 us, 131072 over 128 in 10.8 us;
// three launches with the ranks found twice took 20).

constexpr int kSortWaves = 16;
constexpr int kSortItems = 4;                               // slots per lane
constexpr int kSortChunk = 64 * kSortWaves * kSortItems;    // slots per workgroup
constexpr int kSortMaxKeys = 1024 + 1;                      // weight sets and "none"

struct SortTable {
  int begin[kSortMaxKeys];   // of a key: its first position
  int before[kSortMaxKeys];  // of a key: its slots in earlier workgroups
};
struct SortLds : SortTable {
  int count[kSortWaves][kSortMaxKeys];  // per wave; then the slots of a key in earlier waves
};

// key of slot s
__device__ __forceinline__ int sort_key(const int32_t* ids, int s, int e) {
  const int id = ids[s];
  return (unsigned)id < (unsigned)e ? id : e;
}

// Counts and ranks of this workgroup's slots [first, first + kSortChunk) below
// n: key[i], rank[i] of the lane's i-th slot (rank among the wave's slots
// with the same key), and count[wave][key].
__device__ __forceinline__ void sort_local(SortLds& lds, const int32_t* ids, int64_t first, int64_t n, int e, int bits,
                                           int (&key)[kSortItems], int (&rank)[kSortItems]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int k = lane; k <= e; k += 64) lds.count[wave][k] = 0;
  const int64_t s0 = first + wave * (64 * kSortItems) + lane;
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) key[i] = s0 + 64 * i < n ? sort_key(ids, (int)(s0 + 64 * i), e) : -1;
  __syncthreads();
  int* const mine = lds.count[wave];
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) {
    uint64_t same = __ballot(key[i] >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = __ballot((key[i] >> b) & 1);
      same &= (key[i] >> b) & 1 ? m : ~m;
    }
    const int below = __popcll(same & ((uint64_t(1) << lane) - 1));
    rank[i] = 0;
    if (key[i] >= 0) {
      const int before = mine[key[i]];
      rank[i] = before + below;
      // the highest lane of a key stores the new count, after every lane's read
      __builtin_amdgcn_wave_barrier();
      if (lane == 63 - __clzll(same)) mine[key[i]] = before + below + 1;
    }
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
}

// count[][key] -> the slots of that key in earlier waves; returns the total.
__device__ __forceinline__ int sort_wave_prefix(SortLds& lds, int key) {
  int sum = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    const int c = lds.count[w][key];
    lds.count[w][key] = sum;
    sum += c;
  }
  return sum;
}

// begin[key] holds the totals of all keys: turns them into first positions.
// Runs on wave 0.
__device__ __forceinline__ void sort_scan(SortTable& lds, int keys) {
  const int lane = threadIdx.x & 63;
  int carry = 0;
  for (int k0 = 0; k0 < keys; k0 += 64) {
    const int k = k0 + lane;
    const int c = k < keys ? lds.begin[k] : 0;
    int v = c;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(v, d);
      if (lane >= d) v += o;
    }
    if (k < keys) lds.begin[k] = carry + v - c;
    carry += __shfl(v, 63);
  }
}

__device__ __forceinline__ void sort_write(const SortLds& lds, int64_t first, int64_t n, int e,
                                           const int (&key)[kSortItems], const int (&rank)[kSortItems],
                                           int32_t* order, int32_t* position) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t s0 = first + wave * (64 * kSortItems) + lane;
#pragma unroll
  for (int i = 0; i < kSortItems; ++i)
    if (key[i] >= 0) {
      const int s = (int)(s0 + 64 * i);
      const int p = lds.begin[key[i]] + lds.count[wave][key[i]] + rank[i];
      order[p] = key[i] < e ? s : -1 - s;
      position[s] = key[i] < e ? p : -1;
    }
}

__global__ __launch_bounds__(64 * kSortWaves) void route_sort_kernel(const int32_t* __restrict__ ids, int64_t n, int e,
                                                                     int bits, int32_t* __restrict__ order,
                                                                     int32_t* __restrict__ position,
                                                                     int32_t* __restrict__ offsets) {
  __shared__ SortLds lds;
  int key[kSortItems], rank[kSortItems];
  sort_local(lds, ids, 0, n, e, bits, key, rank);
  for (int k = threadIdx.x; k <= e; k += 64 * kSortWaves) lds.begin[k] = sort_wave_prefix(lds, k);
  __syncthreads();
  if (threadIdx.x < 64) sort_scan(lds, e + 1);
  __syncthreads();
  for (int k = threadIdx.x; k <= e; k += 64 * kSortWaves) offsets[k] = lds.begin[k];
  sort_write(lds, 0, n, e, key, rank, order, position);
}

// The counts of a workgroup's slots by key, and in position[s] (which the next
// kernel overwrites) the number of earlier slots of the workgroup with s's key.
__global__ __launch_bounds__(64 * kSortWaves) void route_count_kernel(const int32_t* __restrict__ ids, int64_t n,
                                                                      int e, int bits, int32_t* __restrict__ counts,
                                                                      int32_t* __restrict__ position) {
  __shared__ SortLds lds;
  int key[kSortItems], rank[kSortItems];
  const int64_t first = (int64_t)blockIdx.x * kSortChunk;
  sort_local(lds, ids, first, n, e, bits, key, rank);
  for (int k = threadIdx.x; k <= e; k += 64 * kSortWaves)
    counts[(int64_t)blockIdx.x * (e + 1) + k] = sort_wave_prefix(lds, k);
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < kSortItems; ++i)
    if (key[i] >= 0)
      position[first + wave * (64 * kSortItems) + lane + 64 * i] = lds.count[wave][key[i]] + rank[i];
}

__global__ __launch_bounds__(64 * kSortWaves) void route_place_kernel(const int32_t* __restrict__ ids, int64_t n,
                                                                      int e, const int32_t* __restrict__ counts,
                                                                      int32_t* __restrict__ order,
                                                                      int32_t* __restrict__ position,
                                                                      int32_t* __restrict__ offsets) {
  __shared__ SortTable lds;
  int key[kSortItems], rank[kSortItems];
  const int64_t s0 = (int64_t)blockIdx.x * kSortChunk + threadIdx.x;
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) {
    const int64_t s = s0 + 64 * kSortWaves * i;
    key[i] = s < n ? sort_key(ids, (int)s, e) : -1;
    rank[i] = s < n ? position[s] : 0;
  }
  for (int k = threadIdx.x; k <= e; k += 64 * kSortWaves) lds.begin[k] = lds.before[k] = 0;
  __syncthreads();
  // slots of each key in earlier workgroups, and in all of them: as many
  // threads a key as there are (integer sums: any order gives the same)
  const int keys = e + 1, share = max(1, 64 * kSortWaves / keys);
  for (int i = threadIdx.x; i < share * keys; i += 64 * kSortWaves) {
    const int part = i / keys, k = i - part * keys;
    int before = 0, all = 0;
    for (int c0 = part; c0 < (int)gridDim.x; c0 += 8 * share) {
      int v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = c0 + j * share;
        v[j] = c < (int)gridDim.x ? counts[(int64_t)c * keys + k] : 0;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        before += c0 + j * share < (int)blockIdx.x ? v[j] : 0;
        all += v[j];
      }
    }
    atomicAdd(&lds.before[k], before);
    atomicAdd(&lds.begin[k], all);
  }
  __syncthreads();
  if (threadIdx.x < 64) sort_scan(lds, e + 1);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int k = threadIdx.x; k <= e; k += 64 * kSortWaves) offsets[k] = lds.begin[k];
#pragma unroll
  for (int i = 0; i < kSortItems; ++i)
    if (key[i] >= 0) {
      const int s = (int)(s0 + 64 * kSortWaves * i);
      const int p = lds.begin[key[i]] + lds.before[key[i]] + rank[i];
      order[p] = key[i] < e ? s : -1 - s;
      position[s] = key[i] < e ? p : -1;
    }
}

static int64_t sort_chunks(int64_t n) { return (n + kSortChunk - 1) / kSortChunk; }

int64_t route_sort_workspace(int64_t n, int64_t e) { return n <= kSortChunk ? 0 : 4 * sort_chunks(n) * (e + 1); }

hipError_t launch_route_sort(const int32_t* ids, int64_t n, int64_t e, int32_t* order, int32_t* position,
                             int32_t* offsets, void* ws, hipStream_t s) {
  int bits = 0;
  while ((e >> bits) != 0) ++bits;  // keys 0 .. e
  if (n <= kSortChunk) {
    hipLaunchKernelGGL(route_sort_kernel, dim3(1), dim3(64 * kSortWaves), 0, s, ids, n, (int)e, bits, order, position,
                       offsets);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)sort_chunks(n));
  int32_t* const counts = static_cast<int32_t*>(ws);
  hipLaunchKernelGGL(route_count_kernel, grid, dim3(64 * kSortWaves), 0, s, ids, n, (int)e, bits, counts, position);
  hipLaunchKernelGGL(route_place_kernel, grid, dim3(64 * kSortWaves), 0, s, ids, n, (int)e, (const int32_t*)counts, order, position, offsets);
  return hipGetLastError();
}

// ---- moving rows --------------------------------------------------------------
//
// Rows are cut into pieces of 8 elements, one per thread, consecutive threads
// taking consecutive pieces.  These kernels only move bytes, so what counts is
// whole-line accesses and loads in flight.  Measured: 8192 rows of 4096 fp16 gathered
// in 20.6 us (4.9 TB/s; a large copy reaches 4.8), 4099 x 2 rows of 4096 fp32 combined to
// bf16 in 32.3 us (5.2 TB/s), the gradient of 2048 x 4 rows of 4096 bf16 in 32.9 us (4.6
// TB/s), 16 x 8 rows combined in 3.4 us (the launch).

// Piece (row, first element, elements) of this thread: the grid covers all rows'
// pieces (of 8 elements, row_pieces of them), 256 a workgroup.  Loose: rows are cut
// where the output's address is a multiple of the piece, so that only a row's first
// and last pieces are partial (8192 rows of 4095 fp16: 23 us; 29 with pieces from the
// row's start, whose stores are in three parts in every other row).  false: no such piece.
struct Piece {
  int64_t row;
  int at, count;
};
template <bool Loose>
__device__ __forceinline__ int row_pieces(int c) {  // route_row_pieces
  return (c + 7) / 8 + (Loose ? 1 : 0);
}
template <bool Loose>
__device__ __forceinline__ bool piece_of(int64_t rows, int c, Piece& out) {
  // the division of the workgroup's first piece is uniform; a thread's own is 32-bit
  const int per = row_pieces<Loose>(c);
  const int64_t first = (int64_t)blockIdx.x * 256;
  const int64_t row0 = first / per;
  const unsigned in = (unsigned)(first - row0 * per) + threadIdx.x;
  const unsigned skip = in / (unsigned)per;
  out.row = row0 + skip;
  const int at = 8 * (int)(in - skip * (unsigned)per) - (Loose ? (int)((out.row * c) & 7) : 0);
  out.at = max(at, 0);
  out.count = min(at + 8, c) - out.at;
  return out.row < rows && out.count > 0;
}

template <typename T, bool Loose, bool Weighted>
__global__ __launch_bounds__(256) void route_gather_kernel(const T* __restrict__ x, const int32_t* __restrict__ order,
                                                           const float* __restrict__ weights, T* __restrict__ out,
                                                           int64_t n, int k, int c, int64_t x_total) {
  Piece p;
  if (!piece_of<Loose>(n, c, p)) return;
  const int slot = order[p.row];
  if ((unsigned)slot >= (unsigned)n) return;  // names no weight set
  Bits<T> b = load_bits<T, Loose>(x, (int64_t)(slot / k) * c + p.at, p.count, x_total);
  if constexpr (Weighted) {
    float v[8];
    from_bits(b, v);
    const float w = weights[slot];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= w;
    b = to_bits<T>(v);
  }
  store_bits<T, Loose>(out, p.row * c + p.at, p.count, b);
}

template <typename TR, typename TY, bool Loose>
__global__ __launch_bounds__(256) void route_combine_kernel(const TR* __restrict__ rows,
                                                            const int32_t* __restrict__ position,
                                                            const float* __restrict__ weights, TY* __restrict__ y,
                                                            int64_t t_count, int k, int c) {
  Piece p;
  if (!piece_of<Loose>(t_count, c, p)) return;
  const int64_t s0 = p.row * k, n = t_count * k;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  for (int j0 = 0; j0 < k; j0 += 4) {  // four rows in flight
    Bits<TR> b[4];
    float w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = j0 + j < k ? position[s0 + j0 + j] : -1;
      const bool live = (uint64_t)(int64_t)at < (uint64_t)n;
      w[j] = 0.f;
      b[j] = Bits<TR>{};
      if (live) {
        w[j] = weights ? weights[s0 + j0 + j] : 1.f;
        b[j] = load_bits<TR, Loose>(rows, (int64_t)at * c + p.at, p.count, n * c);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[8];
      from_bits(b[j], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(w[j], v[i], acc[i]);
    }
  }
  store_bits<TY, Loose>(y, p.row * c + p.at, p.count, to_bits<TY>(acc));
}

// W waves a token, 4 / W tokens a workgroup: dy's pieces are read once for every KJ
// choices, whose rows' dot products with dy are summed in fp32 by thread, then
// across the wave and the waves in a fixed order.
template <typename TD, typename TR, bool Loose, int KJ, int W>
__global__ __launch_bounds__(256) void route_combine_grad_kernel(const TD* __restrict__ dy,
                                                                 const TR* __restrict__ rows,
                                                                 const int32_t* __restrict__ position,
                                                                 const float* __restrict__ weights,
                                                                 TR* __restrict__ drows, float* __restrict__ dweights,
                                                                 int64_t t_count, int k, int c) {
  __shared__ float part[4][KJ];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, in = threadIdx.x % (64 * W);
  const int64_t t = (int64_t)blockIdx.x * (4 / W) + wave / W, s0 = t * k, n = t_count * k;
  const bool here = t < t_count;
  for (int j0 = 0; j0 < k; j0 += KJ) {
    int64_t at[KJ];
    float w[KJ], dot[KJ];
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
      const int p = here && j0 + j < k ? position[s0 + j0 + j] : -1;
      const bool live = (uint64_t)(int64_t)p < (uint64_t)n;
      at[j] = live ? (int64_t)p * c : -1;
      w[j] = live ? weights[s0 + j0 + j] : 0.f;
      dot[j] = 0.f;
    }
    if (here)
      for (int i0 = in * 8; i0 < c; i0 += 64 * W * 8) {
        const int count = min(8, c - i0);
        float d[8];
        from_bits(load_bits<TD, Loose>(dy, t * c + i0, count, t_count * c), d);
#pragma unroll
        for (int j = 0; j < KJ; ++j)
          if (at[j] >= 0) {
            float v[8];
            from_bits(load_bits<TR, Loose>(rows, at[j] + i0, count, n * c), v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              dot[j] = __builtin_fmaf(d[i], v[i], dot[j]);  // (past the row's end both are zero)
              v[i] = w[j] * d[i];
            }
            store_bits<TR, Loose>(drows, at[j] + i0, count, to_bits<TR>(v));
          }
      }
    wave_reduce_dpp<KJ>(dot);
    if (lane == 63)
#pragma unroll
      for (int j = 0; j < KJ; ++j) part[wave][j] = dot[j];
    __syncthreads();
    if (here && in < KJ && j0 + in < k) {
      const int w0 = wave / W * W;
      float sum = part[w0][in];
#pragma unroll
      for (int i = 1; i < W; ++i) sum += part[w0 + i][in];
      dweights[s0 + j0 + in] = sum;
    }
    __syncthreads();
  }
}

// f(element of type `dtype`), f(Int<rows start at any element>).
template <typename F>
static hipError_t with_type(int dtype, F&& f) {
  if (dtype == kF32) return f(float{});
  if (dtype == kF16) return f(_Float16{});
  return f(__bf16{});
}
template <typename F>
static hipError_t with_rows(int64_t c, F&& f) {
  return c % 8 == 0 ? f(Int<0>{}) : f(Int<1>{});
}
hipError_t launch_route_gather(const void* x, const int32_t* order, const float* weights, void* out, int dtype,
                               int64_t t, int64_t k, int64_t c, hipStream_t s) {
  const int64_t n = t * k;
  return with_type(dtype, [&](auto type) {
    typedef decltype(type) T;
    return with_rows(c, [&](auto lc) {
      constexpr bool Loose = decltype(lc)::value != 0;
      const dim3 grid((unsigned)route_move_workgroups(n, c));
      if (weights)
        hipLaunchKernelGGL((route_gather_kernel<T, Loose, true>), grid, dim3(256), 0, s, (const T*)x, order, weights,
                           (T*)out, n, (int)k, (int)c, t * c);
      else
        hipLaunchKernelGGL((route_gather_kernel<T, Loose, false>), grid, dim3(256), 0, s, (const T*)x, order, weights,
                           (T*)out, n, (int)k, (int)c, t * c);
      return hipGetLastError();
    });
  });
}

hipError_t launch_route_combine(const void* rows, int rows_dtype, const int32_t* position, const float* weights,
                                void* y, int y_dtype, int64_t t, int64_t k, int64_t c, hipStream_t s) {
  return with_type(rows_dtype, [&](auto rt) {
    typedef decltype(rt) TR;
    return with_type(y_dtype, [&](auto yt) {
      typedef decltype(yt) TY;
      return with_rows(c, [&](auto lc) {
        constexpr bool Loose = decltype(lc)::value != 0;
        hipLaunchKernelGGL((route_combine_kernel<TR, TY, Loose>), dim3((unsigned)route_move_workgroups(t, c)), dim3(256), 0, s,
                           (const TR*)rows, position, weights, (TY*)y, t, (int)k, (int)c);
        return hipGetLastError();
      });
    });
  });
}

hipError_t launch_route_combine_grad(const void* dy, int dy_dtype, const void* rows, int rows_dtype,
                                     const int32_t* position, const float* weights, void* drows, float* dweights,
                                     int64_t t, int64_t k, int64_t c, hipStream_t s) {
  return with_type(dy_dtype, [&](auto dt) {
    typedef decltype(dt) TD;
    return with_type(rows_dtype, [&](auto rt) {
      typedef decltype(rt) TR;
      return with_rows(c, [&](auto lc) {
        constexpr bool Loose = decltype(lc)::value != 0;
        const auto go = [&](auto kc, auto wc) {
          constexpr int KJ = decltype(kc)::value, W = decltype(wc)::value;
          hipLaunchKernelGGL((route_combine_grad_kernel<TD, TR, Loose, KJ, W>), dim3((unsigned)route_grad_workgroups(t, c)),
                             dim3(256), 0, s, (const TD*)dy, (const TR*)rows, position, weights, (TR*)drows, dweights,
                             t, (int)k, (int)c);
          return hipGetLastError();
        };
        const auto waves = [&](auto kc) { return route_grad_waves(t, c) == 1 ? go(kc, Int<1>{}) : go(kc, Int<4>{}); };
        return k <= 2 ? waves(Int<2>{}) : waves(Int<4>{});
      });
    });
  });
}

}  // namespace qgemv
