// Low-rank adapters of many requests beside a shared projection, for gfx950:
// y[t] = c[t] + scale[e] B_e (A_e x[t]) with e the adapter that token t names
// (include/qroute.h).
//
// Two launches.  The first multiplies tiles of 16 sorted tokens by A_e, split
// over K into parts whose fp32 sums go to the workspace; the second adds the
// parts up in order, multiplies by B_e and adds c.  Both are bound by what they
// read and write: A and B once per adapter in use, x, c and y.  Where the whole
// call fits one round of workgroups (decode), each of them computes its tokens'
// A_e x itself and one launch does it all.
#include "device.hpp"
#include "epilogue.hpp"
#include "launch_route.hpp"
#include "pieces.hpp"
#include "route_plan.hpp"

namespace qgemv {

struct LoraArgs {
  const uint16_t* x;       // [t][k]
  const uint16_t* a;       // [e][r][k]
  const uint16_t* b;       // [e][m][r]
  const float* scale;      // [e] or NULL
  const int32_t* order;    // sorted position -> token
  const int32_t* offsets;  // e + 1
  const void* c;           // [t][m] or NULL
  void* y;
  float* v;                // [parts][t][r]: sums of A_e x over a part of K
  int t, e, r, m, k;
  int y_dtype;
  int parts, part_k;       // K split: part p covers [p * part_k, (p + 1) * part_k)
  int chunks;              // workgroups along r (first kernel) or m (second)
};

constexpr int kLoraDownWaves = 8;
constexpr int kLoraUpWaves = 4;
constexpr int kLoraOneWaves = 16;  // of the single launch
constexpr int kLoraMaxR = 256;
// Offset of a piece that is not there, and the largest span of y that takes offsets.
constexpr uint32_t kDeadPiece = 0xFFFFFFF0u;
constexpr int64_t kLoraMaxSpan = 0xFFFF0000;

template <bool BF>
__device__ __forceinline__ f32x4 lora_mfma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (BF)
    return mfma16_bf(a, b, c);
  else
    return mfma16(a, b, c);
}

// Sums of x[token(p)][i] * A_e[j][i] over [k_begin, k_end) for the 16 tokens of tile
// t and the 16 RT rows j0 .. of A_e, by NW waves; red[w][p][j] = wave w's share.
// The operands' rows go through LDS (16 rows x 64 bytes a copy, four lanes a row:
// a load straight into operands has a row per lane, which takes the address unit
// four times as long).  Each wave has U steps of 32 in flight in its own piece of
// `stage`; granule c of row i sits at position c ^ (i / 4), which puts one
// granule of 16 rows into 16 different bank groups.  red may be `stage`.
template <int RT, int U>
constexpr int kLoraStage = (1 + RT) * U * 1024;  // bytes per wave

template <bool BF, int RT, int NW, int U>
__device__ __forceinline__ void lora_sums(const LoraArgs& g, const RoutedTile& t, int j0, int k_begin, int k_end,
                                          unsigned char* stage, float (*red)[16][16 * RT + 4]) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, q = lane >> 4;
  const uint32_t row = (uint32_t)g.k * 2u;
  const auto xr = make_rsrc(g.x, (uint32_t)g.t * row);
  const auto ar = make_rsrc(g.a + ((int64_t)t.e * g.r + j0) * g.k, (uint32_t)min(16 * RT, g.r - j0) * row);
  const int from = lane >> 2, granule = (lane & 3) ^ ((lane >> 4) & 3);  // what the lane copies
  uint32_t xo = kDeadRow;
  if (from < t.rows) {
    const int token = g.order[t.first + from];
    if ((unsigned)token < (unsigned)g.t) xo = (uint32_t)token * row;
  }
  unsigned char* const mine = stage + wave * kLoraStage<RT, U>;
  f32x4 acc[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int k0 = k_begin + wave * 32 * U; k0 < k_end; k0 += NW * 32 * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = k0 + 32 * u + 8 * granule;
      const uint32_t at = i < k_end ? 2u * (uint32_t)i : kPfDead;
      unsigned char* const to = mine + (1 + RT) * 1024 * u;
      // (rows of no token stay as they are: they reach only their own sums, which nothing reads)
      if (from < t.rows) ld128_lds(xr, to, xo + at);
#pragma unroll
      for (int j = 0; j < RT; ++j) ld128_lds(ar, to + 1024 * (1 + j), (uint32_t)(16 * j + from) * row + at);
    }
    wait_vm<0>();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const unsigned char* const at = mine + (1 + RT) * 1024 * u + 64 * col + 16 * (q ^ (col >> 2));
      const u32x4 xv = *reinterpret_cast<const u32x4*>(at);
#pragma unroll
      for (int j = 0; j < RT; ++j)
        acc[j] = lora_mfma<BF>(xv, *reinterpret_cast<const u32x4*>(at + 1024 * (1 + j)), acc[j]);
    }
  }
  __syncthreads();  // (red may take the place of the stages)
#pragma unroll
  for (int j = 0; j < RT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][4 * q + i][16 * j + col] = acc[j][i];
  __syncthreads();
}

// v[part][p][j]: lora_sums of a part of K.  (2048 tokens, 8 adapters of r = 64, K = 4096:
// 12.5 us for 21 MB; what bounds it is A, read again for every 16 tokens.)
template <bool BF, int RT>
__global__ __launch_bounds__(64 * kLoraDownWaves) void lora_down_kernel(LoraArgs g) {
  constexpr int NW = kLoraDownWaves, kCols = 16 * RT, U = RT == 4 ? 2 : 4;
  __shared__ __attribute__((aligned(1024))) unsigned char stage[NW * kLoraStage<RT, U>];
  auto* const red = reinterpret_cast<float(*)[16][kCols + 4]>(stage);
  static_assert(sizeof(float) * NW * 16 * (kCols + 4) <= sizeof(stage), "the sums fit the stages");
  const int part = (int)(blockIdx.x % (unsigned)g.parts);
  const int rest = (int)(blockIdx.x / (unsigned)g.parts);
  const int tile = rest / g.chunks, j0 = (rest - tile * g.chunks) * kCols;
  const RoutedTile t = find_tile(g.offsets, g.e, g.t, 16, tile);
  if (t.rows == 0) return;
  lora_sums<BF, RT, NW, U>(g, t, j0, part * g.part_k, min((part + 1) * g.part_k, g.k), stage, red);
  float* const out = g.v + ((int64_t)part * g.t + t.first) * g.r + j0;
  for (int i = threadIdx.x; i < t.rows * kCols; i += 64 * NW) {
    const int tok = i / kCols, j = i % kCols;
    if (j0 + j < g.r) {
      float v = red[0][tok][j];
#pragma unroll
      for (int w = 1; w < NW; ++w) v += red[w][tok][j];
      out[(int64_t)tok * g.r + j] = v;
    }
  }
}

// y[token][0..m) of 16 TT tokens: c plus B_e times their v, 64 columns a wave
// at a time on 16x16x32 MFMAs with columns as M: a lane's results are four
// neighbouring columns of one token, and go through LDS to lanes that load c and
// store y in whole lines (eight or sixteen lanes a row).
//
// v (with scale) is kept to fp32's precision: as three bf16 terms against bf16 B
// (24 bits), and against fp16 B as three fp16 terms of v * 2^s, where s puts the
// token's largest v in [2^14, 2^15) and each term holds, times 2^12, what the terms before
// it leave over, and the terms' sums are joined by 2^-12 and 2^-s.  A term's smallest step
// is 2^-24, the third's 2^-48 of v * 2^s: an fp32 v is held bit for bit down to
// 2^-39 of the token's largest, and to 2^-63 of that below it.  (Two terms under one scale
// hold 11 bits of a v of 2^-28 of the largest; 2048 tokens, r = 64, 14336 columns of fp16:
// 47.5 us for the whole call, 49.3 with three.)
//
// 2048 tokens, 8 adapters of r = 64, 14336 columns of bf16: 37.8 us for 132 MB (3.5 TB/s),
// fp32 55 us (4.5 TB/s).  Bound by c and y; before these went through LDS in whole
// lines and each group's loads were issued a group ahead, it took 45 us.
//
// With RT > 0 (then r <= 16 RT) the workgroup computes v itself (lora_sums) instead of adding up parts.
// Loose: rows of y are not whole dwords, or reach past 32-bit offsets.
template <bool BF, typename TY, int TT, int RK, bool Loose, int RT = 0>
__global__ __launch_bounds__(64 * (RT > 0 ? kLoraOneWaves : kLoraUpWaves)) void lora_up_kernel(LoraArgs g) {
  constexpr int BT = 16 * TT, NW = RT > 0 ? kLoraOneWaves : kLoraUpWaves, kTerms = 3;
  constexpr int U = RT == 1 ? 4 : RT == 2 ? 2 : 1;
  static_assert(RT == 0 || TT == 1, "one tile of 16 tokens");
  // c and y in pieces of 16 bytes
  constexpr int kPiece = 16 / (int)sizeof(TY), kRowLanes = 64 / kPiece, kRows = 64 / kRowLanes, kPieces = BT / kRows;
  typedef Bits<TY, kPiece> Piece;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ float undo[BT];
  // the stages of lora_sums, then every wave's results of a group, [BT][64]
  constexpr int kScratch = NW * (RT > 0 && kLoraStage<RT, U> > 256 * BT ? kLoraStage<RT, U> : 256 * BT);
  __shared__ __attribute__((aligned(1024))) unsigned char scratch[kScratch];
  const int rp = (g.r + 31) / 32 * 32, stride = rp + 8;  // 16-bit elements of a token's term (padding: LDS banks)
  uint16_t* const vs = reinterpret_cast<uint16_t*>(lds);  // [kTerms][BT][stride]
  int tile, chunk;
  if constexpr (TT > 1) {  // the tiles that read one piece of B follow each other on an XCD
    const int tiles = (int)gridDim.x / g.chunks, at = xcd_walk((int)blockIdx.x, (int)gridDim.x);
    chunk = at / tiles;
    tile = at - chunk * tiles;
  } else {  // (nothing gained: 500 tokens over 60 adapters 15.2 us, 16.1 with the walk)
    tile = (int)(blockIdx.x / (unsigned)g.chunks);
    chunk = (int)blockIdx.x - tile * g.chunks;
  }
  const RoutedTile t = find_tile<true>(g.offsets, g.e, g.t, BT, tile);
  if (t.rows == 0) return;
  const bool adapted = t.e < g.e;
  const TY* const c = static_cast<const TY*>(g.c);
  TY* const y = static_cast<TY*>(g.y);
  if (!adapted && c == y) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, q = lane >> 4;
  const int pc = kPiece * (lane % kRowLanes), pr = lane / kRowLanes;  // piece p: row kRows p + pr, columns pc ..
  int64_t yrow[kPieces];
  uint32_t yoff[kPieces];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    int token = -1;
    if (kRows * p + pr < t.rows) {
      token = g.order[t.first + kRows * p + pr];
      if (!adapted) token = -1 - token;
      if ((unsigned)token >= (unsigned)g.t) token = -1;
    }
    yrow[p] = token < 0 ? -1 : (int64_t)token * g.m;
    yoff[p] = token < 0 ? kDeadPiece : (uint32_t)token * (uint32_t)g.m * (uint32_t)sizeof(TY);
  }
  // !Loose: c and y through descriptors, whose ranges keep out the pieces that are
  // not there (a piece past a row's end reads what follows and drops it), so that every group has the same number of loads and stores and
  // waits for its own loads alone (a store under a branch makes the compiler wait for
  // the stores as well)
  const uint32_t span = (uint32_t)((int64_t)g.t * g.m * (int)sizeof(TY));
  const auto cr = make_rsrc(c ? c : y, c ? span : 0u), yr = make_rsrc(y, span);
  const int groups = (g.m + 63) / 64;
  const uint32_t brow = (uint32_t)g.r * 2u;
  // c and B of a group are loaded a group ahead of their use: loads and
  // stores complete in the order they were issued, so a load asked for in the
  // group that uses it would wait for the stores before it as well
  const int step = g.chunks * NW;
  uint32_t bo[4];  // row `col` of MFMA tile i
#pragma unroll
  for (int i = 0; i < 4; ++i) bo[i] = (uint32_t)(16 * i + col) * brow;
  const auto load_b = [&](int grp, int k0, u32x4 (&f)[4]) {
    const int c0 = 64 * grp;
    const auto br = make_rsrc(g.b + ((int64_t)t.e * g.m + c0) * g.r, (uint32_t)max(0, min(64, g.m - c0)) * brow);
    const uint32_t at = k0 + 8 * q < g.r ? 2u * (uint32_t)(k0 + 8 * q) : kPfDead;
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = ld128(br, bo[i] + at);
  };
  const TY* const csrc = c ? c : y;  // (without c the loads still go somewhere, and their values are dropped)
  const auto load_c = [&](int grp, Piece (&n)[kPieces]) {
    // Loose: a piece outside y, or a row of no token, loads the first element instead
    const int at = 64 * grp + pc;
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      if constexpr (Loose) {
        const bool live = yrow[p] >= 0 && at < g.m;
        n[p] = load_bits<TY, true, kPiece>(csrc, live ? yrow[p] + at : 0, live ? min(kPiece, g.m - at) : 1,
                                             (int64_t)g.t * g.m);
      } else {
        const u32x4 v = ld128(cr, at < g.m && yoff[p] != kDeadPiece ? yoff[p] + (uint32_t)at * (uint32_t)sizeof(TY) : kDeadPiece);
        n[p] = Piece{{v.x, v.y, v.z, v.w}};
      }
    }
  };
  const auto store_c = [&](int grp, int p, const float (&r)[kPiece]) {
    const int at = 64 * grp + pc;
    const Piece out = to_bits<TY>(r);
    if constexpr (Loose) {
      if (yrow[p] >= 0 && at < g.m) store_bits<TY, true, kPiece>(y, yrow[p] + at, min(kPiece, g.m - at), out);
    } else {
      const uint32_t to = yoff[p] + (uint32_t)at * (uint32_t)sizeof(TY);
      __builtin_amdgcn_raw_buffer_store_b128(u32x4{out.w[0], out.w[1], out.w[2], out.w[3]}, yr,
                                             (int)(at + kPiece <= g.m && yoff[p] != kDeadPiece ? to : kDeadPiece), 0, 0);
      if (64 * grp + 64 > g.m && yoff[p] != kDeadPiece)  // the group that holds the row's end: single dwords of its last piece
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (at + kPiece > g.m && at + (i + 1) * (4 / (int)sizeof(TY)) <= g.m)
            __builtin_amdgcn_raw_buffer_store_b32(out.w[i], yr, (int)to, 4 * i, 0);
    }
  };
  if (!adapted) {
    for (int grp = chunk * NW + wave; grp < groups; grp += step) {
      Piece n[kPieces];
      load_c(grp, n);
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        float r[kPiece];
        from_bits(n[p], r);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) r[j] = c ? r[j] : 0.f;
        store_c(grp, p, r);
      }
    }
    return;
  }
  struct Ahead {
    u32x4 b[RK > 0 ? RK : 1][4];
    Piece c[kPieces];
  };
  const auto load_ahead = [&](int grp, Ahead& n) {
    if constexpr (RK > 0)
#pragma unroll
      for (int k = 0; k < RK; ++k) load_b(grp, 32 * k, n.b[k]);
    load_c(grp, n.c);
  };
  Ahead ahead[2];
  load_ahead(chunk * NW + wave, ahead[0]);
  const float s = g.scale ? g.scale[t.e] : 1.f;
  // kLanes neighbouring lanes take a token, four consecutive values at a time
  constexpr int kLanes = 64 * NW / BT, kQuads = kLoraMaxR / 4 / kLanes;
  const int tok = threadIdx.x / kLanes, in = threadIdx.x % kLanes;
  f32x4 v[kQuads];
#pragma unroll
  for (int i = 0; i < kQuads; ++i) v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  if constexpr (RT > 0) {
    auto* const red = reinterpret_cast<float(*)[16][16 * RT + 4]>(scratch);
    lora_sums<BF, RT, NW, U>(g, t, 0, 0, g.k, scratch, red);
    if (tok < t.rows && 4 * in < g.r)
#pragma unroll
      for (int w = 0; w < NW; ++w) v[0] += *reinterpret_cast<const f32x4*>(&red[w][tok][4 * in]);
  } else {
    // (values that are not there are loaded from the row's start, and dropped: no
    // branch between the loads, so that they are all in flight together)
    const float* const src = g.v + ((int64_t)t.first + min(tok, t.rows - 1)) * g.r;
    const int64_t part = (int64_t)g.t * g.r;
    int at[kQuads];
#pragma unroll
    for (int i = 0; i < kQuads; ++i) at[i] = 4 * (in + kLanes * i) < g.r ? 4 * (in + kLanes * i) : 0;
    for (int p = 0; p < g.parts; p += 2) {
      f32x4 w[2][kQuads];
#pragma unroll
      for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
          w[o][i] = *reinterpret_cast<const f32x4*>(src + min(p + o, g.parts - 1) * part + at[i]);
#pragma unroll
      for (int i = 0; i < kQuads; ++i)
        v[i] += p + 1 < g.parts ? w[0][i] + w[1][i] : w[0][i];
    }
#pragma unroll
    for (int i = 0; i < kQuads; ++i)
      if (tok >= t.rows || 4 * (in + kLanes * i) >= g.r) v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  float up = 1.f, top = 0.f;
#pragma unroll
  for (int i = 0; i < kQuads; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[i][j] *= s;
      const float size = __builtin_fabsf(v[i][j]);
      if (size < __builtin_inff()) top = __builtin_fmaxf(top, size);
    }
  if constexpr (!BF) {
#pragma unroll
    for (int m = kLanes / 2; m >= 1; m >>= 1) top = __builtin_fmaxf(top, shfl_xor(top, m));
    // (infinities and NaN do not count)
    const int ex = (int)((__builtin_bit_cast(unsigned, top) >> 23) & 255) - 127;
    const int sh = min(14 - ex, 126);  // at least -113
    up = __builtin_bit_cast(float, (unsigned)(127 + sh) << 23);
    if (in == 0) undo[tok] = __builtin_bit_cast(float, (unsigned)(127 - sh) << 23);
  }
#pragma unroll
  for (int i = 0; i < kQuads; ++i) {
    const int j = 4 * (in + kLanes * i);
    if (j < rp) {
#pragma unroll
      for (int k = 0; k < kTerms; ++k) {
        unsigned short b[4];  // (an infinite v is one infinite term and zeros)
#pragma unroll
        for (int l = 0; l < 4; ++l) {
          float rest = k == 0 ? v[i][l] * up : v[i][l];
          if constexpr (BF) {
            b[l] = __builtin_bit_cast(unsigned short, (__bf16)rest);
            rest = (b[l] & 0x7FFF) == 0x7F80 ? 0.f : rest - (float)__builtin_bit_cast(__bf16, b[l]);
          } else {
            b[l] = __builtin_bit_cast(unsigned short, (_Float16)rest);
            rest = (b[l] & 0x7FFF) == 0x7C00 ? 0.f : (rest - (float)__builtin_bit_cast(_Float16, b[l])) * 4096.f;
          }
          v[i][l] = rest;
        }
        *reinterpret_cast<u32x2*>(vs + (k * BT + tok) * stride + j) =
            u32x2{b[0] | (unsigned)b[1] << 16, b[2] | (unsigned)b[3] << 16};
      }
    }
  }
  __syncthreads();
  float* const mine = reinterpret_cast<float*>(scratch) + wave * BT * 64;
  const auto one_group = [&](int grp, const Ahead& now, Ahead& next) {
    load_ahead(grp + step, next);
    __builtin_amdgcn_sched_barrier(0);  // (the compiler would put them off until after the products)
    // fp16: the terms' sums are joined smallest first, each scaled to the next term.
    // With B in registers the terms are taken one after the other through one sum; B
    // that is loaded as it goes is loaded once, with a sum for each term (r = 128, 2048
    // tokens, 4096 columns: B loaded three times 57 us, three sums 38).
    constexpr int kSums = !BF && RK == 0 ? kTerms : 1;
    f32x4 acc[kSums][TT][4];
#pragma unroll
    for (int k = 0; k < kSums; ++k)
#pragma unroll
      for (int u = 0; u < TT; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[k][u][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const auto multiply = [&](int term, int k0, const u32x4 (&f)[4]) {
      auto& sum = acc[kSums > 1 ? term : 0];
#pragma unroll
      for (int u = 0; u < TT; ++u) {
        const u32x4 vf = *reinterpret_cast<const u32x4*>(vs + (term * BT + 16 * u + col) * stride + k0 + 8 * q);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[u][i] = lora_mfma<BF>(f[i], vf, sum[u][i]);
      }
    };
    if constexpr (RK > 0) {
#pragma unroll
      for (int term = kTerms - 1; term >= 0; --term) {
#pragma unroll
        for (int k = 0; k < RK; ++k) multiply(term, 32 * k, now.b[k]);
        if (!BF && term > 0)
#pragma unroll
          for (int u = 0; u < TT; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[0][u][i] *= 0x1p-12f;
      }
    } else {
      for (int k0 = 0; k0 < rp; k0 += 32) {
        u32x4 f[4];
        load_b(grp, k0, f);
#pragma unroll
        for (int term = 0; term < kTerms; ++term) multiply(term, k0, f);
      }
      if constexpr (kSums > 1)
#pragma unroll
        for (int u = 0; u < TT; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[0][u][i][j] = __builtin_fmaf(__builtin_fmaf(acc[2][u][i][j], 0x1p-12f, acc[1][u][i][j]), 0x1p-12f, acc[0][u][i][j]);
    }
    // granule i of a row of 16 sits at i ^ row: no bank conflicts
#pragma unroll
    for (int u = 0; u < TT; ++u) {
      const float un = BF ? 1.f : undo[16 * u + col];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f32x4*>(mine + (16 * u + col) * 64 + 4 * ((4 * i + q) ^ col)) = acc[0][u][i] * un;
    }
    compiler_fence();
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      float r[kPiece];
      from_bits(now.c[p], r);
#pragma unroll
      for (int h = 0; h < kPiece / 4; ++h) {
        const int row = kRows * p + pr;
        const f32x4 v = *reinterpret_cast<const f32x4*>(mine + row * 64 + 4 * ((pc / 4 + h) ^ (row & 15)));
#pragma unroll
        for (int j = 0; j < 4; ++j) r[4 * h + j] = v[j] + (c ? r[4 * h + j] : 0.f);
      }
      store_c(grp, p, r);
    }
    compiler_fence();
    __builtin_amdgcn_wave_barrier();  // (the next group's results come after every lane's reads)
  };
  for (int grp = chunk * NW + wave; grp < groups; grp += 2 * step) {
    one_group(grp, ahead[0], ahead[1]);
    if (grp + step >= groups) break;
    one_group(grp + step, ahead[1], ahead[0]);
  }
}

struct LoraPlan {
  int64_t parts, part_k;
  int rt;  // tiles of 16 rows of A per workgroup
};

static LoraPlan lora_plan(int64_t t, int64_t e, int64_t r, int64_t k) {
  LoraPlan p;
  p.rt = r > 32 ? 4 : r > 16 ? 2 : 1;
  const int64_t blocks = max_tiles(t, e, 16) * ((r + 16 * p.rt - 1) / (16 * p.rt));
  // parts of K until there are two workgroups a CU, each wave with at least a
  // round of loads
  constexpr int64_t kStep = 128 * kLoraDownWaves;
  const int64_t steps = (k + kStep - 1) / kStep;
  int64_t parts = 512 / blocks;
  if (parts > steps) parts = steps;
  if (parts < 1) parts = 1;
  p.part_k = (steps + parts - 1) / parts * kStep;
  p.parts = (k + p.part_k - 1) / p.part_k;
  return p;
}

int64_t lora_workspace(int64_t t, int64_t e, int64_t r, int64_t, int64_t k) {
  if (t == 0) return 0;
  return lora_plan(t, e, r, k).parts * t * r * 4;
}

// f(element of y's type, Int<rows of y are not whole dwords, or reach past 32-bit offsets>)
template <typename F>
static hipError_t with_y(const LoraArgs& g, F&& f) {
  const int size = g.y_dtype == kF32 ? 4 : 2;
  if (g.m * (int64_t)size % 4 != 0 || (int64_t)g.t * g.m * size > kLoraMaxSpan) {
    if (g.y_dtype == kF32) return f(float{}, Int<1>{});
    if (g.y_dtype == kF16) return f(_Float16{}, Int<1>{});
    return f(__bf16{}, Int<1>{});
  }
  if (g.y_dtype == kF32) return f(float{}, Int<0>{});
  if (g.y_dtype == kF16) return f(_Float16{}, Int<0>{});
  return f(__bf16{}, Int<0>{});
}

// Work items: at most 2^20 + 2^10 tiles of 16 tokens (t <= 2^24, e <= 1024) times 4 pieces
// of r times 512 threads for the first product, parts of K and chunks of m only while
// tiles are few: below 2^32.
template <bool BF>
static hipError_t launch_lora(LoraArgs g, const LoraPlan& p, hipStream_t s) {
  const size_t row_lds = (size_t)3 * ((g.r + 31) / 32 * 32 + 8) * 2;  // bytes of a token's v
  // One launch where it takes at most a workgroup a CU and reading the adapter's
  // whole A in each of them costs less than the second launch: r is small (24
  // tokens, r = 16, 4096 x 4096: at the time 9.0 us of GPU time against 8.4 with two, but
  // 9.1 against 11.8 a call of a program whose own launches bound it), or all
  // columns are one workgroup's and A is small (1000 tokens, r = 72, 117 x 416: 9.1 us
  // against 13.4; 200 tokens, r = 128, 512 x 1024: 11.7 and 12.3; but 24 tokens, r = 64, 4096 x
  // 4096: 19.6 and 11.5).
  const int64_t tiles16 = max_tiles(g.t, (int64_t)g.e + 1, 16);
  const int64_t one_chunks = ((int64_t)g.m + 64 * kLoraOneWaves - 1) / (64 * kLoraOneWaves);
  const bool small_a = g.r <= 128 && one_chunks == 1 && (int64_t)g.r * g.k <= 1 << 17;
  if ((g.r <= 32 || small_a) && tiles16 * one_chunks <= 256) {
    g.chunks = (int)one_chunks;
    const auto one = [&](auto rc, auto kc) {
      return with_y(g, [&](auto type, auto lc) {
        hipLaunchKernelGGL((lora_up_kernel<BF, decltype(type), 1, decltype(kc)::value, decltype(lc)::value != 0, decltype(rc)::value>),
                           dim3((unsigned)(tiles16 * one_chunks)), dim3(64 * kLoraOneWaves), 16 * row_lds, s, g);
        return hipGetLastError();
      });
    };
    return g.r <= 16   ? one(Int<1>{}, Int<1>{})
           : g.r <= 32 ? one(Int<2>{}, Int<1>{})
           : g.r <= 64 ? one(Int<4>{}, Int<2>{})
                       : one(Int<8>{}, Int<0>{});
  }
  const auto down = [&](auto rc) {
    constexpr int RT = decltype(rc)::value;
    g.chunks = (g.r + 16 * RT - 1) / (16 * RT);
    hipLaunchKernelGGL((lora_down_kernel<BF, RT>), dim3((unsigned)(max_tiles(g.t, g.e, 16) * g.chunks * g.parts)),
                       dim3(64 * kLoraDownWaves), 0, s, g);
  };
  if (p.rt == 4)
    down(Int<4>{});
  else if (p.rt == 2)
    down(Int<2>{});
  else
    down(Int<1>{});
  const auto up = [&](auto tc, auto kc) {
    constexpr int TT = decltype(tc)::value, BT = 16 * TT;
    const int64_t tiles = max_tiles(g.t, (int64_t)g.e + 1, BT);
    // workgroups for two a CU, each with at least 64 columns a wave
    int64_t chunks = 512 / tiles;
    const int64_t most = ((int64_t)g.m + 64 * kLoraUpWaves - 1) / (64 * kLoraUpWaves);
    if (chunks > most) chunks = most;
    if (chunks < 1) chunks = 1;
    g.chunks = (int)chunks;
    return with_y(g, [&](auto type, auto lc) {
      hipLaunchKernelGGL((lora_up_kernel<BF, decltype(type), TT, decltype(kc)::value, decltype(lc)::value != 0>),
                         dim3((unsigned)(tiles * chunks)), dim3(64 * kLoraUpWaves), BT * row_lds, s, g);
      return hipGetLastError();
    });
  };
  // tiles of 32 tokens read B half as often, where adapters have that many and
  // their v leaves room for two workgroups a CU (2048 tokens, r = 64, 14336 columns,
  // before c and y went through LDS: 46 us; 60 us with 16, and 51 us with 64, which
  // leaves too few waves on a CU); B is read ahead into registers up to r = 64 (r =
  // 128 so, 2048 tokens, 4096 columns: 29 us, 23 without)
  if (g.t >= 32 * (int64_t)(g.t < g.e ? g.t : g.e) && g.r <= 128)
    return g.r <= 32 ? up(Int<2>{}, Int<1>{}) : g.r <= 64 ? up(Int<2>{}, Int<2>{}) : up(Int<2>{}, Int<0>{});
  return g.r <= 32 ? up(Int<1>{}, Int<1>{}) : g.r <= 64 ? up(Int<1>{}, Int<2>{}) : up(Int<1>{}, Int<0>{});
}

hipError_t launch_lora(bool bf16, const void* x, const void* a, const void* b, const float* scale,
                       const int32_t* order, const int32_t* offsets, const void* c, void* y, int y_dtype, int64_t t,
                       int64_t e, int64_t r, int64_t m, int64_t k, void* ws, hipStream_t s) {
  const LoraPlan p = lora_plan(t, e, r, k);
  const LoraArgs g{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(a), static_cast<const uint16_t*>(b),
                   scale, order, offsets, c, y, static_cast<float*>(ws), (int)t, (int)e, (int)r, (int)m, (int)k,
                   y_dtype, (int)p.parts, (int)p.part_k, 0};
  return bf16 ? launch_lora<true>(g, p, s) : launch_lora<false>(g, p, s);
}

}  // namespace qgemv
