// Routed products for gfx950: y[p] = x[row(p)] . dequant(W_e)^T for the rows p
// that a plan (include/qroute.h) gives to each weight set e, on packed Q4_K,
// NVFP4 and TQ1_0 matrices.
//
// Kernels, chosen by the number of rows and tiles (routed_plan):
//  - few rows (decode), or too few tiles for the CUs: every wave streams its own
//    weight rows through LDS and decodes them straight into matrix-core operands,
//    once per 16 rows (routed_rows_kernel);
//  - many rows (prefill) of NVFP4 and TQ1_0, whose weights are exact in 16 bits:
//    decoded once per tile of tokens into LDS, with the prefill's loop
//    (routed_tile_kernel);
//  - many rows of Q4_K, whose weights are not (a 16-bit weight is off by up to 2^-11
//    of itself): the first kernel's arithmetic with 64 tokens a workgroup
//    (routed_q4k_kernel).
#include <type_traits>

#include "device.hpp"
#include "epilogue.hpp"
#include "launch_route.hpp"
#include "prefill_tile.hpp"
#include "route_plan.hpp"

namespace qgemv {

// What one launch works on.
struct RoutedArgs {
  const uint8_t* w;        // [e_count] packed matrices of `expert_bytes` bytes
  const uint16_t* x;
  const int32_t* order;    // sorted position -> slot, or NULL: row p of x
  const int32_t* offsets;  // e_count + 1
  void* y;
  int64_t expert_bytes;
  int n;        // slots
  int choices;  // slots per token
  int e_count;
  int m, k;
  int t_count;
  int y_dtype;
  int groups;  // workgroups along the weight rows: workgroup b is group b % groups of tile b / groups
};

// Uniform offset of a unit that is not there: beyond every descriptor's range by
// itself and with what a lane adds to it (at most kPfDead, or two dead rows).
constexpr uint32_t kDeadUnit = 0x60000000u;

// Byte offset of tile row i's activations in the descriptor of x_rsrc.
__device__ __forceinline__ uint32_t x_offset(const RoutedArgs& a, const RoutedTile& t, int i) {
  if (i >= t.rows) return kDeadRow;
  if (!a.order) return (uint32_t)i * (uint32_t)a.k * 2u;
  const int slot = a.order[t.first + i];
  return (unsigned)slot < (unsigned)a.n ? (uint32_t)(slot / a.choices) * (uint32_t)a.k * 2u : kDeadRow;
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t x_rsrc(const RoutedArgs& a, const RoutedTile& t) {
  if (a.order) return make_rsrc(a.x, (uint32_t)a.t_count * (uint32_t)a.k * 2u);
  return make_rsrc(a.x + (int64_t)t.first * a.k, (uint32_t)t.rows * (uint32_t)a.k * 2u);
}

// ---- few rows -------------------------------------------------------------------
//
// v_mfma_f32_16x16x32_{f16,bf16}: A[m][k] at lane m + 16 (k / 8) element k % 8,
// B[k][n] at lane n + 16 (k / 8) element k % 8, D[m][n] at lane n + 16 (m / 4)
// register m % 4.  Tokens are M, weight rows N, so a lane's B operands all come
// from one weight row, and the order of K is free as long as A and B agree: the
// lane takes a contiguous piece of its row's packed block and decodes it in
// place.
//
// A wave takes 16 weight rows, in units of 256 weights of K.  Everything goes
// through LDS in whole lines: a load straight into operands has a row per lane,
// and the address unit then takes 64 cycles a load instead of 16 (such a kernel
// stayed at 3.3 TB/s, whatever it decoded).  Functor F:
//   staged, copy   the wave's copies of a stage of packed bytes, global -> LDS;
//   store_x        brings 8 activations of one token into operand order and LDS;
//   read_x, read   A operands and one weight row's packed bytes of a unit, from LDS;
//   mma            decodes them and adds the unit's products to acc.
// `g` is lane / 16.

// (e0 e1)(e2 e3)(e4 e5)(e6 e7) -> (e0 e2)(e1 e3)(e4 e6)(e5 e7): the order in which
// masking even and odd bytes of a dword yields them.
__device__ __forceinline__ u32x4 even_odd(u32x4 v) {
  return u32x4{__builtin_amdgcn_perm(v.y, v.x, 0x05040100u), __builtin_amdgcn_perm(v.y, v.x, 0x07060302u),
               __builtin_amdgcn_perm(v.w, v.z, 0x05040100u), __builtin_amdgcn_perm(v.w, v.z, 0x07060302u)};
}

// LDS offset of lane (token, g)'s 16 bytes of A operand s of a unit: operands of
// 1 KiB, whose 16 tokens are permuted by s and g so that the threads that store
// one token's pieces hit different banks (a read takes all 16 in any order).  Of
// the permutations tried (TQ1_0, 74 slots of 4096 x 14336 / Q4_K, one token of 14336 x
// 4096): none 61.9 / 16.8 us, by s alone 56.8 / 16.8, s + 8 (g % 2) 55.1 / 17.4, this
// one 53.1 / 16.8.
__device__ __forceinline__ int x_frag(int s, int g, int token) {
  return 1024 * s + 256 * g + 16 * (token ^ ((s + 2 * g) & 15));
}

// ld128_lds_s, reading zeros when !live (uniform).
__device__ __forceinline__ void ld128_lds_live(__amdgpu_buffer_rsrc_t r, void* lds, uint32_t voff, uint32_t soff,
                                               bool live) {
  ld128_lds_s(r, lds, voff, live ? soff : kDeadUnit);
}

// Copies chunk c = 64 i + lane (c < Chunks, 16 bytes each) to lds + 16 c; at[i] is
// the lane's source offset.  The last copy runs on the lanes that it needs, so
// that nothing past the chunks is written.
template <int Chunks, int N>
__device__ __forceinline__ void copy_chunks(__amdgpu_buffer_rsrc_t r, unsigned char* lds, const uint32_t (&at)[N],
                                            uint32_t soff, bool live) {
  static_assert(N == (Chunks + 63) / 64, "copies");
#pragma unroll
  for (int i = 0; i < Chunks / 64; ++i) ld128_lds_live(r, lds + 1024 * i, at[i], soff, live);
  if constexpr (Chunks % 64 != 0)
    if ((int)(threadIdx.x & 63) < Chunks % 64) ld128_lds_live(r, lds + 1024 * (Chunks / 64), at[Chunks / 64], soff, live);
}

__device__ __forceinline__ unsigned bf16_bits(float v) {
  return (unsigned)__builtin_bit_cast(unsigned short, (__bf16)v);
}

// Q4_K: lane g takes qs bytes 32 g .. + 32 of the block, whose low nibbles are
// group 2 g and whose high nibbles are group 2 g + 1.  The exact integers
// scale * q (at most 63 * 15, as multiples of 2^-14 in fp16) are multiplied on the
// matrix cores and d * 2^14 is applied to the fp32 sums of the block: weights are
// not rounded.
// The mins need sum_g min_g X_g with X_g the group's activation sum in fp32:
// one bf16 MFMA, X_g split into three bf16 terms (24 bits) in the K slots of
// its lane, against min_g (6 bits, exact).
struct Q4kRows {
  static constexpr bool kDefinition = true;
  static constexpr int kUnit = 256;
  static constexpr bool kWholeUnits = true;
  struct X {
    u32x4 f[8];
    u32x4 sums;
  };
  struct Desc {
    __amdgpu_buffer_rsrc_t r;
  };
  struct Raw {
    u32x4 hdr, q0, q1;
  };
  static __device__ __forceinline__ Desc desc(const uint8_t* w, int, int k, int n0, int nv) {
    const uint32_t rb = (uint32_t)(k / 256 * 144);
    return Desc{make_rsrc(w + (int64_t)n0 * rb, (uint32_t)nv * rb)};
  }
  // the sums of two groups as the K slots of min_0 (3), min_1 (3) and nothing (2)
  static __device__ __forceinline__ u32x4 split_sums(float s0, float s1) {
    unsigned b[2][3];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v = h ? s1 : s0;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        b[h][i] = bf16_bits(v);
        v -= __builtin_bit_cast(float, b[h][i] << 16);
      }
    }
    return u32x4{b[0][0] | b[0][1] << 16, b[0][2] | b[1][0] << 16, b[1][1] | b[1][2] << 16, 0u};
  }
  // A nibble masked in place is an fp16 subnormal, q * 2^-24 (low) or q * 2^-20
  // (high); times scale * 2^10 or scale * 2^6 it is scale * q * 2^-14, at most
  // 945 * 2^-14 and a multiple of 2^-14: exact, and a normal number for the
  // matrix cores.
  // What a unit of one weight row is scaled by: both groups' scales as fp16 pairs, the
  // mins as the K slots of split_sums, and d * 2^14 and dmin of the block.
  struct Scales {
    f16x2 a0, a1;
    u32x4 mins;
    float d, dmin;
  };
  static __device__ __forceinline__ Scales scales(const Raw& raw, int g) {
    // 6-bit scales and mins of groups 2 g and 2 g + 1, as bytes 0 and 1
    const bool hi = g >= 2;
    const unsigned sh = 16u * (unsigned)(g & 1), shm = hi ? sh + 4u : sh;
    const unsigned ma = hi ? 0x0F0Fu : 0x3F3Fu, mb = hi ? 0x3030u : 0u;
    const unsigned sa = hi ? raw.hdr.w : raw.hdr.y, na = hi ? raw.hdr.w : raw.hdr.z;
    const unsigned sc = ((sa >> sh) & ma) | ((raw.hdr.y >> (sh + 2u)) & mb);
    const unsigned mn = ((na >> shm) & ma) | ((raw.hdr.z >> (sh + 2u)) & mb);
    // both scales as fp16: 1024 + scale under the exponent of 1024, minus 1024
    const f16x2 s2 = (as_h2(__builtin_amdgcn_perm(0x64646464u, sc, 0x04010400u)) + f16x2{-1024, -1024}) * f16x2{1024, 64};
    // mins as bf16: the upper halves of the (exact) fp32 values
    const unsigned m0 = __builtin_bit_cast(unsigned, (float)(mn & 0xFFu));
    const unsigned m1 = __builtin_bit_cast(unsigned, (float)((mn >> 8) & 0xFFu));
    return Scales{f16x2{s2.x, s2.x}, f16x2{s2.y, s2.y},
                  u32x4{__builtin_amdgcn_perm(m0, m0, 0x07060302u), __builtin_amdgcn_perm(m1, m0, 0x07060302u),
                        __builtin_amdgcn_perm(m1, m1, 0x07060302u), 0u},
                  f16lo(raw.hdr.x) * 16384.f, f16hi(raw.hdr.x)};
  }
  // B operands of qs bytes 8 s .. + 8 of the lane's 32: low nibbles (x operand s)
  // and high ones (operand 4 + s)
  static __device__ __forceinline__ void weights(const Raw& raw, const Scales& sc, int s, u32x4& lo, u32x4& hi) {
    const u32x4 v = s < 2 ? raw.q0 : raw.q1;
    const unsigned b0 = s % 2 ? v.z : v.x, b1 = s % 2 ? v.w : v.y;
    const auto low = [&](unsigned b) { return __builtin_bit_cast(unsigned, as_h2(b & 0x000F000Fu) * sc.a0); };
    const auto high = [&](unsigned b) { return __builtin_bit_cast(unsigned, as_h2(b & 0x00F000F0u) * sc.a1); };
    lo = u32x4{low(b0), low(b0 >> 8), low(b1), low(b1 >> 8)};
    hi = u32x4{high(b0), high(b0 >> 8), high(b1), high(b1 >> 8)};
  }
  // One output by the definition, sum of (d * scale * q - dmin * min) * x.
  static __device__ __forceinline__ float definition(const uint8_t* row, const uint16_t* x, int k) {
    float sum = 0.f;
    for (int b = 0; b < k / 256; ++b) {
      const uint8_t* const blk = row + 144 * (int64_t)b;
      const u32x4 hdr = *reinterpret_cast<const u32x4*>(blk);
      const float d = f16lo(hdr.x), dmin = f16hi(hdr.x);
      for (int g = 0; g < 8; ++g) {
        const unsigned sh = 8u * (unsigned)(g & 3), lo = hdr.y >> sh, mid = hdr.z >> sh, hi = hdr.w >> sh;
        const unsigned sc = g < 4 ? lo & 63u : (hi & 15u) | ((lo >> 2) & 48u);
        const unsigned mn = g < 4 ? mid & 63u : ((hi >> 4) & 15u) | ((mid >> 2) & 48u);
        const float ds = d * (float)sc, least = dmin * (float)mn;
        for (int i = 0; i < 32; ++i) {
          const unsigned q = ((unsigned)blk[16 + 32 * (g >> 1) + i] >> (4 * (g & 1))) & 15u;
          const float v = (float)__builtin_bit_cast(_Float16, x[256 * b + 32 * g + i]);
          sum = __builtin_fmaf(__builtin_fmaf(ds, (float)q, -least), v, sum);
        }
        if (sum != sum) return sum;  // (and stays NaN)
      }
    }
    return sum;
  }
  static __device__ __forceinline__ void mma(const Raw& raw, const X& x, int g, f32x4& acc) {
    const Scales sc = scales(raw, g);
    f32x4 q = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u32x4 lo, hi;
      weights(raw, sc, s, lo, hi);
      q = mfma16(x.f[s], lo, q);
      q = mfma16(x.f[4 + s], hi, q);
    }
    const f32x4 least = mfma16_bf(x.sums, sc.mins, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(sc.d, q[i], __builtin_fmaf(-sc.dmin, least[i], acc[i]));
  }

  // Staged: a unit's 144-byte blocks of 16 rows, row after row, so that a
  // wave's copies are contiguous but for one gap a row; 16 rows' pieces at one
  // offset then lie in 16 different bank groups.
  static constexpr int kStageUnits = 1;
  static constexpr int kXBytes = 9 * 1024;  // eight operands and the group sums
  static constexpr int kCopies = 3;
  static constexpr int kStage = 16 * 144;  // bytes
  struct Staged {
    uint32_t at[kCopies];
  };
  static __device__ __forceinline__ Staged staged(const Desc&, int k, int lane) {
    Staged st;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int c = 64 * i + lane, r = c / 9;
      st.at[i] = (uint32_t)r * (uint32_t)(k / 256 * 144) + 16u * (uint32_t)(c % 9);
    }
    return st;
  }
  static __device__ __forceinline__ void copy(const Desc& d, const Staged& st, unsigned char* lds, int stage, bool live) {
    copy_chunks<144>(d.r, lds, st.at, 144u * (uint32_t)stage, live);
  }
  // weight row r of the wave, unit `unit` of the stage
  static __device__ __forceinline__ Raw read(const Desc&, const unsigned char* lds, int, int r, int g, int, int) {
    const unsigned char* const b = lds + 144 * r;
    return Raw{*reinterpret_cast<const u32x4*>(b), *reinterpret_cast<const u32x4*>(b + 16 + 32 * g),
               *reinterpret_cast<const u32x4*>(b + 32 + 32 * g)};
  }
  // 16-byte granule j of a unit of one token (elements 8 j .. + 8), for the wave's
  // 64 threads' (token, j): lane t holds j = t % 32
  // their sum over the granule's group of 32, in all four lanes that hold it
  static __device__ __forceinline__ float group_sum(u32x4 v) {
    float s = dot2h(v.x, 0x3C003C00u, dot2h(v.y, 0x3C003C00u, dot2h(v.z, 0x3C003C00u, dot2h(v.w, 0x3C003C00u, 0.f))));
    s += dpp_xor1(s);
    s += dpp_xor2(s);
    return s;
  }
  static __device__ __forceinline__ void store_x(unsigned char* xs, int token, int j, u32x4 v) {
    const float s = group_sum(v), t = shfl_xor(s, 4);
    *reinterpret_cast<u32x4*>(xs + x_frag(j & 7, j >> 3, token)) = even_odd(v);
    if ((j & 7) == 0) *reinterpret_cast<u32x4*>(xs + x_frag(8, j >> 3, token)) = split_sums(s, t);
  }
  static __device__ __forceinline__ void read_x(const unsigned char* xs, int col, int g, X& x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x.f[i] = *reinterpret_cast<const u32x4*>(xs + x_frag(i, g, col));
    x.sums = *reinterpret_cast<const u32x4*>(xs + x_frag(8, g, col));
  }
};

// NVFP4: lane g takes 64 weights, 32 nibble bytes and 4 scale bytes; e2m1 *
// |scale| is exact in bf16.
struct Nvfp4Rows {
  static constexpr bool kDefinition = false;
  static constexpr int kUnit = 256;
  static constexpr bool kWholeUnits = false;
  struct X {
    u32x4 f[8];
  };
  struct Desc {
    __amdgpu_buffer_rsrc_t nib, sc;
  };
  struct Raw {
    u32x4 q0, q1;
    unsigned sc;
  };
  static __device__ __forceinline__ Desc desc(const uint8_t* w, int m, int k, int n0, int nv) {
    const uint32_t nr = (uint32_t)(k / 2), sr = (uint32_t)(k / 16);
    return Desc{make_rsrc(w + (int64_t)n0 * nr, (uint32_t)nv * nr),
                make_rsrc(w + (int64_t)m * nr + (int64_t)n0 * sr, (uint32_t)nv * sr)};
  }
  static __device__ __forceinline__ void mma(const Raw& raw, const X& x, int, f32x4& acc) {
    const unsigned v[8] = {raw.q0.x, raw.q0.y, raw.q0.z, raw.q0.w, raw.q1.x, raw.q1.y, raw.q1.z, raw.q1.w};
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const float sc = __builtin_fabsf(s / 2 == 0   ? __builtin_amdgcn_cvt_f32_fp8((int)raw.sc, 0)
                                       : s / 2 == 1 ? __builtin_amdgcn_cvt_f32_fp8((int)raw.sc, 1)
                                       : s / 2 == 2 ? __builtin_amdgcn_cvt_f32_fp8((int)raw.sc, 2)
                                                    : __builtin_amdgcn_cvt_f32_fp8((int)raw.sc, 3));
      u32x4 b;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x2 e = fp4x2_f32(v[s], i);
        // exact products of 6 significant bits: the upper halves are the bf16 codes
        b[i] = __builtin_amdgcn_perm(__builtin_bit_cast(unsigned, e.y * sc), __builtin_bit_cast(unsigned, e.x * sc),
                                     0x07060302u);
      }
      acc = mfma16_bf(x.f[s], b, acc);
    }
  }

  // Staged: a unit of 16 rows: 128 nibble bytes a row, whose 16-byte granules
  // are permuted by the row (rows are a multiple of the banks apart), then 16
  // scale bytes a row.
  static constexpr int kStageUnits = 1;
  static constexpr int kXBytes = 8 * 1024;  // eight operands
  static constexpr int kCopies = 3;
  static constexpr int kStage = 16 * 144;  // bytes
  struct Staged {
    uint32_t at[2], sc[1];
  };
  static __device__ __forceinline__ Staged staged(const Desc&, int k, int lane) {
    Staged st;
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // copy i: rows 8 i ..
      const int r = 8 * i + (lane >> 3);
      st.at[i] = (uint32_t)r * (uint32_t)(k / 2) + 16u * (uint32_t)((lane ^ r) & 7);
    }
    st.sc[0] = (uint32_t)lane * (uint32_t)(k / 16);
    return st;
  }
  static __device__ __forceinline__ void copy(const Desc& d, const Staged& st, unsigned char* lds, int stage, bool live) {
    copy_chunks<128>(d.nib, lds, st.at, 128u * (uint32_t)stage, live);
    copy_chunks<16>(d.sc, lds + 2048, st.sc, 16u * (uint32_t)stage, live);
  }
  static __device__ __forceinline__ Raw read(const Desc&, const unsigned char* lds, int, int r, int g, int u, int k) {
    const unsigned char* const b = lds + 128 * r;
    const unsigned sc = *reinterpret_cast<const unsigned*>(lds + 2048 + 16 * r + 4 * g);
    // (past the end of K the copies hold the next row's bytes, or zeros: finite
    // nibbles, and scales that are taken as zero)
    return Raw{*reinterpret_cast<const u32x4*>(b + 16 * ((2 * g) ^ (r & 7))),
               *reinterpret_cast<const u32x4*>(b + 16 * ((2 * g + 1) ^ (r & 7))), 256 * u + 64 * g < k ? sc : 0u};
  }
  static __device__ __forceinline__ void store_x(unsigned char* xs, int token, int j, u32x4 v) {
    *reinterpret_cast<u32x4*>(xs + x_frag(j & 7, j >> 3, token)) = v;
  }
  static __device__ __forceinline__ void read_x(const unsigned char* xs, int col, int g, X& x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x.f[i] = *reinterpret_cast<const u32x4*>(xs + x_frag(i, g, col));
  }
};

// TQ1_0: lane g takes qs bytes 4 g .. + 4 and 16 + 4 g .. + 4 (digit k feeds elements
// 32 k + 4 g .. and 32 k + 16 + 4 g ..; the 16 rows' dwords at these bytes lie in
// all 64 banks), bytes 32 + 4 g .. + 4 (digit k: elements 160 + 16 k + 4 g ..) and digit g of the
// four qh bytes (elements 240 + 4 g ..).  Digits come from the recurrence
// L = 3 L mod 256, digit = 3 L / 256, on two bytes at a time; digit - 1 is
// exact in fp16 and d is applied to the fp32 sums of the block.
struct Tq1Rows {
  static constexpr bool kDefinition = true;
  static constexpr int kUnit = 256;
  static constexpr bool kWholeUnits = true;
  struct X {
    u32x4 f[8];
  };
  struct Desc {
    __amdgpu_buffer_rsrc_t r;
    uint32_t lead;
    int last;               // the last row
    unsigned short last_d;  // and its last block's d
  };
  struct Raw {
    // the dwords that hold qs bytes 4 g .. + 4, 16 + 4 g .. + 4 and 32 + 4 g .. + 4, and the qh bytes
    u32x2 a0, a1, b, c;
    unsigned short d;
    uint32_t shift;
  };
  static __device__ __forceinline__ Desc desc(const uint8_t* w, int, int k, int n0, int nv) {
    const uint32_t rb = (uint32_t)(k / 256 * 54);
    const uint8_t* const first = w + (int64_t)n0 * rb;
    const uint32_t lead = (uint32_t)reinterpret_cast<uintptr_t>(first) & 3u;
    const uint32_t bytes = (uint32_t)nv * rb;
    return Desc{make_rsrc(first - lead, nv > 0 ? (bytes + lead) & ~3u : 0u), lead, nv - 1,
                ld16(make_rsrc(first, bytes), bytes - 2u)};
  }
  static __device__ __forceinline__ uint32_t row_offset(int k, int r) { return (uint32_t)r * (uint32_t)(k / 256 * 54); }
  // one output by the definition, sum of (d * (digit - 1)) * x
  static __device__ __forceinline__ float definition(const uint8_t* row, const uint16_t* x, int k) {
    float sum = 0.f;
    for (int b = 0; b < k / 256; ++b) {
      const uint8_t* const blk = row + 54 * (int64_t)b;
      const float d = (float)__builtin_bit_cast(_Float16, *reinterpret_cast<const unsigned short*>(blk + 52));
      for (int e = 0; e < 256; ++e) {
        const int at = e < 160 ? e % 32 : e < 240 ? 32 + e % 16 : 48 + e % 4;
        const int dg = e < 160 ? e / 32 : e < 240 ? (e - 160) / 16 : (e - 240) / 4;
        const unsigned l = (unsigned)blk[at] * pow3_u16(dg) & 255u;
        const float v = (float)__builtin_bit_cast(_Float16, x[256 * b + e]);
        sum = __builtin_fmaf(d * (float)((int)(3u * l >> 8) - 1), v, sum);
        if (sum != sum) return sum;  // (and stays NaN)
      }
    }
    return sum;
  }
  // fp16 codes of digit - 1 of the two bytes in the halves of l; l moves to the next digit
  static __device__ __forceinline__ unsigned digit(unsigned& l) {
    const unsigned p = __builtin_bit_cast(unsigned, __builtin_bit_cast(u16x2, l) * u16x2{3, 3});
    l = p & 0x00FF00FFu;
    const f16x2 t = as_h2(__builtin_amdgcn_perm(0x64646464u, p, 0x04030401u));  // 1024 + digit
    return __builtin_bit_cast(unsigned, t + f16x2{-1025, -1025});
  }
  static __device__ __forceinline__ void mma(const Raw& raw, const X& x, int g, f32x4& acc) {
    const unsigned a0 = __builtin_amdgcn_alignbyte(raw.a0.y, raw.a0.x, raw.shift);
    const unsigned a1 = __builtin_amdgcn_alignbyte(raw.a1.y, raw.a1.x, raw.shift);
    const unsigned b = __builtin_amdgcn_alignbyte(raw.b.y, raw.b.x, raw.shift);
    const unsigned h = __builtin_amdgcn_alignbyte(raw.c.y, raw.c.x, raw.shift);
    const float d = (float)__builtin_bit_cast(_Float16, raw.d);
    f32x4 q = {0.f, 0.f, 0.f, 0.f};
    unsigned l0 = a0 & 0x00FF00FFu, l1 = (a0 >> 8) & 0x00FF00FFu, l2 = a1 & 0x00FF00FFu, l3 = (a1 >> 8) & 0x00FF00FFu;
#pragma unroll
    for (int s = 0; s < 5; ++s) {
      const unsigned w0 = digit(l0), w1 = digit(l1), w2 = digit(l2), w3 = digit(l3);
      q = mfma16(x.f[s], u32x4{w0, w1, w2, w3}, q);
    }
    unsigned e = b & 0x00FF00FFu, o = (b >> 8) & 0x00FF00FFu;
#pragma unroll
    for (int s = 5; s < 7; ++s) {
      const unsigned w0 = digit(e), w1 = digit(o), w2 = digit(e), w3 = digit(o);
      q = mfma16(x.f[s], u32x4{w0, w1, w2, w3}, q);
    }
    const unsigned short p = pow3_u16(g);
    const u16x2 pp = {p, p};
    unsigned he = __builtin_bit_cast(unsigned, __builtin_bit_cast(u16x2, h & 0x00FF00FFu) * pp) & 0x00FF00FFu;
    unsigned ho = __builtin_bit_cast(unsigned, __builtin_bit_cast(u16x2, (h >> 8) & 0x00FF00FFu) * pp) & 0x00FF00FFu;
    const unsigned w0 = digit(e), w1 = digit(o), w2 = digit(he), w3 = digit(ho);
    q = mfma16(x.f[7], u32x4{w0, w1, w2, w3}, q);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(d, q[i], acc[i]);
  }

  // Staged: two units of 16 rows, per row the 112 bytes from the dword at or
  // below the two blocks' first byte (108 bytes and up to 2 before them), which
  // 16 rows put in 16 different bank groups.  A dword partly past the last row's end
  // is not read (the matrix may end there), and the d in it is loaded by itself.
  static constexpr int kStageUnits = 2;
  static constexpr int kXBytes = 8 * 1024;  // eight operands
  static constexpr int kCopies = 2;
  static constexpr int kStage = 16 * 112;  // bytes
  struct Staged {
    uint32_t at[kCopies];
  };
  static __device__ __forceinline__ Staged staged(const Desc& d, int k, int lane) {
    Staged st;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int c = 64 * i + lane, r = c / 7;
      st.at[i] = ((d.lead + row_offset(k, r)) & ~3u) + 16u * (uint32_t)(c % 7);
    }
    return st;
  }
  static __device__ __forceinline__ void copy(const Desc& d, const Staged& st, unsigned char* lds, int stage, bool live) {
    copy_chunks<112>(d.r, lds, st.at, 108u * (uint32_t)stage, live);
  }
  static __device__ __forceinline__ Raw read(const Desc& d, const unsigned char* lds, int unit, int row, int g, int u,
                                             int k) {
    const uint32_t blk = ((d.lead + row_offset(k, row)) & 2u) + 54u * (uint32_t)unit;  // in the row's 112 bytes
    const unsigned char* const b = lds + 112 * row + (blk & ~3u);
    const auto dword = [&](int at) { return *reinterpret_cast<const unsigned*>(b + at); };
    Raw r;
    r.a0 = u32x2{dword(4 * g), dword(4 * g + 4)};
    r.a1 = u32x2{dword(16 + 4 * g), dword(20 + 4 * g)};
    r.b = u32x2{dword(32 + 4 * g), dword(36 + 4 * g)};
    r.c = u32x2{dword(48), dword(52)};
    const unsigned short own = *reinterpret_cast<const unsigned short*>(lds + 112 * row + blk + 52);
    r.d = row == (u == k / 256 - 1 ? d.last : -1) ? d.last_d : own;
    r.shift = blk & 3u;
    return r;
  }
  // granules 0 .. 19: digit j / 4 of qs bytes 8 (j % 4) .. + 8; 20 ..: digit k = (j - 20) / 2
  // of bytes 32 .. 47 (then of qh), half of its 16 elements.  Four elements each
  // go to lanes g and g + 1.
  static __device__ __forceinline__ void store_x(unsigned char* xs, int token, int j, u32x4 v) {
    const u32x4 p = even_odd(v);
    const int k = (j - 20) >> 1, s = j < 20 ? j >> 2 : 5 + (k >> 1), h = j < 20 ? (j >> 1) & 1 : k & 1, g = 2 * (j & 1);
    *reinterpret_cast<u32x2*>(xs + x_frag(s, g, token) + 8 * h) = u32x2{p.x, p.y};
    *reinterpret_cast<u32x2*>(xs + x_frag(s, g + 1, token) + 8 * h) = u32x2{p.z, p.w};
  }
  static __device__ __forceinline__ void read_x(const unsigned char* xs, int col, int g, X& x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x.f[i] = *reinterpret_cast<const u32x4*>(xs + x_frag(i, g, col));
  }
};

// Q4_K and TQ1_0 apply a block's scales to its sum.  Where an activation or a scale is infinite
// that is not what the definition gives: 0 * inf and inf - inf are NaN, and the
// infinite scale of a zero weight is NaN only in the definition.  An output that is not finite
// is therefore computed again by the definition, on one lane, up to where it is NaN: one infinite
// activation adds 180 us to a call with K = 4096 of Q4_K, 3 ms with 14336 of TQ1_0; where
// all activations are NaN, 2048 tokens x 2 of 14336 x 4096 take 2.5 ms.

__device__ __forceinline__ bool finite(float v) { return __builtin_fabsf(v) < __builtin_inff(); }

// Stores output (tile row i, weight row `row`) again as F's definition gives it.
template <typename F>
__device__ __forceinline__ void store_definition(const RoutedArgs& a, const RoutedTile& t, int i, int row) {
  int64_t at = t.first + i;
  if (a.order) {
    const int slot = a.order[at];
    if ((unsigned)slot >= (unsigned)a.n) return;
    at = slot / a.choices;
  }
  const float v = F::definition(a.w + t.e * a.expert_bytes + row * (a.expert_bytes / a.m), a.x + at * a.k, a.k);
  store_y(a.y, a.y_dtype, (int64_t)(t.first + i) * a.m + row, v);
}

// A workgroup takes 16 RW weight rows, 16 a wave, times KW parts of K whose sums
// meet in LDS at the end.  A wave copies its rows' packed bytes global -> LDS two
// stages ahead.  The threads of a K part load the 16 tokens' activations two
// stages ahead into registers, bring them into operand order (with the group
// sums) and store them to LDS once for all its waves, one unit ahead of their
// use, in two buffers: one barrier a unit.
//
// Measured: Q4_K, one token through two sets of 14336 x 4096 in 16.8 us (66 MB, 3.9 TB/s,
// a launch's start included); NVFP4, 64 tokens x 8 over 64 sets of 1024 x 4096 in 40.8
// us (3.7 TB/s); TQ1_0, 74 slots over 8 sets of 4096 x 14336 in 50 to 57 us by box, of
// which its VALU instructions (digits, mostly) are 31 by themselves and the rest operand
// reads from LDS and barriers that nothing covers.
constexpr int kStRing = 3;

template <typename F, int RW, int KW>
__global__ __launch_bounds__(64 * RW * KW, RW * KW == 4 ? 3 : 2) void routed_rows_kernel(RoutedArgs a) {
  constexpr int BT = 16, NW = RW * KW, SU = F::kStageUnits;
  constexpr int kStage = F::kStage, kXUnit = F::kXBytes;
  constexpr int XG = 8 / RW;  // 16-byte granules of a unit per thread
  __shared__ __attribute__((aligned(256))) unsigned char ws0[NW * kStage];
  __shared__ __attribute__((aligned(256))) unsigned char ws1[NW * kStage];
  __shared__ __attribute__((aligned(256))) unsigned char ws2[NW * kStage];
  __shared__ __attribute__((aligned(256))) unsigned char xs[KW * 2 * kXUnit];
  const int tile = (int)(blockIdx.x / (unsigned)a.groups), group = (int)blockIdx.x - tile * a.groups;
  const RoutedTile t = find_tile(a.offsets, a.e_count, a.n, BT, tile);
  if (t.rows == 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rw = wave % RW, kw = wave / RW;
  const int col = lane & 15, g = lane >> 4;
  const int n0 = (group * RW + rw) * 16;
  const int units = (a.k + F::kUnit - 1) / F::kUnit, stages = (units + SU - 1) / SU;
  const int rounds = (stages + KW - 1) / KW;  // part kw takes stages kw, kw + KW, ..
  const auto wd = F::desc(a.w + t.e * a.expert_bytes, a.m, a.k, n0, max(0, min(16, a.m - n0)));
  const auto st = F::staged(wd, a.k, lane);
  const auto ring = [&](int i) { return (i % 3 == 0 ? ws0 : i % 3 == 1 ? ws1 : ws2) + wave * kStage; };

  // granule j of tokens 2 RW h + (thread of the part) / 32
  const auto xr = x_rsrc(a, t);
  const int token = 2 * rw + (lane >> 5), j = lane & 31;
  unsigned char* const xmine = xs + kw * 2 * kXUnit;
  uint32_t xo[XG];
#pragma unroll
  for (int h = 0; h < XG; ++h) xo[h] = x_offset(a, t, 2 * RW * h + token) + 16u * (uint32_t)j;
  u32x4 xq[kStRing][SU][XG];
  const auto load = [&](int round, u32x4 (&q)[SU][XG], unsigned char* lds) {
    const int s = round * KW + kw;
#pragma unroll
    for (int v = 0; v < SU; ++v) {
      const int u = SU * s + v;
      // (K ends on a unit but for NVFP4, whose rows then end on a granule)
      const uint32_t cut = F::kWholeUnits || 256 * u + 8 * j < a.k ? 0u : kDeadRow;
#pragma unroll
      for (int h = 0; h < XG; ++h) q[v][h] = ld128s(xr, xo[h] + cut, u < units ? 512u * (uint32_t)u : kDeadUnit);
    }
    compiler_fence();
    F::copy(wd, st, lds, s, s < stages);
    compiler_fence();
  };
  // a unit's activations into buffer b; tokens that are not there stay zero
  const auto store_x = [&](int b, const u32x4 (&q)[XG]) {
#pragma unroll
    for (int h = 0; h < XG; ++h)
      if (2 * RW * h + 2 * rw < t.rows) F::store_x(xmine + b * kXUnit, 2 * RW * h + token, j, q[h]);
  };
  for (int i = threadIdx.x; i < KW * 2 * kXUnit / 16; i += 64 * NW) reinterpret_cast<u32x4*>(xs)[i] = u32x4{0u, 0u, 0u, 0u};
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};

  constexpr int kStageLoads = XG * SU + F::kCopies;
#pragma unroll
  for (int i = 0; i < kStRing - 1; ++i) load(i, xq[i], ring(i));
  lds_barrier();  // the zeros
  store_x(0, xq[0][0]);
  int buf = 0;
  for (int i0 = 0; i0 < rounds; i0 += kStRing) {
    static_for<0, kStRing>([&](auto ic) {
      constexpr int I = decltype(ic)::value;
      constexpr int N1 = (I + 1) % kStRing, N2 = (I + 2) % kStRing;  // N2: read last in the round before
      const int i = i0 + I;
      load(i + 2, xq[N2], ring(N2));
      wait_vm<(kStRing - 1) * kStageLoads>();  // this wave's copies of round i are in
      if (i < rounds) {
#pragma unroll
        for (int v = 0; v < SU; ++v) {
          lds_barrier();  // this unit's activations are in, and the other buffer has been read
          store_x(buf ^ 1, v + 1 < SU ? xq[I][v + 1 < SU ? v + 1 : 0] : xq[N1][0]);
          const int u = SU * (i * KW + kw) + v;
          if (u < units) {
            typename F::X x;
            F::read_x(xmine + buf * kXUnit, col, g, x);
            F::mma(F::read(wd, ring(I), v, col, g, u, a.k), x, g, acc);
          }
          buf ^= 1;
        }
      }
    });
  }
  wait_vm<0>();  // (no copy outlives the workgroup's LDS)
  if constexpr (KW > 1) {
    lds_barrier();
    f32x4* const sums = reinterpret_cast<f32x4*>(xs);
    if (kw > 0) sums[((kw - 1) * RW + rw) * 64 + lane] = acc;
    lds_barrier();
    if (kw > 0) return;
#pragma unroll
    for (int p = 0; p < KW - 1; ++p) acc += sums[(p * RW + rw) * 64 + lane];
  }
  unsigned again = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (4 * g + i < t.rows && n0 + col < a.m) {
      store_y(a.y, a.y_dtype, (int64_t)(t.first + 4 * g + i) * a.m + n0 + col, acc[i]);
      again |= finite(acc[i]) ? 0u : 1u << i;
    }
  if constexpr (F::kDefinition)
    for (; again; again &= again - 1) store_definition<F>(a, t, 4 * g + __builtin_ctz(again), n0 + col);
}

// ---- many rows, Q4_K -----------------------------------------------------------------
//
// The arithmetic of Q4kRows with 64 tokens a workgroup, so that weights are decoded once
// for 64 rows: a wave takes 32 weight rows and multiplies them with every 16
// tokens' operands, which the workgroup's 8 waves read from LDS.  No weight is rounded:
// scale * q is exact in fp16, and the sums of a block are scaled by its d and its mins
// subtracted in fp32.
//
// While a unit is multiplied, its successor's packed bytes are copied to LDS and read
// into registers at the unit's end; the activations go from registers, loaded a unit
// ahead, into operand order in the other of two LDS buffers.  One barrier a unit.
//
// Q4_K, 2048 tokens x 2 over 8 sets of 14336 x 4096: 700 to 725 us (0.67 PFLOP/s of the
// weights' own products; eight qgemm_q4k calls of 512 rows each, whose weights are
// rounded, take 590 to 650), bound by issue: 370 VALU instructions (decoding 200,
// activations and their sums 75, scaling 64) and 72 MFMAs a unit and wave.  With weights
// rounded to fp16 in LDS and tiles of 256 x 256 the same took 615 us, but 24 to 64 rows of
// each of the sets took 117 to 160 us, 83 to 139 like this.  Tiles of 96 tokens: 719 us, but 128 us
// against 101 for 512 rows of one set; 48 weight rows a wave: 728, 133; 16 waves of 16
// rows: 788, 104.
__global__ __launch_bounds__(64 * kQ4kWaves, 2) void routed_q4k_kernel(RoutedArgs a) {
  typedef Q4kRows F;
  constexpr int BT = kQ4kBT, TT = BT / 16, RW = kQ4kWaves, NR = kQ4kBN / (16 * RW);
  constexpr int XG = 8 * TT / RW;  // granules of a unit per thread
  static_assert(XG == 4, "a quad's four lanes hold the sums of a thread's four tokens");
  constexpr int kStage = NR * F::kStage, kChunks = NR * 144, kCopies = (kChunks + 63) / 64;
  __shared__ __attribute__((aligned(256))) unsigned char ws[RW * kStage];
  __shared__ __attribute__((aligned(256))) unsigned char xs[2 * TT * F::kXBytes];
  const int tile = (int)(blockIdx.x / (unsigned)a.groups), group = (int)blockIdx.x - tile * a.groups;
  const RoutedTile t = find_tile(a.offsets, a.e_count, a.n, BT, tile);
  if (t.rows == 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int n0 = (group * RW + wave) * 16 * NR;
  const int units = a.k / 256;
  const auto wd = F::desc(a.w + t.e * a.expert_bytes, a.m, a.k, n0, max(0, min(16 * NR, a.m - n0)));
  uint32_t wo[kCopies];
#pragma unroll
  for (int i = 0; i < kCopies; ++i) {
    const int c = 64 * i + lane, r = c / 9;
    wo[i] = (uint32_t)r * (uint32_t)(a.k / 256 * 144) + 16u * (uint32_t)(c % 9);
  }
  unsigned char* const mine = ws + wave * kStage;
  const auto copy_w = [&](int u) {
    copy_chunks<kChunks>(wd.r, mine, wo, 144u * (uint32_t)u, u < units);
    compiler_fence();
  };
  const auto xr = x_rsrc(a, t);
  const int token = 2 * wave + (lane >> 5), j = lane & 31;  // of 2 RW tokens a round
  uint32_t xo[XG];
#pragma unroll
  for (int h = 0; h < XG; ++h) xo[h] = x_offset(a, t, 2 * RW * h + token) + 16u * (uint32_t)j;
  u32x4 xq[XG];
  const auto load_x = [&](int u, int h) { xq[h] = ld128s(xr, xo[h], u < units ? 512u * (uint32_t)u : kDeadUnit); };
  float sum;  // of the group that lane j % 4 = h of each four holds for token h
  const auto store_x = [&](int u, int h) {
    const int i = 2 * RW * h + token;
    const float v = F::group_sum(xq[h]);
    *reinterpret_cast<u32x4*>(xs + ((u & 1) * TT + (i >> 4)) * F::kXBytes + x_frag(j & 7, j >> 3, i & 15)) = even_odd(xq[h]);
    sum = h == 0 || (j & 3) == h ? v : sum;
  };
  const auto store_sums = [&](int u) {  // (both halves of eight lanes write the same)
    const int i = 2 * RW * (j & 3) + token;
    const float other = shfl_xor(sum, 4);
    *reinterpret_cast<u32x4*>(xs + ((u & 1) * TT + (i >> 4)) * F::kXBytes + x_frag(8, j >> 3, i & 15)) =
        F::split_sums(j & 4 ? other : sum, j & 4 ? sum : other);
  };
  typename F::Raw raw[NR];
  const auto read_w = [&]() {
#pragma unroll
    for (int r = 0; r < NR; ++r) raw[r] = F::read(wd, mine, 0, 16 * r + col, g, 0, a.k);
  };
  f32x4 acc[TT][NR];
#pragma unroll
  for (int i = 0; i < TT; ++i)
#pragma unroll
    for (int r = 0; r < NR; ++r) acc[i][r] = f32x4{0.f, 0.f, 0.f, 0.f};

  copy_w(0);
#pragma unroll
  for (int h = 0; h < XG; ++h) load_x(0, h);
#pragma unroll
  for (int h = 0; h < XG; ++h) {
    store_x(0, h);
    load_x(1, h);
  }
  store_sums(0);
  wait_vm<XG>();
  read_w();
  lds_barrier();
  const auto run = [&](auto nc) {
    constexpr int NT = decltype(nc)::value;
    for (int u = 0; u < units; ++u) {
      // the packed bytes of this unit are in registers
      copy_w(u + 1);
      const unsigned char* const xu = xs + (u & 1) * TT * F::kXBytes;
      f32x4 q[NT][NR];
      typename F::Scales sc[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) sc[r] = F::scales(raw[r], g);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        u32x4 lo[NR], hi[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) F::weights(raw[r], sc[r], s, lo[r], hi[r]);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const u32x4 x0 = *reinterpret_cast<const u32x4*>(xu + i * F::kXBytes + x_frag(s, g, col));
          const u32x4 x1 = *reinterpret_cast<const u32x4*>(xu + i * F::kXBytes + x_frag(4 + s, g, col));
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            q[i][r] = mfma16(x0, lo[r], s == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : q[i][r]);
            q[i][r] = mfma16(x1, hi[r], q[i][r]);
          }
        }
        // the next unit's activations, and loads of the one after it
#pragma unroll
        for (int h = s * XG / 4; h < (s + 1) * XG / 4; ++h) {
          store_x(u + 1, h);
          load_x(u + 2, h);
        }
      }
      store_sums(u + 1);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const u32x4 xsum = *reinterpret_cast<const u32x4*>(xu + i * F::kXBytes + x_frag(8, g, col));
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const f32x4 least = mfma16_bf(xsum, sc[r].mins, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[i][r][v] = __builtin_fmaf(sc[r].d, q[i][r][v], __builtin_fmaf(-sc[r].dmin, least[v], acc[i][r][v]));
        }
      }
      wait_vm<XG>();  // the copy (the activations' loads came after it)
      read_w();
      lds_barrier();
    }
  };
  if (t.rows > BT / 2)
    run(Int<TT>{});
  else
    run(Int<TT / 2>{});
  wait_vm<0>();  // (no copy outlives the workgroup's LDS)
  unsigned again = 0;  // bit 4 NR i + NR v + r: outputs to compute again
  static_assert(4 * TT * NR <= 32, "a bit for each of a lane's outputs");
#pragma unroll
  for (int i = 0; i < TT; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int tok = 16 * i + 4 * g + v;
      if (tok < t.rows) {
        const int64_t at = (int64_t)(t.first + tok) * a.m + n0 + col;
#pragma unroll
        for (int r = 0; r < NR; ++r)
          if (n0 + 16 * r + col < a.m) {
            store_y(a.y, a.y_dtype, at + 16 * r, acc[i][r][v]);
            again |= finite(acc[i][r][v]) ? 0u : 1u << (4 * NR * i + NR * v + r);
          }
      }
    }
  for (; again; again &= again - 1) {
    const int b = __builtin_ctz(again);
    store_definition<F>(a, t, 16 * (b / (4 * NR)) + 4 * g + b / NR % 4, n0 + 16 * (b % NR) + col);
  }
}

// ---- many rows --------------------------------------------------------------------

// Tile t of at most BT tokens times the 128 NB weight rows of `group`, on
// stages as for prefill_loop.
template <typename F, int BT, int NB, int XS>
__device__ __forceinline__ void routed_tile(const RoutedArgs& a, const RoutedTile& t, int group, unsigned char* xs0,
                                            unsigned char* xs1, unsigned char* xs2, unsigned char* ws0,
                                            unsigned char* ws1) {
  typedef PfShape<BT, NB> S;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = group * kPfBN * NB;
  const auto wd = F::desc(a.w + t.e * a.expert_bytes, a.m, a.k, n0, min(kPfBN * NB, a.m - n0));
  const auto xr = x_rsrc(a, t);
  constexpr int C = S::kCopies;
  uint32_t xo[C];
#pragma unroll
  for (int j = 0; j < C; ++j)
    xo[j] = x_offset(a, t, 8 * (C * wave + j) + (lane >> 3)) + pf_granule(lane, (C * wave + j) & 1);
  auto copy = [&](unsigned char* stage, uint32_t so) {
#pragma unroll
    for (int j = 0; j < C; ++j) ld128_lds_s(xr, stage + 8 * (C * wave + j) * kPfRowB, xo[j], so);
  };
  f32x16 acc[S::kMI][S::kNJ];
  prefill_loop<F, BT, XS, NB>(wd, copy, a.k, a.k / kPfKS, 0, xs0, xs1, xs2, ws0, ws1, acc);
  wait_vm<0>();  // (no copy outlives the workgroup's LDS)
  // D[m][n] of an MFMA tile: see prefill.hip
  const int wt = S::tokens(wave), wn = S::rows(wave);
#pragma unroll
  for (int i = 0; i < S::kMI; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int tok = wt + 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
      if (tok < t.rows) {
        const int64_t at = (int64_t)(t.first + tok) * a.m;
#pragma unroll
        for (int j = 0; j < S::kNJ; ++j) {
          const int c = n0 + wn + 32 * j + (lane & 31);
          if (c < a.m) store_y(a.y, a.y_dtype, at + c, acc[i][j][r]);
        }
      }
    }
}

// Tiles of 64 tokens x 128 weight rows, or of 256 x 256; a weight set's last tile
// of 256 may have few tokens, and runs as one of 64 or 128 when it has no more (48 rows
// in each of 32 sets of 4096 x 4096: NVFP4 165 us, 172 without the 64; TQ1_0 175, 188).
// Bound as the prefill is, by the matrix cores' operands through LDS: 2048 tokens x 2
// over 8 sets of 14336 x 4096 in 525 us (NVFP4, 0.92 PFLOP/s) and 615 us (TQ1_0, whose digits
// take longer); eight qgemm_* calls of 512 rows each take 604 and 638.
template <typename F, int BT, int NB>
__global__ __launch_bounds__(64 * kPfWaves, BT == 64 ? 2 : 1) void routed_tile_kernel(RoutedArgs a) {
  typedef PfShape<BT, NB> S;
  constexpr int XS = BT == 64 ? 3 : 2;
  __shared__ __attribute__((aligned(1024))) unsigned char xs0[S::kXTile];
  __shared__ __attribute__((aligned(1024))) unsigned char xs1[S::kXTile];
  __shared__ __attribute__((aligned(1024))) unsigned char xs2[XS == 3 ? S::kXTile : 16];
  __shared__ __attribute__((aligned(1024))) unsigned char ws0[S::kWTile];
  __shared__ __attribute__((aligned(1024))) unsigned char ws1[S::kWTile];
  const int tile = (int)(blockIdx.x / (unsigned)a.groups), group = (int)blockIdx.x - tile * a.groups;
  const RoutedTile t = find_tile(a.offsets, a.e_count, a.n, BT, tile);
  if (t.rows == 0) return;
  if constexpr (BT == 256) {
    if (t.rows <= 64) {
      routed_tile<F, 64, NB, XS>(a, t, group, xs0, xs1, xs2, ws0, ws1);
      return;
    }
    if (t.rows <= 128) {
      routed_tile<F, 128, NB, XS>(a, t, group, xs0, xs1, xs2, ws0, ws1);
      return;
    }
  }
  routed_tile<F, BT, NB, XS>(a, t, group, xs0, xs1, xs2, ws0, ws1);
}

template <typename FR, typename FT>
static hipError_t launch_routed(int fmt, RoutedArgs a, hipStream_t s) {
  const RoutedPlan p = routed_plan(fmt, a.n, a.e_count, a.m);
  a.groups = (int)p.groups;
  const dim3 grid((unsigned)(p.groups * p.tiles)), block((unsigned)p.threads);
  const auto rows = [&](auto rw, auto kw) {
    hipLaunchKernelGGL((routed_rows_kernel<FR, decltype(rw)::value, decltype(kw)::value>), grid, block, 0, s, a);
    return hipGetLastError();
  };
  if (p.kernel == kRoutedRows)
    return p.rw == 2   ? rows(Int<2>{}, Int<4>{})
           : p.kw == 2 ? rows(Int<4>{}, Int<2>{})
                       : rows(Int<4>{}, Int<1>{});
  if constexpr (std::is_same<FT, Q4kRows>::value) {
    hipLaunchKernelGGL(routed_q4k_kernel, grid, block, 0, s, a);
  } else {
    static_assert(kPfWaves == 8, "threads of a tile's workgroup");
    if (p.bt == 64)
      hipLaunchKernelGGL((routed_tile_kernel<FT, 64, 1>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((routed_tile_kernel<FT, 256, 2>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

hipError_t launch_routed(int fmt, const void* w, const void* x, const int32_t* order, const int32_t* offsets, void* y,
                         int y_dtype, int64_t t, int64_t choices, int64_t e, int64_t m, int64_t k, int64_t expert_bytes,
                         hipStream_t s) {
  const RoutedArgs a{static_cast<const uint8_t*>(w), static_cast<const uint16_t*>(x), order, offsets, y, expert_bytes,
                     (int)(t * choices), (int)choices, (int)e, (int)m, (int)k, (int)t, y_dtype, 0};
  if (fmt == kRouteQ4k) return launch_routed<Q4kRows, Q4kRows>(fmt, a, s);
  if (fmt == kRouteNvfp4) return launch_routed<Nvfp4Rows, Nvfp4Prefill>(fmt, a, s);
  return launch_routed<Tq1Rows, Tq1Tile<true>>(fmt, a, s);
}

}  // namespace qgemv
