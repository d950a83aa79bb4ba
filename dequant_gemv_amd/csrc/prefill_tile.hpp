// The tile of a many-row product on packed weights: the formats' weight steps
// (packed bytes to 16-bit MFMA inputs) and the K loop of one workgroup, whose
// caller copies the activations and stores the sums.  Used by the prefill
// (prefill.hip, which describes the work split and the lane layouts) and by the
// routed products (routed.hip).
#pragma once
#include "device.hpp"
#include "launch.hpp"
#include "prefill_plan.hpp"

namespace qgemv {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kPfRowB = 128;  // LDS bytes per tile row per step (64 16-bit values)
constexpr int kPfWTile = kPfBN * kPfRowB;  // 16 KiB of weights per stage
constexpr int kPfWaves = 8;

// A load whose step lies past the end of the K range starts at this offset,
// which is beyond every descriptor's range (each covers < 2^31 bytes): it
// reads zero without touching memory.
constexpr uint32_t kPfDead = 0x80000000u;

// LDS byte offset of 16-byte granule g (0..7) of tile row t.  Rows are 128
// bytes, so the 256-byte bank space of the LDS holds two: the granules of a
// row pair are permuted by (t / 2) % 8, and any 16 consecutive rows put a
// given granule in 16 different 16-byte bank groups (a fragment read of 16
// rows, or the 16 lanes of a store, is conflict-free).
__device__ __forceinline__ int pf_off(int t, int g) { return t * kPfRowB + 16 * (g ^ ((t >> 1) & 7)); }

// fp16 pair (fma(a_H, s, m), fma(b_H, s, m)), each rounded once from the
// exact value, where a_H, b_H are the fp16 values in half H of a and b:
// v_fma_mix reads an fp16 operand from either half of a register and writes
// either half of the result (the compiler forms the low write but packs the
// high one with a shift and an or).
template <int H>
__device__ __forceinline__ unsigned mix_pair(unsigned a, unsigned b, float s, float m, Int<H>) {
  unsigned d;
  if constexpr (H == 0) {
    __asm__("v_fma_mixlo_f16 %0, %1, %2, %3 op_sel_hi:[1,0,0]" : "=v"(d) : "v"(a), "v"(s), "v"(m));
    __asm__("v_fma_mixhi_f16 %0, %1, %2, %3 op_sel_hi:[1,0,0]" : "+v"(d) : "v"(b), "v"(s), "v"(m));
  } else {
    __asm__("v_fma_mixlo_f16 %0, %1, %2, %3 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(d) : "v"(a), "v"(s), "v"(m));
    __asm__("v_fma_mixhi_f16 %0, %1, %2, %3 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "+v"(d) : "v"(b), "v"(s), "v"(m));
  }
  return d;
}

// Two fp32 values -> two 16-bit codes of T (round to nearest even), packed.
template <typename T>
__device__ __forceinline__ unsigned pf_pack2(float a, float b) {
  const T lo = (T)pin_f32(a), hi = (T)pin_f32(b);
  return (unsigned)__builtin_bit_cast(unsigned short, lo) | ((unsigned)__builtin_bit_cast(unsigned short, hi) << 16);
}

// ---- per-format weight steps ------------------------------------------------
// A functor gives, for thread (row r of the tile, quarter q) and step s, the
// 16 weights [64 s + 16 q, 64 s + 16 q + 16) of the row as 8 packed 16-bit
// codes.  load() only issues loads (raw packed bytes, kLoads of them; all
// zero when `live` is false); make() does the arithmetic once they are in,
// and turns zero bytes into zero weights.  Offsets split into a per-thread
// part (voff) and a wave-uniform part (soff, an SGPR).  The four quarters of
// a row sit on neighbouring lanes, so their packed bytes are next to each
// other in a load.

// Q4_K ("Writing a high performant GEMV + dequant for Metal", sections "What
// is a weight block?" and "Kernel code"): step s is chunk c = s % 4 of block
// b = s / 4, i.e. the 32 qs bytes whose low nibbles are group 2c and whose
// high nibbles are group 2c + 1; quarter q = nibbles h = q / 2 of qs bytes
// 32 c + 16 (q % 2) .. + 16.
struct Q4kPrefill {
  using T = _Float16;
  static constexpr bool kBf16 = false;
  static constexpr int kKMultiple = 256;
  static constexpr int kLoads = 2;
  struct Desc {
    __amdgpu_buffer_rsrc_t r;  // the tile's rows
    uint32_t row_bytes;
  };
  struct Raw {
    u32x4 hdr, qs;
  };
  static __device__ __forceinline__ Desc desc(const uint8_t* w, int, int k, int n0, int nv) {
    const uint32_t rb = (uint32_t)(k / 256 * 144);
    return Desc{make_rsrc(w + (int64_t)n0 * rb, (uint32_t)nv * rb), rb};
  }
  static __device__ __forceinline__ Raw load(const Desc& d, int r, int s, int q, bool live) {
    const uint32_t ro = (uint32_t)r * d.row_bytes;
    const uint32_t so = live ? (uint32_t)(s >> 2) * 144u : kPfDead;
    Raw raw;
    raw.hdr = ld128s(d.r, ro, so);
    raw.qs = ld128s(d.r, ro + 16u * (uint32_t)(q & 1), so + 16u + 32u * (uint32_t)(s & 3));
    return raw;
  }
  // weight = d * scale * q - dmin * min, rounded once from the exact value to
  // fp16: a nibble masked in place is the fp16 subnormal q * 2^-24 (low
  // nibble) or q * 2^-20 (high nibble), exact, and one mixed-precision fma
  // (v_fma_mix) multiplies it by the fp32 d * scale * 2^24 (or 2^20), adds
  // -dmin * min and rounds once to fp16.
  static __device__ __forceinline__ void make(const Raw& raw, int s, int q, unsigned (&out)[8]) {
    const int c = s & 3;
    const unsigned h = (unsigned)q >> 1;
    // 6-bit scale and min of group 2c + h (same packing as the GEMV kernels)
    const bool hi = c >= 2;
    const unsigned sh = 16u * (unsigned)(c & 1) + 8u * h;
    const unsigned ma = hi ? 0x0Fu : 0x3Fu;
    const unsigned sa = hi ? raw.hdr.w : raw.hdr.y, mb = hi ? raw.hdr.w : raw.hdr.z;
    const unsigned sg = ((sa >> sh) & ma) | (hi ? (((raw.hdr.y >> (sh + 6)) & 3u) << 4) : 0u);
    const unsigned mg = ((mb >> (sh + (hi ? 4u : 0u))) & ma) | (hi ? (((raw.hdr.z >> (sh + 6)) & 3u) << 4) : 0u);
    // d * scale (exact in fp32: 11 x 6 significant bits) times 2^24 / 2^20
    const float ds = f16lo(raw.hdr.x) * (float)sg * (h ? 1048576.f : 16777216.f);
    const float ndm = -(f16hi(raw.hdr.x) * (float)mg);
    const unsigned mask = h ? 0x00F000F0u : 0x000F000Fu;
    const unsigned qw[4] = {raw.qs.x, raw.qs.y, raw.qs.z, raw.qs.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned a = qw[i] & mask;         // elements 4i, 4i + 2 of the 16
      const unsigned b = (qw[i] >> 8) & mask;  // elements 4i + 1, 4i + 3
      out[2 * i] = mix_pair(a, b, ds, ndm, Int<0>{});
      out[2 * i + 1] = mix_pair(a, b, ds, ndm, Int<1>{});
    }
  }
};

// NVFP4 (Mojo module "fp4_gemv"): step s, quarter q = weights [64 s + 16 q,
// +16) of a row, one 16-weight block: 8 nibble bytes and its scale byte.
// Every e2m1 * |scale| is exact in fp32 and in bf16, so the bf16 weights are
// exact and the MFMA runs on bf16 (the activations' type).
struct Nvfp4Prefill {
  using T = __bf16;
  static constexpr bool kBf16 = true;
  static constexpr int kKMultiple = 64;
  static constexpr int kLoads = 2;
  struct Desc {
    __amdgpu_buffer_rsrc_t nib, sc;  // the tile's nibble rows, its scale rows
    uint32_t nib_row, sc_row;
  };
  struct Raw {
    u32x2 q;
    unsigned char sc;
  };
  static __device__ __forceinline__ Desc desc(const uint8_t* w, int n, int k, int n0, int nv) {
    const uint32_t nr = (uint32_t)(k / 2), sr = (uint32_t)(k / 16);
    return Desc{make_rsrc(w + (int64_t)n0 * nr, (uint32_t)nv * nr),
                make_rsrc(w + (int64_t)n * nr + (int64_t)n0 * sr, (uint32_t)nv * sr), nr, sr};
  }
  static __device__ __forceinline__ Raw load(const Desc& d, int r, int s, int q, bool live) {
    Raw raw;
    raw.q = ld64s(d.nib, (uint32_t)r * d.nib_row + 8u * (uint32_t)q, live ? 32u * (uint32_t)s : kPfDead);
    raw.sc = ld8s(d.sc, (uint32_t)r * d.sc_row + (uint32_t)q, live ? 4u * (uint32_t)s : kPfDead);
    return raw;
  }
  static __device__ __forceinline__ void make(const Raw& raw, int, int, unsigned (&out)[8]) {
    const float sc = __builtin_fabsf(__builtin_amdgcn_cvt_f32_fp8((int)raw.sc, 0));
    const unsigned q[2] = {raw.q.x, raw.q.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // byte i: weights 2i, 2i + 1
      const f32x2 e = fp4x2_f32(q[i >> 2], i);
      out[i] = pf_pack2<T>(e.x * sc, e.y * sc);
    }
  }
};

// TQ1_0 ("metal: TQ1_0 kernel performance", sections 1, 2 and "Not
// applicable"): step s covers elements [64 c, 64 c + 64) of block b = s / 4
// (c = s % 4); quarter q the 16 starting at e0 = 64 c + 16 q, which are one
// digit of 16 bytes of qs[0..31] (e0 < 160: digit e0 / 32 of bytes e0 % 32
// ..), one digit of qs[32..47] (e0 = 160 .. 224: digit (e0 - 160) / 16) or
// the four digits of qh[0..3] (e0 = 240).  The block is only 2-byte aligned,
// so the bytes are read as five aligned dwords (single-dword loads: one past
// the range reads zero and is never needed) and realigned with alignbyte; d
// is a 16-bit load.  Each weight is one of d * -1, d * 0, d * 1, exact in
// fp16: two weights' digits come from one packed 16-bit multiply and one
// byte permute picks their fp16 codes (as in the row materialisation).
// AnyBase: w may be only 2-byte aligned (an expert's matrix inside a larger
// array); otherwise the tile's first row is 4-byte aligned.
template <bool AnyBase>
struct Tq1Tile {
  using T = _Float16;
  static constexpr bool kBf16 = false;
  static constexpr int kKMultiple = 256;
  static constexpr int kLoads = 3;
  struct Desc {
    __amdgpu_buffer_rsrc_t r;  // the tile's rows (from the dword at or below their first byte)
    uint32_t row_bytes;
    uint32_t lead;  // bytes of the descriptor before the first row
  };
  struct Raw {
    unsigned wd[5];
    unsigned short d;
    unsigned char sh;  // bytes to drop at the front of the window
  };
  static __device__ __forceinline__ Desc desc(const uint8_t* w, int, int k, int n0, int nv) {
    const uint32_t rb = (uint32_t)(k / 256 * 54);
    const uint8_t* const first = w + (int64_t)n0 * rb;
    const uint32_t lead = AnyBase ? (uint32_t)reinterpret_cast<uintptr_t>(first) & 3u : 0u;
    return Desc{make_rsrc(first - lead, (uint32_t)nv * rb + lead), rb, lead};
  }
  // first byte of quarter q's window within the block
  static __device__ __forceinline__ uint32_t window(int e0) {
    return e0 < 160 ? 16u * (uint32_t)((e0 >> 4) & 1) : e0 < 240 ? 32u : 48u;
  }
  static __device__ __forceinline__ Raw load(const Desc& d, int r, int s, int q, bool live) {
    const uint32_t blk = (AnyBase ? d.lead : 0u) + (uint32_t)r * d.row_bytes + (uint32_t)(s >> 2) * 54u;
    const uint32_t a = blk + window(64 * (s & 3) + 16 * q);
    const uint32_t al = a & ~3u;
    const uint32_t dead = live ? 0u : kPfDead;  // uniform
    Raw raw;
    // the 20 bytes from the dword below the window: one dwordx4 and one
    // dword load (dword-aligned, as multi-dword buffer loads require; the
    // range check is per dword, so the dwords of a qh window that lie past
    // the tile's last row read as zero, and only its first two are used)
    const u32x4 lo = ld128s(d.r, al, dead);
    raw.wd[0] = lo.x;
    raw.wd[1] = lo.y;
    raw.wd[2] = lo.z;
    raw.wd[3] = lo.w;
    raw.wd[4] = ld32s(d.r, al, dead + 16u);
    raw.d = ld16s(d.r, blk + 52u, dead);
    raw.sh = (unsigned char)(a & 3u);
    return raw;
  }
  // weights (2 pr, 2 pr + 1) from bytes bi, bi + 1 of the window, digit k
  static __device__ __forceinline__ unsigned pair(const unsigned (&q)[4], int bi, int k, unsigned vm, unsigned vp) {
    const unsigned word = q[bi >> 2];
    const unsigned b = (unsigned)(bi & 3);
    const unsigned pr = __builtin_amdgcn_perm(0u, word, 0x0C000C00u | b | ((b + 1u) << 16));
    const u16x2 dg = tq1_digits2(__builtin_bit_cast(u16x2, pr), pow3_u16(k));
    const u16x2 sel = dg * u16x2{0x0202, 0x0202} + u16x2{0x0100, 0x0100};
    return __builtin_amdgcn_perm(vp, vm, __builtin_bit_cast(unsigned, sel));
  }
  static __device__ __forceinline__ void make(const Raw& raw, int s, int qt, unsigned (&out)[8]) {
    unsigned q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = __builtin_amdgcn_alignbyte(raw.wd[j + 1], raw.wd[j], raw.sh);
    const float d = (float)__builtin_bit_cast(_Float16, raw.d);
    const unsigned vm = pf_pack2<T>(d * -1.f, d * 0.f);  // codes of d*(t-1), t = 0, 1
    const unsigned vp = pf_pack2<T>(d * 1.f, 0.f);        // and t = 2
    const int e0 = 64 * (s & 3) + 16 * qt;
    if (e0 < 240) {  // one digit of 16 consecutive bytes (lanes differ only in steps with c = 3)
      const int k = e0 < 160 ? e0 >> 5 : (e0 - 160) >> 4;
#pragma unroll
      for (int p = 0; p < 8; ++p) out[p] = pair(q, 2 * p, k, vm, vp);
    } else {  // element 240 + 4 k + m is digit k of qh[m]
#pragma unroll
      for (int p = 0; p < 8; ++p) out[p] = pair(q, (2 * p) & 3, p >> 1, vm, vp);
    }
  }
};
using Tq1Prefill = Tq1Tile<false>;

// ---- the kernel ---------------------------------------------------------------

constexpr int kPfWQ = 3;      // packed-weight register slots: loads run kPfWQ - 1 steps ahead of the decode
static_assert(kPfUnroll % kPfWQ == 0, "steps per loop iteration: a multiple of the weight register slots");

// Step s, with XS activation stages: the activations of step s + XS - 1 are
// copied into activation stage (s + XS - 1) % XS and the packed weights of
// step s + 3 are loaded into registers; the weights of step s + 1 (loaded
// during step s - 2) are decoded, the MFMAs consume activation stage s % XS
// and weight stage s % 2, and the decoded weights go to weight stage
// (s + 1) % 2.
// Before the step's barrier each wave waits for its own copy of step s + 1's
// activations (an LDS copy by one wave is read by all), so every copy has
// XS - 1 steps to land.  The stages are separate LDS arrays indexed at
// compile time (the loop runs kPfUnroll steps per iteration): the compiler
// then knows that the copies in flight into one stage never alias the
// fragment reads of another, and does not wait for them there.
// Shape of a tile of BT tokens x 128 NB weight rows for 8 waves.
template <int BT, int NB = 1>
struct PfShape {
  static_assert(BT == 64 || (NB == 1 && BT == 512) || (NB == 2 && BT == 128) || BT == 256, "tokens per tile");
  static_assert(NB == 1 || NB == 2, "weight rows per tile");
  static constexpr int kWT = BT == 64 || NB == 2 ? 2 : 4;  // waves along the tokens
  static constexpr int kWN = kPfWaves / kWT;               // waves along the weight rows
  static constexpr int kMI = BT / (32 * kWT);              // 32-token MFMA tiles per wave
  static constexpr int kNJ = kPfBN * NB / (32 * kWN);      // 32-row MFMA tiles per wave
  static constexpr int kXTile = BT * kPfRowB;              // bytes of activations per stage
  static constexpr int kWTile = NB * kPfWTile;             // bytes of weights per stage
  static constexpr int kCopies = BT / 64;                  // 1 KiB activation copies per wave per step
  // first token and weight row of a wave's sub-tile
  static __device__ __forceinline__ int tokens(int wave) { return 32 * kMI * (wave % kWT); }
  static __device__ __forceinline__ int rows(int wave) { return 32 * kNJ * (wave / kWT); }
};

// Activation copy: wave v copies tile rows 8C v .. 8C v + 8C - 1 of a step in
// C = kCopies wave-wide loads of 8 rows; lane i of load j lands at LDS row
// t = 8C v + 8 j + i / 8, position i % 8, which holds granule (i % 8) ^
// ((t / 2) % 8) = (i % 8) ^ (i / 16) ^ (4 if C v + j is odd) of the row.
__device__ __forceinline__ uint32_t pf_granule(int lane, int odd) {
  return 16u * (uint32_t)((lane & 7) ^ (lane >> 4) ^ (odd ? 4 : 0));
}

// The K loop of one workgroup's tile: K split z (steps [z * split_steps, ...)),
// weight rows described by wd, with XS activation stages in the LDS arrays
// xs0..xs2 (at least BT * 128 bytes each, xs2 used when XS = 3) and the weight
// stages ws0, ws1.  copy(stage, so) issues this wave's kCopies activation
// copies of the step whose bytes start so bytes into each row (zeros when so
// is kPfDead).  The sums are left in acc.
template <typename F, int BT, int XS, int NB = 1, typename Copy>
__device__ __forceinline__ void prefill_loop(const typename F::Desc& wd, Copy&& copy, int k, int split_steps, int z,
                                             unsigned char* xs0, unsigned char* xs1, unsigned char* xs2,
                                             unsigned char* ws0, unsigned char* ws1,
                                             f32x16 (&acc)[PfShape<BT, NB>::kMI][PfShape<BT, NB>::kNJ]) {
  typedef PfShape<BT, NB> S;
  constexpr int kPfXS = XS;                       // activation stages
  constexpr int kPfMI = S::kMI, kPfNJ = S::kNJ, kPfCopies = S::kCopies;
  static_assert(XS == 2 || XS == 3, "two or three activation stages");
  static_assert(kPfXS * S::kXTile + 2 * S::kWTile <= 160 * 1024, "activation and weight stages fit the LDS");
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // K split z: steps [z * split_steps, ...) of the K / 64 steps
  const int s_begin = z * split_steps;
  const int steps = min(split_steps, k / kPfKS - s_begin);
  auto copy_x = [&](unsigned char* stage, int s) {
    copy(stage, s < steps ? (uint32_t)(s_begin + s) * 128u : kPfDead);  // uniform
  };

  // Weight decode: thread i takes weights [16 dq, 16 dq + 16) of weight rows
  // dr + 128 b of each step.
  const int dr = tid >> 2, dq = tid & 3;
  auto store_w = [&](unsigned char* stage, int b, const unsigned (&v)[8]) {  // rows 128 b ..
#pragma unroll
    for (int g = 0; g < 2; ++g)
      *reinterpret_cast<u32x4*>(stage + b * kPfWTile + pf_off(dr, 2 * dq + g)) = u32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
  };

#pragma unroll
  for (int i = 0; i < kPfMI; ++i)
#pragma unroll
    for (int j = 0; j < kPfNJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  // wave sub-tile: tokens wt .., rows wn ..
  const int wt = S::tokens(wave), wn = S::rows(wave);
  const int fl = lane & 31, fq = lane >> 5;  // fragment row / column and k-granule
  auto xstage = [&](int m) { return m % kPfXS == 0 ? xs0 : m % kPfXS == 1 ? xs1 : xs2; };

  // Loads return in issue order, and the wait counts below count the loads
  // issued after the one waited for: per step the activation copy (4), then
  // the weights (kLoads for each block of 128 rows).
  constexpr int kWLoads = NB * F::kLoads;
  constexpr int kStepLoads = kPfCopies + kWLoads;
  // prologue: activations of steps 0 .. XS - 2, weights of steps 0 .. 2; step 0 decoded
  // Each group is fenced: the compiler may otherwise interleave independent
  // loads, and a weight load issued after a copy would let part of the copy
  // still be in flight when the count is reached.
  typename F::Raw wq[kPfWQ][NB];
  auto load_w = [&](typename F::Raw (&q)[NB], int s) {
#pragma unroll
    for (int b = 0; b < NB; ++b) q[b] = F::load(wd, dr + 128 * b, s_begin + s, dq, s < steps);
  };
  copy_x(xs0, 0);
  compiler_fence();
  load_w(wq[0], 0);
  compiler_fence();
  if constexpr (kPfXS == 3) {
    copy_x(xs1, 1);
    compiler_fence();
  }
  load_w(wq[1], 1);
  compiler_fence();
  load_w(wq[2], 2);
  compiler_fence();
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    unsigned v[8];
    F::make(wq[0][b], s_begin, dq, v);
    store_w(ws0, b, v);
  }
  // this wave's copy of step 0's activations (what may still be in flight:
  // the copy of step 1 and the weights of steps 1 and 2)
  wait_vm<(kPfXS == 3 ? kPfCopies : 0) + 2 * kWLoads>();
  lds_barrier();

  // Every iteration runs kPfUnroll steps with no branch around their loads
  // (a branch around a step's loads makes the compiler's load-wait
  // bookkeeping merge paths and wait for every load in flight).  Steps past
  // `steps` load nothing and skip their arithmetic.
  for (int s0 = 0; s0 < steps; s0 += kPfUnroll) {
    static_for<0, kPfUnroll>([&](auto ic) {
      constexpr int I = decltype(ic)::value;  // = s % kPfUnroll
      const int s = s0 + I;
      unsigned char* const xa = xstage(I);              // consumed this step
      unsigned char* const xc = xstage(I + kPfXS - 1);  // filled for step s + XS - 1
      unsigned char* const wa = I % 2 ? ws1 : ws0;
      unsigned char* const wb = I % 2 ? ws0 : ws1;  // filled for step s + 1
      copy_x(xc, s + kPfXS - 1);
      compiler_fence();
      load_w(wq[I % kPfWQ], s + kPfWQ);
      compiler_fence();
      // (no decode arithmetic above the loads: it would wait for step s + 1's
      // weights before this step's loads are even issued)
      __builtin_amdgcn_sched_barrier(0);
      // A step past the end (the last iteration's) skips its decode, MFMAs
      // and weight store; the branch holds no global load, so the load waits
      // stay exact.
      if (s < steps) {
      unsigned v[8];
#pragma unroll
      for (int kc = 0; kc < 4; ++kc) {  // 16 weights of K per MFMA
        // a block of rows is decoded beside each 4 / NB of them
        if (kc % (4 / NB) == 0) F::make(wq[(I + 1) % kPfWQ][kc / (4 / NB)], s_begin + s + 1, dq, v);
        const int g = 2 * kc + fq;
        u32x4 af[kPfMI], bf[kPfNJ];
#pragma unroll
        for (int i = 0; i < kPfMI; ++i) af[i] = *reinterpret_cast<const u32x4*>(xa + pf_off(wt + 32 * i + fl, g));
#pragma unroll
        for (int j = 0; j < kPfNJ; ++j) bf[j] = *reinterpret_cast<const u32x4*>(wa + pf_off(wn + 32 * j + fl, g));
#pragma unroll
        for (int i = 0; i < kPfMI; ++i)
#pragma unroll
          for (int j = 0; j < kPfNJ; ++j) {
            if constexpr (F::kBf16)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, af[i]),
                                                                   __builtin_bit_cast(bf16x8, bf[j]), acc[i][j],
                                                                   0, 0, 0);
            else
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, af[i]),
                                                                  __builtin_bit_cast(half8, bf[j]), acc[i][j], 0,
                                                                  0, 0);
          }
        if (kc % (4 / NB) == 4 / NB - 1) store_w(wb, kc / (4 / NB), v);
      }
      }
      wait_vm<(kPfXS - 2) * kStepLoads + kWLoads>();  // this wave's copy of step s + 1's activations
      lds_barrier();  // all reads of this step's stages and all writes of the next are done
    });
  }
}

}  // namespace qgemv
