// The pieces that the prefill kernels share: the tile sizes and shared-memory layout, the online
// softmax of one key block with the deferred rescale, and the q4_0 dequant of a raw tile's items.
// fa_prefill.cu states the method and its sources; fa_prefill_paged.cu runs the same tiles over
// page pools.
#pragma once

#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kBM = 128;                      // query rows per tile
constexpr int kBN = 128;                      // keys per tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMarginLog2 = 10.0f * kLog2e; // the 10-point margin, in base-2 units
constexpr uint32_t kTmemCols = 512;
// TMEM column of the S block of query tile t (0: A, 1: B); P overwrites its first half
__host__ __device__ constexpr uint32_t col_s(int t) { return t ? 128u : 0u; }

// WIDE: the sixteen-warp layout with q4_0 K or V (both prefill kernels use it)
template <int D, bool KQ4, bool VQ4, bool WIDE = false>
struct Cfg {
  static constexpr bool kAnyQ4 = KQ4 || VQ4;
  static constexpr int kTileBytes = kBN * D * 2;          // one f16/bf16 K or V tile
  static constexpr int kQBytes = kBM * D * 2;             // one Q tile
  // ring of K/V tiles in MMA order K0 V0 K1 V1 ...; with one q4_0 side the stage count is even,
  // so K tiles always land on even stages and V tiles on odd ones (fixed arrival counts)
  static constexpr int kStages = (KQ4 && VQ4) ? 3 : (D == 128 ? 4 : 6);
  static constexpr int kRawStages = (KQ4 && VQ4) ? 3 : (kAnyQ4 ? 2 : 0);
  static_assert(KQ4 == VQ4 || kStages % 2 == 0, "mixed formats need an even ring");
  // dense K and V: the ring is used as kStages / 2 slots of two stages, slot g holding the V
  // tile of block j and the K tile of block j + 1 (the first slot of a unit or segment: K of
  // its first block alone), so that the MMA issuer waits for one slot and commits one release
  // per block step.  Each wait or commit costs the single issuing thread 120-350 clk of its
  // block period (measured), during which the tensor pipe drains.  A slot whose K tile tile B
  // multiplies is released by tile B's softmax on seeing that QK complete (the issuer's commit
  // covers every MMA it issued before, so also the earlier reads of the slot); the issuer
  // commits the release only of the others.
  static constexpr bool kPaired = !kAnyQ4;
  static constexpr int kSlots = kStages / 2;
  static_assert(!kPaired || kStages % 2 == 0, "paired ring");
  static constexpr int kNibRow = D / 2;                   // bytes of nibbles per key
  static constexpr int kScaleRow = D / 32 * 2;            // bytes of scales per key
  static constexpr int kRawNib = kBN * kNibRow;
  static constexpr int kRawBytes = ((kRawNib + kBN * kScaleRow) + 1023) / 1024 * 1024;
  static constexpr int kOffQ = 0;                         // Q_A, Q_B
  static constexpr int kOffRing = kOffQ + 2 * kQBytes;
  static constexpr int kOffRaw = kOffRing + kStages * kTileBytes;
  static constexpr int kOffBar = kOffRaw + kRawStages * kRawBytes;
  static constexpr int kBarBytes = 512 + 1024;  // barriers, flags, then the segment table
  static constexpr int kSmemBytes = kOffBar + kBarBytes + 1024;  // + alignment slack
  // warps: 0 producer, 1 MMA issuer, 4-11 softmax (one thread per query row), 2-3 dequant
  // with q4_0 K or V; WIDE adds dequant warps 12-15 (sixteen warps, 128 registers a thread at
  // launch; fa_prefill.cu then moves registers from warpgroups 0 and 3 to the two softmax
  // warpgroups, 88 and 168 a thread).  Measured at 16K keys, q4_0 K and V: with two dequant
  // warps the step waits for dequantized tiles; six of them took the cut kernel from 0.477 to
  // 0.410 ms and the one-unit kernel from 0.484 to 0.443 ms.
  static constexpr bool kWide = WIDE && kAnyQ4;
  static constexpr int kDqWarps = kAnyQ4 ? (kWide ? 6 : 2) : 0;
  static constexpr int kDqThreads = kDqWarps * 32;
  static constexpr int kWarps = kWide ? 16 : 12;
  static __device__ __forceinline__ bool is_dq_warp(int w) {
    return w == 2 || w == 3 || (kWide && w >= 12);
  }
  static __device__ __forceinline__ int dq_index(int w, int lane) {
    return (w < 4 ? w - 2 : w - 10) * 32 + lane;
  }
  static constexpr int kThreads = kWarps * 32;
  static constexpr uint32_t kColO0 = 256, kColO1 = 256 + D;     // O of tile A / B
};

// ------------------------------------------------------------------------------------------
// q4_0 nibble pair -> f16/bf16 pair
// ------------------------------------------------------------------------------------------
template <bool BF16>
struct Dq;
template <>
struct Dq<false> {
  // low nibbles at bits 0-3 / 16-19 -> (n - 8) exactly; mg = 0x64006400 in a register
  static __device__ __forceinline__ __half2 lo(uint32_t w, uint32_t mg) {
    uint32_t x = and_or<0x000F000Fu>(w, mg);  // 1024 + n
    return __hsub2(*reinterpret_cast<__half2*>(&x), __halves2half2(__ushort_as_half(0x6408),
                                                                    __ushort_as_half(0x6408)));
  }
  // high nibbles at bits 4-7 / 20-23 -> (n - 8) exactly
  static __device__ __forceinline__ __half2 hi(uint32_t w, uint32_t mg) {
    uint32_t x = and_or<0x00F000F0u>(w, mg);  // 1024 + 16 n
    const __half2 s = __halves2half2(__ushort_as_half(0x2C00), __ushort_as_half(0x2C00));  // 1/16
    const __half2 c = __halves2half2(__ushort_as_half(0xD480), __ushort_as_half(0xD480));  // -72
    return __hfma2(*reinterpret_cast<__half2*>(&x), s, c);
  }
  static __device__ __forceinline__ __half block(__half d) { return d; }
  static __device__ __forceinline__ uint32_t scale(__half2 v, __half d) {
    __half2 r = __hmul2(v, __halves2half2(d, d));
    return *reinterpret_cast<uint32_t*>(&r);
  }
};
template <>
struct Dq<true> {
  static __device__ __forceinline__ __nv_bfloat162 lo(uint32_t w, uint32_t mg) {
    uint32_t x = and_or<0x000F000Fu>(w, mg);  // 128 + n (mg = 0x43004300)
    const uint32_t c = 0x43084308u;           // 136
    return __hsub2(*reinterpret_cast<__nv_bfloat162*>(&x),
                   *reinterpret_cast<const __nv_bfloat162*>(&c));
  }
  // bf16 has 7 mantissa bits, so a high nibble at bits 4-7 would reach the exponent: shift it
  // down to bits 0-3 first
  static __device__ __forceinline__ __nv_bfloat162 hi(uint32_t w, uint32_t mg) {
    return lo(w >> 4, mg);
  }
  static __device__ __forceinline__ float block(__half d) { return __half2float(d); }
  static __device__ __forceinline__ uint32_t scale(__nv_bfloat162 v, float d) {
    // (n - 8) * d rounded once to bf16: the product of a 4-bit integer and an fp16 value is
    // exact in f32, so round only after the f32 multiply.
    const float2 f = __bfloat1622float2(v);
    __nv_bfloat162 r = __floats2bfloat162_rn(f.x * d, f.y * d);
    return *reinterpret_cast<uint32_t*>(&r);
  }
};


template <bool BF16>
__device__ __forceinline__ float block_row_exp_regs(uint32_t scol, const float (&s)[kBN],
                                                    float sl2, float nf) {
  // the scale-and-shift and the row sum run two keys per instruction (packed f32 pairs)
  const uint64_t sl2x2 = f2_pack(sl2, sl2), nfx2 = f2_pack(nf, nf);
  uint64_t acc0 = f2_pack(0.f, 0.f), acc1 = acc0;
#pragma unroll
  for (int c = 0; c < kBN / 32; ++c) {
    uint32_t pr[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 t =
          f2_unpack(f2_fma(f2_pack(s[32 * c + 2 * i], s[32 * c + 2 * i + 1]), sl2x2, nfx2));
      const float p0 = ex2(t.x), p1 = ex2(t.y);
      const uint64_t pp = f2_pack(p0, p1);
      if (i & 1) acc1 = f2_add(acc1, pp); else acc0 = f2_add(acc0, pp);
      pr[i] = pack2<BF16>(p0, p1);
    }
    tmem_st16(scol + 16 * c, pr);
  }
  const float2 a = f2_unpack(f2_add(acc0, acc1));
  return a.x + a.y;
}

// the scores of S(j) for this row with one TMEM wait, keys past rel_lim set to -inf (MASK)
template <bool MASK>
__device__ __forceinline__ void block_row_scores(uint32_t scol, int rel_lim, float (&s)[kBN]) {
  uint32_t r0[32], r1[32], r2[32], r3[32];
  tmem_ld32(scol, r0);
  tmem_ld32(scol + 32, r1);
  tmem_ld32(scol + 64, r2);
  tmem_ld32(scol + 96, r3);
  tmem_wait_ld();
  reg_fence32(r0);
  reg_fence32(r1);
  reg_fence32(r2);
  reg_fence32(r3);
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    s[i] = __uint_as_float(r0[i]);
    s[32 + i] = __uint_as_float(r1[i]);
    s[64 + i] = __uint_as_float(r2[i]);
    s[96 + i] = __uint_as_float(r3[i]);
    if (MASK) {
      if (i > rel_lim) s[i] = -INFINITY;
      if (32 + i > rel_lim) s[32 + i] = -INFINITY;
      if (64 + i > rel_lim) s[64 + i] = -INFINITY;
      if (96 + i > rel_lim) s[96 + i] = -INFINITY;
    }
  }
}
__device__ __forceinline__ float row_max_regs(const float (&s)[kBN]) {
  float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    m0 = fmax3(m0, s[i], s[i + 1]);
    m1 = fmax3(m1, s[32 + i], s[33 + i]);
    m2 = fmax3(m2, s[64 + i], s[65 + i]);
    m3 = fmax3(m3, s[96 + i], s[97 + i]);
  }
  return fmax3(fmaxf(m0, m1), m2, m3);
}

// Single-read form: a block's P is first formed in the row's current frame f.  Its row sum can exceed
// kSumTrigger only when some P does, and every P stays below 2^margin = e^10 unless the block
// max outgrows the frame by more than the margin; so a warp in which no row's sum exceeds it
// keeps those P without ever forming the block max.  Otherwise (or on a row's first block,
// f = -inf) the frame test proper runs: the block max, the frame move when it exceeds f by
// more than the margin, and P formed again in the new frame.  The frame decisions are exactly
// those of testing every block's max.  kSumTrigger sits just below e^10, so that the rounding
// of the exponential cannot hide a P at the bound.
constexpr float kSumTrigger = 21800.f;


// One key block of the online softmax for this thread's query row: read S(j), move the frame f
// to the block max when that exceeds f by more than the margin (l and, when it already holds
// earlier blocks (o_live), O are scaled by 2^(f_old - f)), write P = 2^(s - f) over S and add
// its row sum to l.  O may be rescaled in place: S(j) being ready means PV(j-1) has completed
// (QK(j) was issued after it).  The caller waits for the TMEM stores.
//
// One TMEM wait per block: the 128 scores stay in registers (168 a thread; in fa_prefill.cu's
// layouts with q4_0 sides by a register split between warpgroups) and P is formed in the current
// frame first.
//
// pmx tracks a bound on the largest P written (before its rounding to the dtype), each in the
// frame in force for its block: the exact largest P of a block that ran the frame test (P is
// monotonic in the score), the block's sum of P otherwise (at least its largest P, and below
// kSumTrigger).  Either way pmx <= e^10 whenever the frame rule holds.
struct NoWait {
  __device__ void operator()() const {}
};
// wait_o runs before O is rescaled in tensor memory (a PV MMA may still be adding to it when the
// S buffers alternate within one query tile)
template <int D, bool BF16, class WaitO = NoWait>
__device__ __forceinline__ void softmax_block(uint32_t scol, uint32_t ocol, bool need_mask,
                                              int rel_lim, float sl2, bool o_live, float& f,
                                              float& l, int& nres, float& pmx,
                                              const WaitO& wait_o = WaitO()) {
  auto rescale_o = [&](float alpha) {
    wait_o();
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t r[32];
      tmem_ld32(ocol + 32 * c, r);
      tmem_wait_ld();
      reg_fence32(r);
#pragma unroll
      for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
      tmem_st32(ocol + 32 * c, r);
    }
  };
  // the frame test proper: block max mx (scaled to m2), frame move, O rescale; true if any row
  // of the warp moved its frame
  auto frame_test = [&](float mx, float& alpha) -> bool {
    const float m2 = mx * sl2;
    const bool need = m2 > f + kMarginLog2;
    alpha = 1.f;
    if (need) {
      alpha = ex2(f - m2);
      l *= alpha;
      f = m2;
      ++nres;
    }
    return __any_sync(0xffffffffu, need);
  };
  const bool first = __any_sync(0xffffffffu, f == -INFINITY);
  float s[kBN];
  if (need_mask)
    block_row_scores<true>(scol, rel_lim, s);
  else
    block_row_scores<false>(scol, rel_lim, s);
  float sum = 0.f;
  bool done = false;
  if (!first) {
    sum = block_row_exp_regs<BF16>(scol, s, sl2, -f);
    done = !__any_sync(0xffffffffu, sum > kSumTrigger);
  }
  if (done) {
    pmx = fmaxf(pmx, sum);
  } else {
    const float mx = row_max_regs(s);
    float alpha;
    const bool any = frame_test(mx, alpha);
    if (any || first) {
      sum = block_row_exp_regs<BF16>(scol, s, sl2, -f);
      if (any && o_live) rescale_o(alpha);
    }
    pmx = fmaxf(pmx, ex2(fmaf(mx, sl2, -f)));  // -inf keys (a masked row) give 0
  }
  l += sum;
}

// One q4_0 dequant item: the 32 elements of block blk of key row t of a raw tile (nibble rows of
// NIB bytes, 64B-swizzled at D = 128 and 32B-swizzled at D = 64, then the fp16 scale rows of SROW
// bytes from byte RAWNIB), expanded to (q - 8) * d in f16/bf16 into the 128B-swizzled ring stage.
template <int D, bool BF16, int NIB, int SROW, int RAWNIB, class Q = Dq<BF16>>
__device__ __forceinline__ void dequant_item(const uint8_t* raw, uint8_t* dst, int t, int blk,
                                             uint32_t mg) {
  const uint8_t* nrow = raw + t * NIB;
  const __half* srow = reinterpret_cast<const __half*>(raw + RAWNIB + t * SROW);
    // 16 bytes of nibbles of this key, 64B-swizzled (D=128) or 32B-swizzled (D=64)
    const int chunk = (D == 128) ? (blk ^ ((t >> 1) & 3)) : (blk ^ ((t >> 2) & 1));
    const uint4 wv = *reinterpret_cast<const uint4*>(nrow + 16 * chunk);
    const uint32_t w[4] = {wv.x, wv.y, wv.z, wv.w};
    const __half dh = srow[blk];
    uint32_t outv[16];  // 32 dequantized elements, packed in pairs, natural order
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      // bytes 4q..4q+3 -> elements 4q..4q+3 (low) and 4q+16..4q+19 (high)
      const uint32_t a = __byte_perm(w[q], 0u, 0x5150);   // byte0 at b0, byte1 at b2
      const uint32_t c2 = __byte_perm(w[q], 0u, 0x5352);  // byte2 at b0, byte3 at b2
      const auto d = Q::block(dh);
      outv[2 * q + 0] = Q::scale(Q::lo(a, mg), d);
      outv[2 * q + 1] = Q::scale(Q::lo(c2, mg), d);
      outv[8 + 2 * q + 0] = Q::scale(Q::hi(a, mg), d);
      outv[8 + 2 * q + 1] = Q::scale(Q::hi(c2, mg), d);
    }
    // elements 32 blk + 8 cc .. +7 form 16-byte chunk (4 blk + cc) of the row
#pragma unroll
    for (int cc = 0; cc < 4; ++cc) {
      const int col16 = 4 * blk + cc;        // 16-byte chunk index along D
      const int atom = col16 >> 3;           // 64-element swizzle atom
      const int ch = (col16 & 7) ^ (t & 7);  // 128B swizzle
      *reinterpret_cast<uint4*>(dst + atom * (kBN * 128) + t * 128 + ch * 16) =
          make_uint4(outv[4 * cc], outv[4 * cc + 1], outv[4 * cc + 2], outv[4 * cc + 3]);
    }
}

}  // namespace
}  // namespace fa
