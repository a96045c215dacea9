// The pieces that the mma.sync kernels over few query rows share: stage layout, fragment loads, the
// MMA forms and the conversion of nibble pairs.  fa_decode.cu states the method and its sources;
// fa_prefill_paged_few.cu runs the same stages over ragged batches.
#pragma once

#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kConsumers = 4;  // consumer warps per CTA
constexpr float kLog2e = 1.4426950408889634f;

template <int D, bool KQ4, bool VQ4>
struct DCfg {
  static constexpr bool kAnyQ4 = KQ4 || VQ4;
  static constexpr int kSub = kAnyQ4 ? 2 : 1;                  // 16-key sub-tiles per warp step
  static constexpr int kTileKeys = 16 * kSub * kConsumers;     // keys per stage
  static constexpr int kNB = D / 32;                           // q4_0 blocks per key row
  static constexpr int kRow = kNB * 2;                         // scale bytes per key row
  static_assert(kRow > 0, "scale row");
  static constexpr int kNibBytes = kTileKeys * D / 2;
  // scales as the producer leaves them: K as f32 [key][block] (times the softmax scale in base
  // 2); V as f32 [key][block] (bf16) or as fp16 key pairs [16-key group][t][half][block] (f16)
  static constexpr int kScaleBytes = kTileKeys * kNB * 4;
  static constexpr int kDenseBytes = kTileKeys * D * 2;
  static constexpr int kKBytes = KQ4 ? kNibBytes : kDenseBytes;
  static constexpr int kVBytes = VQ4 ? kNibBytes : kDenseBytes;
  // stage: K tile | V tile | K scales (q4_0 K) | V scales (q4_0 V)
  static constexpr int kOffV = (kKBytes + 1023) / 1024 * 1024;
  static constexpr int kOffKs = kOffV + (kVBytes + 1023) / 1024 * 1024;
  static constexpr int kOffVs = kOffKs + (KQ4 ? kScaleBytes : 0);
  static constexpr int kStageBytes = ((kOffVs + (VQ4 ? kScaleBytes : 0)) + 1023) / 1024 * 1024;
  // one dense side of 128 keys makes a stage ~42 KB (D = 128): two stages and two CTAs per SM
  static constexpr int kStages = (KQ4 == VQ4) ? (D == 128 ? 3 : 6) : (D == 128 ? 2 : 4);
  static constexpr int kCtasPerSm = (KQ4 && VQ4) ? 3 : 2;
  static constexpr int kOffBar = kStages * kStageBytes;
  static constexpr int kOffQ = kOffBar + 256;  // the group's query rows, [8][D] 16-bit
  static constexpr int kSmemBytes = kOffQ + 8 * D * 2 + 1024;
  static constexpr int kThreads = 32 * (1 + kConsumers);
  static constexpr int kPartStride = D + 4;  // m, l, pad, pad, O[D]
  // cross-warp merge buffer (reuses the stages): per warp 8 heads x (D + 2) floats
  static_assert(kConsumers * 8 * (D + 2) * 4 <= kStages * kStageBytes, "merge buffer");
};

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                        uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t& r0, uint32_t& r1,
                                          uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t movtrans(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// d = A B + c with separate accumulator input and output registers
template <bool BF16>
__device__ __forceinline__ void mma16816_c(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                           uint32_t a3, uint32_t b0, uint32_t b1, float c0,
                                           float c1, float c2, float c3) {
  if (BF16)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2),
          "f"(c3));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2),
          "f"(c3));
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if (BF16)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------------------------------------
// nibble pairs -> f16/bf16 pairs.  Low nibbles sit at bits 0-3 / 16-19 of the word, high
// nibbles at bits 4-7 / 20-23.
// ---------------------------------------------------------------------------------------------
// raw values (one LOP3 with the exponent pattern `mg` in a register): f16 (1024 + q) from low
// nibbles, (1024 + 16 q) from high nibbles; bf16 (128 + q) from low nibbles only (bf16 has 7
// mantissa bits).  mg = 0x64006400 (f16) or 0x43004300 (bf16).
__device__ __forceinline__ uint32_t raw_lo(uint32_t w, uint32_t mg) {
  return and_or<0x000F000Fu>(w, mg);
}
__device__ __forceinline__ uint32_t raw_hi_f16(uint32_t w, uint32_t mg) {
  return and_or<0x00F000F0u>(w, mg);
}
// exact (q - 8) pairs
template <bool BF16>
__device__ __forceinline__ uint32_t nib_lo(uint32_t w, uint32_t mg) {
  uint32_t x = raw_lo(w, mg);
  if (BF16) {
    const uint32_t c = 0x43084308u;  // 136
    __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&x),
                               *reinterpret_cast<const __nv_bfloat162*>(&c));
    return *reinterpret_cast<uint32_t*>(&r);
  } else {
    const uint32_t c = 0x64086408u;  // 1032
    __half2 r = __hsub2(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<const __half2*>(&c));
    return *reinterpret_cast<uint32_t*>(&r);
  }
}
template <bool BF16>
__device__ __forceinline__ uint32_t nib_hi(uint32_t w, uint32_t mg) {
  if (BF16) {
    return nib_lo<true>(w >> 4, mg);
  } else {
    uint32_t x = raw_hi_f16(w, mg);                   // 1024 + 16 q
    const uint32_t s = 0x2C002C00u, c = 0xD480D480u;  // 1/16, -72
    __half2 r = __hfma2(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<const __half2*>(&s),
                        *reinterpret_cast<const __half2*>(&c));
    return *reinterpret_cast<uint32_t*>(&r);
  }
}

template <bool BF16>
__device__ __forceinline__ float h2f(uint16_t bits) {
  return BF16 ? __uint_as_float(static_cast<uint32_t>(bits) << 16)
              : __half2float(__ushort_as_half(bits));
}
template <bool BF16>
__device__ __forceinline__ uint16_t f2h(float v) {
  return BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v))
              : __half_as_ushort(__float2half_rn(v));
}

}  // namespace
}  // namespace fa
