// Causal attention of a ragged batch of new tokens over page pools (fa_prefill_paged), sm_103a; K
// and V each dense or q4_0.
//
// What it computes: for row t of sequence b (position p = lens[b] - n_b + its place in the
// sequence's rows) and query head h
//     O[t, h] = sum_{j <= p} softmax_j(scale <Q[t, h], K[b, g, j]>) V[b, g, j],  g = h / (Hq / Hkv),
// K[b, g, j] being the pool row that the block table gives for position j; causal = 0 lets every row
// see all lens[b] keys, and a row that sees no key gives zeros.  The chunked-prefill call and the
// deferred rescale are those of "perf(rocm): defer SDPA accumulator rescale, stage Q once per block
// (#2306)" (Conversation; What changed) as fa_prefill.cu builds them; the softmax, dequant and tile
// layout are the same code (fa_prefill_tile.cuh).
//
//  * A 128-row query tile holds all G = Hq / Hkv query heads of floor(128 / G) consecutive tokens:
//    one TMA box {64, G, tokens} of Q, rows in token-major order.  A K/V tile is then read once for
//    the whole group, and a few new tokens fill G times as many rows as they would head by head.
//  * A work unit is a pair of consecutive tiles (A, B) of one sequence and kv head; its steps are
//    the 128-key blocks that the pair sees, at least one.  All units' steps are concatenated
//    (sequence, then pair, then kv head) and cut evenly over one CTA per SM, whatever the mix of
//    long chunks and single tokens (short units stay whole, see PagedPlan); a unit cut between CTAs
//    is merged by the piece that finds all its siblings published.  Lengths live on the device, so every CTA finds its own run: one warp
//    sums the steps of the batch, locates the run and feeds the other roles one segment (a run of
//    steps of one unit) at a time through a small queue in shared memory.
//  * A 128-key tile is fetched as 128 / box boxes of box = gcd(page_size, 128) keys, each with its
//    own page.  Boxes that hold no key of the sequence are fetched from outside the pool, which TMA
//    fills with zeros without reading memory; the rows of a dense V tile between the sequence's end
//    and its box's are cleared in shared memory, so that what an unused slot holds (NaN included)
//    never meets a zero weight.  q4_0 rows past the end get a zero scale.
//
// What bounds it, measured on one GB300 (GQA 32/8, D = 128; us a call from a CUDA graph): long chunks
// by each tile's softmax and hand-offs behind the other tile's MMAs, 2048 tokens at the end of 16384
// f16 keys 330 (1560 TFLOP/s, tensor pipe active 66 %), over q4_0 pools 407, where the dequant takes
// issue slots and shared-memory bandwidth; single tokens over dense pools by HBM, 64 sequences of
// 8192 bf16 keys 330 (6.5 TB/s); over q4_0 pools by the lone tile's block step (dequant and operand
// reads in shared memory, 1.2 us with f16, 1.5 with bf16), the same batch 271 and 335; small calls by
// the 13 us of launch, plan, first loads and merges.
//
// Warp roles: as in fa_prefill.cu (0 producer and scheduler, 1 TMEM and MMA issuer, 2-3 and 12-15
// q4_0 dequant, 4-7 softmax of tile A, 8-11 of tile B), without moving registers between them.
#include <limits.h>
#include <stddef.h>

#include "fa_internal.h"
#include "fa_paged.cuh"
#include "fa_prefill_tile.cuh"
#include "fa_ptx.cuh"

namespace fa {

__device__ uint32_t g_prefill_paged_error;

namespace {

// barrier slots (8 bytes each) inside the barrier area
enum {
  pbQFull = 0,
  pbSFull = 1,       // + tile (2)
  pbPReady = 3,      // + tile (2)
  pbODone = 5,       // + tile (2): after the tile's last PV MMA of a segment
  pbDrain = 7,
  pbRingFull = 8,    // + stage (up to 8)
  pbRingEmpty = 16,  // + stage
  pbRawFull = 24,    // + raw stage (up to 4)
  pbRawEmpty = 28,   // + raw stage
  pbQEmpty = 32,     // the segment's last QK MMA has read the Q tiles
  pbOFree = 33,      // + tile (2): the segment's epilogue has read O out of TMEM
  pbTail = 37,       // a V tile that needs rows cleared has landed
  pbSegFull = 38,    // + queue slot (kSegQ)
  pbSegEmpty = 42,   // + queue slot
  pbSAlt = 46,       // lone tile A: scores in, and P of, the second S buffer
  pbPAlt = 47,
  pbPvAlt = 48,      // lone tile A: after every PV MMA
  // a run cuts two units at most: that of its first segment (+ 0), which others began, and that of
  // its last (+ 1), which others go on with
  pbPiece = 49,      // all 256 softmax threads have stored their rows of the piece
  pbDecided = 51,    // whether all pieces were there is decided
  pbEarly = 53,      // the last: whether all others are there before its own is stored
  pbCount = 54
};
constexpr int kSegQ = 4;
constexpr int kOffTmem = pbCount * 8;
constexpr int kOffAbort = kOffTmem + 8;
constexpr int kOffMerge = kOffAbort + 8;  // decisions: first piece, last piece, last piece early
constexpr int kOffPlan = kOffMerge + 16;  // int: the run has segments; raw tiles before its end
constexpr int kOffSegQ = 512;            // the segment queue

// one segment: steps [j0, j1) of a unit
struct alignas(16) PSeg {
  int row0;       // packed row of tile A's first token
  int g;          // kv head
  int tokA, tokB; // tokens of the tiles (0: tile absent)
  int pos0;       // position of tile A's first token
  int len;        // keys of the sequence
  int nbA, nbB;   // key blocks of the tiles
  int j0, j1;     // j1 = -1: no more segments
  int c_first, c_last;  // CTAs of the unit's first and last step (equal: not cut)
  int slot_first;       // partial slot of the first one's piece (the others' is 0)
  int own_slot;         // and of this CTA's
  int unused[2];
};
static_assert(offsetof(PSeg, pos0) == 16 && offsetof(PSeg, j0) == 32 &&
                  offsetof(PSeg, slot_first) == 48 && sizeof(PSeg) == 64, "read_seg");
constexpr int kOffFirst = kOffSegQ + kSegQ * 64;  // the first segment, kept for its merge
static_assert(sizeof(PSeg) <= 64 && kOffFirst + 64 <= 512 + 1024, "segment queue");
static_assert(kOffPlan + 8 <= kOffSegQ, "barrier area");

struct PArgs {
  PagedPlan plan;
  uint8_t* o;
  int64_t o_row_stride, o_head_stride;  // bytes
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  int G, tile_tok, box, box_bits;  // box = 1 << box_bits
  float scale_log2;
  float* part;       // partial rows of units cut between CTAs, 2 slots a CTA, 2 tiles a slot
  uint32_t* pflags;  // [CTAs][2] publication flags, tagged per call, then the tag of an abandoned call
  uint32_t tag;
};

// One tile of a piece, column-major, so that a warp's 32 rows of one column are 128 contiguous
// bytes: [D + 2 columns][128 rows] f32, columns O[0..D), frame, row sum.  (Row-major pieces, stored
// 16 bytes a lane and row, took the 2048-token chunk at 16384 keys from 346 to 368 us.)  A CTA has
// two slots: 0 for the piece its run begins with, 1 for one that it reaches after other units (an
// address stays within them whatever the slot).
template <int D>
__device__ __forceinline__ float* piece_tile(float* part, int c, int slot, int t) {
  return part + ((static_cast<int64_t>(c) * 2 + (slot & 1)) * 2 + t) * (D + 2) * kBM;
}

// The last key that a row of the segment sees: tok counts from tile A's first token
__device__ __forceinline__ int last_key(const PSeg& sg, int causal, int tok) {
  return causal ? min(sg.len - 1, sg.pos0 + tok) : sg.len - 1;
}
// A piece's frame as the merges take it: -inf where the row sees no key of the piece (its sums are not
// used), +inf where its sum is NaN, so that the merged row is NaN however small the piece's weight.
__device__ __forceinline__ float piece_frame(bool sees, float f, float l) {
  return !sees ? -INFINITY : l == l ? f : INFINITY;
}

// the thread's number, formed anew where it is asked for
__device__ __forceinline__ int opaque_tid() {
  uint32_t tid;
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
  return static_cast<int>(tid);
}
// mbar_wait with the abort flag at a shared address (no generic pointer kept in registers)
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, uint32_t abort_at) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    if (lds32(abort_at)) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      asm volatile("st.volatile.shared.b32 [%0], 1;" ::"r"(abort_at) : "memory");
      atomicCAS(&g_prefill_paged_error, kErrNone, kErrTimeout);
      return false;
    }
  }
}
// Dq<true> with (n - 8) d formed in bf16 pairs: d = hi + lo, each exact in bf16 (an f16 scale's 11
// bits), (n - 8) lo is exact (4 and 3 bits), and the fused (n - 8) hi + (n - 8) lo rounds the exact
// sum once, as the product in f32 does, in four instructions a pair for seven.  (One token each
// against 64 sequences of 8192 q4_0 keys, 8 kv heads, D = 128: 377 -> 339 us.)
struct DqSplit : Dq<true> {
  struct Scale {
    __nv_bfloat162 hi, lo;
  };
  static __device__ __forceinline__ Scale block(__half d) {
    const float f = __half2float(d);
    const __nv_bfloat16 hi = __float2bfloat16_rn(f);
    const float lo = f - __bfloat162float(hi);
    // (an infinite d has no low part)
    return {__bfloat162bfloat162(hi), __float2bfloat162_rn(lo == lo ? lo : 0.f)};
  }
  static __device__ __forceinline__ uint32_t scale(__nv_bfloat162 v, Scale d) {
    const __nv_bfloat162 r = __hfma2(v, d.hi, __hmul2(v, d.lo));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
template <bool BF16>
struct DqOf {
  using type = Dq<false>;
};
template <>
struct DqOf<true> {
  using type = DqSplit;
};
// A segment out of shared memory, whole and unconditionally.  (Builds that moved registers from the other
// warps to the softmax warps, as fa_prefill.cu does, and left it to the compiler to read some fields
// under a condition, now and then saw 512 for 0 in the selection `own CTA first ? slot_first : 0`, a
// whole warp at a time, whose rows then went outside the workspace.  Why is not known.  Builds without
// either were clean; this one has neither.)
__device__ __forceinline__ int4 lds_int4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ PSeg read_seg(uint32_t addr) {
  const int4 a = lds_int4(addr), b = lds_int4(addr + 16), c = lds_int4(addr + 32),
             d = lds_int4(addr + 48);
  return PSeg{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w, d.x, d.y, {0, 0}};
}
// 16-byte asynchronous copy of which src_bytes are read, the rest zeros
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(src_bytes)
               : "memory");
}

// softmax_block in fewer registers, for the sixteen-warp layout's 128 a thread.  A block that every row of
// the warp sees whole is read 64 keys at a time, the second 64 under way while the first are turned into
// P.  The first half's P stays packed in registers until the second half's scores are there and their
// max shows, with the first half's row sum (see kSumTrigger), that no row of the warp needs the frame
// test; from then on P goes over S as it is formed.  Otherwise -- a row's first block, a masked one, or
// one that needs the test -- S is whole still and is read twice, 32 keys at a time and no further than
// some row sees: for the block's max, and to form P in the frame that follows.  Frames, P and sums are
// those of softmax_block to the bit (a row that sees nothing of the block apart, whose are not used).
//
// (softmax_block's 128 scores in registers need 168 of them a thread, which sixteen warps have only
// where the other warps hand theirs over.  Measured against that, us: 16 x 5 draft tokens over q4_0
// 46.9 -> 42.3, 256 sequences of 64 q4_0 keys 74.0 -> 57.9, five prompts with q4_0 V 18.9 -> 20.4, 2048
// tokens at 16384 q4_0 keys 396 -> 408.  The second way unrolled, over all 128 keys: 46.9 / 84.8 / 20.6 /
// 410; all of P kept until the row sum is known 43.3 / 59.7 / 20.8 / 412, three quarters of it 42.5 /
// 59.1 / 20.4 / 413.)
__device__ __forceinline__ float max_chunk(const uint32_t (&r)[32]) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < 32; i += 2) m = fmax3(m, __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
  return m;
}
struct RowSum {
  uint64_t acc0, acc1;
};
template <bool BF16>
__device__ __forceinline__ void exp_chunk(const uint32_t (&r)[32], uint32_t (&p)[16], uint64_t sl2x2,
                                          uint64_t nfx2, RowSum& s) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 t = f2_unpack(f2_fma(
        f2_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), sl2x2, nfx2));
    const float p0 = ex2(t.x), p1 = ex2(t.y);
    const uint64_t pp = f2_pack(p0, p1);
    if (i & 1) s.acc1 = f2_add(s.acc1, pp); else s.acc0 = f2_add(s.acc0, pp);
    p[i] = pack2<BF16>(p0, p1);
  }
}
__device__ __forceinline__ float row_sum(const RowSum& s) {
  const float2 a = f2_unpack(f2_add(s.acc0, s.acc1));
  return a.x + a.y;
}
__device__ __forceinline__ void load_chunk(uint32_t scol, int c, uint32_t (&r)[32]) {
  tmem_ld32(scol + 32 * c, r);
}
// P in frame f over S unless a row needs the frame test (then nothing is stored): the row sum
template <bool BF16>
__device__ __forceinline__ bool exp_in_frame(uint32_t scol, float sl2, float f, float& sum) {
  const uint64_t sl2x2 = f2_pack(sl2, sl2), nfx2 = f2_pack(-f, -f);
  RowSum acc = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
  uint32_t r0[32], r1[32], r2[32], r3[32], p0[16], p1[16];
  load_chunk(scol, 0, r0);
  load_chunk(scol, 1, r1);
  tmem_wait_ld();
  reg_fence32(r0);
  reg_fence32(r1);
  exp_chunk<BF16>(r0, p0, sl2x2, nfx2, acc);
  load_chunk(scol, 2, r2);
  exp_chunk<BF16>(r1, p1, sl2x2, nfx2, acc);
  load_chunk(scol, 3, r3);
  tmem_wait_ld();
  reg_fence32(r2);
  reg_fence32(r3);
  const float m = fmaxf(max_chunk(r2), max_chunk(r3)) * sl2;
  if (__any_sync(0xffffffffu, row_sum(acc) > kSumTrigger || m > f + kMarginLog2)) return false;
  tmem_st16(scol, p0);
  tmem_st16(scol + 16, p1);
  exp_chunk<BF16>(r2, p0, sl2x2, nfx2, acc);
  tmem_st16(scol + 32, p0);
  exp_chunk<BF16>(r3, p1, sl2x2, nfx2, acc);
  tmem_st16(scol + 48, p1);
  sum = row_sum(acc);
  return true;
}
// 32 keys' scores, those past lim set to -inf; false, and nothing loaded, where no row of the warp sees
// any of them
__device__ __forceinline__ bool seen_chunk(uint32_t scol, int lim, uint32_t (&r)[32]) {
  if (__all_sync(0xffffffffu, lim < 0)) return false;
  load_chunk(scol, 0, r);
  tmem_wait_ld();
  reg_fence32(r);
  if (__any_sync(0xffffffffu, lim < 31)) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i > lim) r[i] = __float_as_uint(-INFINITY);
  }
  return true;
}
__device__ __forceinline__ float block_max(uint32_t scol, int rel_lim) {
  float m = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32];
    if (!seen_chunk(scol + 32 * c, rel_lim - 32 * c, r)) break;
    m = fmaxf(m, max_chunk(r));
  }
  return m;
}
// P in frame f over S, P of keys 32 c .. over S of keys 16 c .., which are read by then: the row sum
template <bool BF16>
__device__ __forceinline__ float exp_block(uint32_t scol, int rel_lim, float sl2, float f) {
  const uint64_t sl2x2 = f2_pack(sl2, sl2), nfx2 = f2_pack(-f, -f);
  RowSum acc = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32], p[16];
    if (seen_chunk(scol + 32 * c, rel_lim - 32 * c, r)) {
      exp_chunk<BF16>(r, p, sl2x2, nfx2, acc);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) p[i] = 0u;
    }
    tmem_st16(scol + 16 * c, p);
  }
  return row_sum(acc);
}
template <int D, bool BF16, class WaitO>
__device__ __forceinline__ void softmax_block_lean(uint32_t scol, uint32_t ocol, bool need_mask,
                                                   int rel_lim, float sl2, bool o_live, float& f,
                                                   float& l, const WaitO& wait_o) {
  if (!__any_sync(0xffffffffu, f == -INFINITY)) {
    float sum;
    if (!need_mask && exp_in_frame<BF16>(scol, sl2, f, sum)) {
      l += sum;
      return;
    }
  }
  const float m2 = block_max(scol, rel_lim) * sl2;
  const bool need = m2 > f + kMarginLog2;
  float alpha = 1.f;
  if (need) {
    alpha = ex2(f - m2);
    l *= alpha;
    f = m2;
  }
  if (__any_sync(0xffffffffu, need) && o_live) {
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
  }
  l += exp_block<BF16>(scol, rel_lim, sl2, f);
}

// Merge of one unit's pieces by the 256 softmax threads.  A tile's threads (both tiles' where tile
// B is absent) are laid out as Rp rows x column groups, Rp the rows in use rounded up to a power of
// two: a few rows spread over many column groups.  kCols columns of kFly pieces are loaded together
// and joined with a running frame.  (Frames: piece_frame.)
template <int D, bool BF16>
__device__ __forceinline__ void merge_pieces(const PArgs& args, const PSeg& sg) {
  constexpr int kFly = 4, kCols = 16;
  const bool both = sg.tokB == 0;
  const int th = threadIdx.x - 128;
  const int t = both ? 0 : th >> 7;
  const int u = both ? th : th & 127;
  const int threads = both ? 256 : 128;
  const int rows = (t ? sg.tokB : sg.tokA) * args.G;
  int Rp = 512 / D;  // (at least two columns a thread)
  while (Rp < rows) Rp *= 2;
  const int r = u & (Rp - 1);
  if (r >= rows) return;
  const int cols = D * Rp / threads, col0 = (u / Rp) * cols;
  const int n = sg.c_last - sg.c_first + 1;
  // CTA c_first's piece may lie in its second slot, the others' are in their first
  const float* p_first = piece_tile<D>(args.part, sg.c_first, sg.slot_first, t) + r;
  const float* p_rest = piece_tile<D>(args.part, sg.c_first, 0, t) + r;
  const int64_t step = 4 * (D + 2) * kBM;  // floats from a CTA's slot 0 to the next CTA's
  const int tok = r / args.G;
  uint8_t* orow = args.o + (sg.row0 + t * args.tile_tok + tok) * args.o_row_stride +
                  (sg.g * args.G + (r - tok * args.G)) * args.o_head_stride;
#pragma unroll 1
  for (int k0 = col0; k0 < col0 + cols; k0 += kCols) {
    float F = -INFINITY, L = 0.f;
    float acc[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
#pragma unroll 1
    for (int c0 = 0; c0 < n; c0 += kFly) {
      float f[kFly], l[kFly], v[kFly][kCols];
#pragma unroll
      for (int c = 0; c < kFly; ++c) {
        const bool in = c0 + c < n;
        const float* p = c0 + c == 0 ? p_first : p_rest + (c0 + c) * step;
        f[c] = in ? __ldcg(p + D * kBM) : -INFINITY;
        l[c] = in ? __ldcg(p + (D + 1) * kBM) : 0.f;
#pragma unroll
        for (int i = 0; i < kCols; ++i)
          v[c][i] = in && i < cols ? __ldcg(p + (k0 + i) * kBM) : 0.f;
      }
      const float top = fmaxf(F, fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])));
      if (top == -INFINITY) continue;
      const float a = ex2(F - top);  // F = -inf: 0
      L *= a;
#pragma unroll
      for (int i = 0; i < kCols; ++i) acc[i] *= a;
      F = top;
#pragma unroll
      for (int c = 0; c < kFly; ++c) {
        const float w = f[c] == -INFINITY ? 0.f : ex2(f[c] - F);
        if (w == 0.f) continue;  // (frame -inf: its O may be no number)
        L = fmaf(w, l[c], L);
#pragma unroll
        for (int i = 0; i < kCols; ++i) acc[i] = fmaf(w, v[c][i], acc[i]);
      }
    }
    const float inv = F == -INFINITY ? 0.f : 1.f / L;
    uint32_t w[kCols / 2];
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) w[i] = pack2<BF16>(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    if (cols >= kCols) {
      reinterpret_cast<uint4*>(orow + k0 * 2)[0] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint4*>(orow + k0 * 2)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i)
        if (2 * i < cols) reinterpret_cast<uint32_t*>(orow + k0 * 2)[i] = w[i];
    }
  }
}

// The same for a thread's own row of a unit of two pieces, where this CTA began the unit and the other
// piece is published: the own one still in tensor memory, FLY columns of the other one's in flight
// (D, or what 128 registers hold).
// Joined in CTA order with the arithmetic of merge_pieces, so that the result does not depend on which
// CTA came last.  f: the own piece's, by piece_frame.
template <int D, bool BF16, int FLY>
__device__ __forceinline__ void merge_with_own(const PArgs& args, const PSeg& sg, int t, int row,
                                               uint32_t ocol, bool active, bool valid, float f,
                                               float l) {
  const float* p = piece_tile<D>(args.part, sg.c_last, 0, t) + row;
  const float fo = valid ? __ldcg(p + D * kBM) : -INFINITY;
  const float lo = valid ? __ldcg(p + (D + 1) * kBM) : 0.f;
  float v[FLY];
  auto load = [&](int k) {
    if (valid) {
#pragma unroll
      for (int i = 0; i < FLY; ++i) v[i] = __ldcg(p + (k + i) * kBM);
    }
  };
  load(0);
  const float F = fmaxf(f, fo);
  const float w = f == -INFINITY ? 0.f : ex2(f - F);    // 0: the piece's O may be no number
  const float wo = fo == -INFINITY ? 0.f : ex2(fo - F);
  float L = 0.f;
  if (w != 0.f) L = fmaf(w, l, L);
  if (wo != 0.f) L = fmaf(wo, lo, L);
  const float inv = F == -INFINITY ? 0.f : 1.f / L;
  const int tok = row / args.G;
  uint8_t* orow = args.o + (sg.row0 + t * args.tile_tok + tok) * args.o_row_stride +
                  (sg.g * args.G + (row - tok * args.G)) * args.o_head_stride;
#pragma unroll
  for (int k = 0; k < D; k += 32) {
    uint32_t r[32];
    __syncwarp();  // the loads from tensor memory are the whole warp's
    if (active) {
      tmem_ld32(ocol + k, r);
      tmem_wait_ld();
      reg_fence32(r);
    }
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float x[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float a = w != 0.f ? __uint_as_float(r[2 * e + i]) : 0.f;
        const float b = wo != 0.f ? v[k % FLY + 2 * e + i] : 0.f;
        x[i] = fmaf(wo, b, fmaf(w, a, 0.f)) * inv;
      }
      pk[e] = pack2<BF16>(x[0], x[1]);
    }
    if (valid) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        reinterpret_cast<uint4*>(orow + 2 * k)[i] =
            make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
    }
    if ((k + 32) % FLY == 0 && k + 32 < D) load(k + 32);
  }
}
// Publication flag of CTA c's piece: its slot is slot_first for the unit's first CTA, 0 for the others,
// and the address stays within CTA c's two flags whatever the segment holds.
__device__ __forceinline__ uint32_t* flag_at(const PArgs& args, int c, int slot) {
  return args.pflags + 2 * c + (slot & 1);
}
__device__ __forceinline__ uint32_t* piece_flag(const PArgs& args, const PSeg& sg, int c) {
  return flag_at(args, c, sg.slot_first & -static_cast<int>(c == sg.c_first));
}
// A call that a CTA abandoned leaves flags set, which a replay of the same captured call (the same tag)
// would take for its own: the CTA leaves the call's tag behind the flags, and until the workspace is
// overwritten such a replay merges nothing and is reported as the abandoned call was.
__device__ __forceinline__ uint32_t* abandoned_tag(const PArgs& args) {
  return args.pflags + 2 * gridDim.x;
}
// whether all pieces but CTA `but`'s (-1: all pieces) are published, by one warp; their rows may be
// read after it
__device__ __forceinline__ bool pieces_there(const PArgs& args, const PSeg& sg, int but) {
  const uint32_t gone = ld_relaxed_gpu(abandoned_tag(args));
  bool all = true;
  for (int c = sg.c_first + (threadIdx.x & 31); c <= sg.c_last; c += 32)
    all = all && (c == but || ld_relaxed_gpu(piece_flag(args, sg, c)) == args.tag);
  if (gone == args.tag) {
    atomicCAS(&g_prefill_paged_error, kErrNone, kErrTimeout);
    all = false;
  }
  all = __all_sync(0xffffffffu, all);
  if (all) {
    fence_acq_rel_gpu();  // each lane acquires the pieces whose flags it has read,
    __syncwarp();         // all before the lane that tells the other warps
  }
  return all;
}

// Store of a thread's row of a piece into one of the CTA's slots; f by piece_frame
template <int D>
__device__ __forceinline__ void store_piece(const PArgs& args, int slot, int t, int row,
                                            uint32_t ocol, bool active, bool valid, float f,
                                            float l) {
  float* pt = piece_tile<D>(args.part, static_cast<int>(blockIdx.x), slot, t) + row;
  if (active) {
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t r[32];
      __syncwarp();
      tmem_ld32(ocol + 32 * c, r);
      tmem_wait_ld();
      reg_fence32(r);
      if (valid) {
#pragma unroll
        for (int i = 0; i < 32; ++i) pt[(32 * c + i) * kBM] = __uint_as_float(r[i]);
      }
    }
  }
  if (valid) {
    pt[D * kBM] = f;
    pt[(D + 1) * kBM] = l;
  }
}

// Publication of this CTA's piece by one warp, once all rows are stored; whether all pieces are there
// by then.  Of two pieces published at the same time at least one sees the other's flag (release
// store, then a sequentially consistent fence before the flag loads), so at least one CTA finds
// them all and merges; every CTA that does writes the same bytes.
__device__ __forceinline__ bool publish_piece(const PArgs& args, const PSeg& sg, uint32_t stored,
                                              uint32_t stop) {
  if (!__all_sync(0xffffffffu, wait_bounded(stored, 0, stop))) return false;
  if ((threadIdx.x & 31) == 0)
    st_release_gpu(flag_at(args, static_cast<int>(blockIdx.x), sg.own_slot), args.tag);
  __syncwarp();
  fence_sc_gpu();
  return pieces_there(args, sg, -1);
}
// for the next call (or graph replay) with this tag
__device__ __forceinline__ void clear_flags(const PArgs& args, const PSeg& sg) {
  for (int c = sg.c_first + (threadIdx.x & 31); c <= sg.c_last; c += 32)
    st_relaxed_gpu(piece_flag(args, sg, c), 0u);
}

template <int D, bool BF16, bool KQ4, bool VQ4>
__global__ void __launch_bounds__(Cfg<D, KQ4, VQ4, true>::kThreads, 1)
    prefill_paged_kernel(const __grid_constant__ CUtensorMap tm_q,
                         const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ PArgs args) {
  using C = Cfg<D, KQ4, VQ4, true>;
  constexpr int kChunks = D / 64;  // 64-element column chunks of a tile
  // a lone tile's blocks alternate between the S buffers; not with one q4_0 side, whose ring ties
  // K and V to even and odd stages
  constexpr bool kAlt = KQ4 == VQ4;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - smem_u32(smem_raw));
  const uint32_t bar0 = sbase + C::kOffBar;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * i; };
  uint8_t* bgen = sgen + C::kOffBar;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bgen + kOffAbort);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bgen + kOffTmem);
  volatile int* has_run = reinterpret_cast<volatile int*>(bgen + kOffPlan);
  volatile int* raw_end = has_run + 1;
  const uint32_t segs = bar0 + kOffSegQ;
  auto seg_at = [&](int i) -> PSeg* {
    return reinterpret_cast<PSeg*>(bgen + kOffSegQ + (i % kSegQ) * 64);
  };

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int cta = static_cast<int>(blockIdx.x);
  const PagedPlan& plan = args.plan;

  PagedWalk w;                      // warp 0 only
  const int nbox = kBN >> args.box_bits;  // boxes of a tile
  // lane i < nbox looks up the page of box i of block j
  auto look_up = [&](int j) -> int {
    return lane < nbox ? w.look_up(plan, j * kBN + (lane << args.box_bits)) : -1;
  };
  int page0 = -1;  // of the next segment's first block, looked up ahead
  if (warp == 0) {
    if (lane == 0) {
      prefetch_tmap(&tm_q);
      prefetch_tmap(&tm_k);
      prefetch_tmap(&tm_v);
    }
    w.find(plan, cta, gridDim.x, &g_prefill_paged_error, kErrBadIndex);
    if (lane == 0) {
      *has_run = w.t < w.t_end;
      *raw_end = INT_MAX;
    }
    if (w.t < w.t_end) page0 = look_up(w.j0(plan));
  } else if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  } else if (warp == 2) {
    if (lane == 0) {
      mbar_init(bar(pbQFull), 1);
      for (int t = 0; t < 2; ++t) {
        mbar_init(bar(pbSFull + t), 1);
        mbar_init(bar(pbPReady + t), 128);
        mbar_init(bar(pbODone + t), 1);
        mbar_init(bar(pbOFree + t), 128);
      }
      mbar_init(bar(pbDrain), 1);
      mbar_init(bar(pbQEmpty), 1);
      mbar_init(bar(pbTail), 1);
      mbar_init(bar(pbSAlt), 1);
      mbar_init(bar(pbPAlt), 128);
      mbar_init(bar(pbPvAlt), 1);
      mbar_init(bar(pbEarly), 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(pbPiece + i), 256);
        mbar_init(bar(pbDecided + i), 1);
      }
      for (int s = 0; s < kSegQ; ++s) {
        mbar_init(bar(pbSegFull + s), 1);
        mbar_init(bar(pbSegEmpty + s), 1 + 8);  // the issuer and the eight softmax warps
      }
      for (int s = 0; s < C::kStages; ++s) {
        const bool q4s = (C::kStages % 2 == 0) ? ((s & 1) ? VQ4 : KQ4) : (KQ4 && VQ4);
        mbar_init(bar(pbRingFull + s), q4s ? C::kDqWarps : 1);
        mbar_init(bar(pbRingEmpty + s), 1);
      }
      for (int s = 0; s < C::kRawStages; ++s) {
        mbar_init(bar(pbRawFull + s), 1 + 32);  // TMA lane + 32 cp.async arrivals
        mbar_init(bar(pbRawEmpty + s), C::kDqWarps);
      }
      *abort_flag = 0;
      fence_mbar_init();
    }
  } else if (warp >= 4 && warp < 12) {
    // query rows that no token fills (G does not divide 128): zeros, so that their scores are
    const int used = args.G * args.tile_tok;
    const int row = threadIdx.x - 128 - (warp >= 8 ? 128 : 0);
    if (row >= used) {
      uint8_t* q = sgen + C::kOffQ + (warp >= 8 ? C::kQBytes : 0) + row * 128;
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4*>(q + c * (kBM * 128) + i * 16) = make_uint4(0, 0, 0, 0);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool run = *has_run != 0;

  if (warp < 4 || warp >= 12) {
    if (warp == 0) {
      // -------------------------------------------------- scheduler and producer
      bool ok = true;
      int n = 0;      // ring tiles
      int rt = 0;     // raw q4_0 tiles
      int pg = 0;     // paired ring: slots filled
      int qn = 0;     // Q loads issued
      int tails = 0;  // V tiles cleared past the sequence's end
      bool tail_out = false;  // one more is loaded or on its way
      auto box_row = [&](int j) -> int {  // first row in its page of box `lane` of block j
        return PagedWalk::page_row(plan, j * kBN + (lane << args.box_bits));
      };
      auto box_at = [&](int j, int page) -> int {
        return lane < nbox ? w.block_of(plan, j * kBN + (lane << args.box_bits), page,
                                        &g_prefill_paged_error, kErrBadIndex)
                           : -1;
      };
      // dense tile boxes: lane (box, chunk) of 16 copies one box's 64 columns
      auto copy_dense = [&](const CUtensorMap* tm, uint32_t dst, uint32_t full, int at, int row,
                            int i, int c) {
        tma_load_3d(dst + c * (kBN * 128) + i * args.box * 128, tm, full, c * 64, row, at);
      };
      // rows [len, end of its box) of a dense V tile hold no key: clear them once the tile has
      // landed (only the last block of a sequence has such rows)
      auto tail_rows = [&](int j) -> int {  // first such row of the tile, kBN if none
        const int r0 = w.s.len - j * kBN;
        return (r0 > 0 && r0 < kBN && (r0 & (args.box - 1)) != 0) ? r0 : kBN;
      };
      auto clear_tail = [&](uint32_t stage, int r0) -> bool {
        bool w = mbar_wait(bar(pbTail), tails & 1, abort_flag, &g_prefill_paged_error);
        w = __all_sync(0xffffffffu, w);
        tail_out = !w;
        if (!w) return false;
        const int r1 = (r0 + args.box - 1) & -args.box;
        uint8_t* p = sgen + (stage - sbase);
        for (int i = lane; i < (r1 - r0) * 8; i += 32)
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            *reinterpret_cast<uint4*>(p + c * (kBN * 128) + r0 * 128 + i * 16) =
                make_uint4(0, 0, 0, 0);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        ++tails;
        return true;
      };
      const int di = (lane % 16) / kChunks, dc = (lane % 16) % kChunks;  // dense box and chunk
      // one slot of the paired ring: K of block j + 1 (where `k`) by lanes 0-15, at the boxes at_k /
      // row_k that lanes 0 .. nbox - 1 hold, V of block j (where `v`) by lanes 16-31 at at_v / row_v
      auto produce_pair = [&](bool k, int at_k, int row_k, bool v, int j, int at_v, int row_v) {
        const bool vhalf = lane >= 16;
        const int ak = __shfl_sync(0xffffffffu, at_k, di), av = __shfl_sync(0xffffffffu, at_v, di);
        const int rk = __shfl_sync(0xffffffffu, row_k, di);
        const int rv = __shfl_sync(0xffffffffu, row_v, di);
        const int p = pg % C::kSlots;
        if (lane == 0 && pg >= C::kSlots)
          ok = mbar_wait(bar(pbRingEmpty + p), ((pg / C::kSlots) - 1) & 1, abort_flag,
                         &g_prefill_paged_error);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) return;
        const uint32_t dst = sbase + C::kOffRing + 2 * p * C::kTileBytes;
        const int r0 = v ? tail_rows(j) : kBN;  // (below kBN only with k false: the last block)
        if (lane == 0) {
          if (r0 < kBN)
            mbar_arrive_expect_tx(bar(pbTail), C::kTileBytes);
          else
            mbar_arrive_expect_tx(bar(pbRingFull + p),
                                  ((k ? 1 : 0) + (v ? 1 : 0)) * C::kTileBytes);
        }
        __syncwarp();
        if ((vhalf ? v : k) && di < nbox)
          copy_dense(vhalf ? &tm_v : &tm_k, dst + (vhalf ? C::kTileBytes : 0),
                     r0 < kBN ? bar(pbTail) : bar(pbRingFull + p), vhalf ? av : ak,
                     vhalf ? rv : rk, di, dc);
        if (r0 < kBN) {
          ok = clear_tail(dst + C::kTileBytes, r0);
          if (!ok) return;
          if (lane == 0) mbar_arrive(bar(pbRingFull + p));
        }
        ++pg;
      };
      // one tile of the unpaired ring (a q4_0 side), at the boxes that lanes 0 .. nbox - 1 hold
      auto produce = [&](bool is_v, int j, int at, int row) {
        if (!ok) return;
        if (!(is_v ? VQ4 : KQ4)) {
          const int s = n % C::kStages;
          const int da = __shfl_sync(0xffffffffu, at, di), dr = __shfl_sync(0xffffffffu, row, di);
          if (lane == 0 && n >= C::kStages)
            ok = mbar_wait(bar(pbRingEmpty + s), ((n / C::kStages) - 1) & 1, abort_flag,
                           &g_prefill_paged_error);
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) return;
          const uint32_t dst = sbase + C::kOffRing + s * C::kTileBytes;
          const int r0 = is_v ? tail_rows(j) : kBN;
          const uint32_t full = r0 < kBN ? bar(pbTail) : bar(pbRingFull + s);
          if (lane == 0) mbar_arrive_expect_tx(full, C::kTileBytes);
          __syncwarp();
          if (lane < 16 && di < nbox)
            copy_dense(is_v ? &tm_v : &tm_k, dst, full, da, dr, di, dc);
          if (r0 < kBN) {
            ok = clear_tail(dst, r0);
            if (!ok) return;
            if (lane == 0) mbar_arrive(bar(pbRingFull + s));
          }
        } else if constexpr (C::kAnyQ4) {
          const int s = rt % C::kRawStages;
          if (lane == 0 && rt >= C::kRawStages)
            ok = mbar_wait(bar(pbRawEmpty + s), ((rt / C::kRawStages) - 1) & 1, abort_flag,
                           &g_prefill_paged_error);
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) return;
          const uint32_t dst = sbase + C::kOffRaw + s * C::kRawBytes;
          if (lane == 0) mbar_arrive_expect_tx(bar(pbRawFull + s), C::kRawNib);
          __syncwarp();
          if (lane < nbox)
            tma_load_3d(dst + lane * args.box * C::kNibRow, is_v ? &tm_v : &tm_k,
                        bar(pbRawFull + s), 0, row, at);
          // scales: four keys a lane (they share a box), 16 or 32 contiguous bytes, zero past the
          // sequence's end
          const uint8_t* sp = is_v ? args.v_scale : args.k_scale;
          const int kr = 4 * lane, i = kr >> args.box_bits;
          const int kat = __shfl_sync(0xffffffffu, at, i);
          const int krow = __shfl_sync(0xffffffffu, row, i) + (kr & (args.box - 1));
          const int in = kat >= 0 ? max(0, min(4, w.s.len - j * kBN - kr)) : 0;  // keys with data
          const uint8_t* src =
              in > 0 ? sp + (static_cast<int64_t>(kat) * plan.bt.page_size + krow) * C::kScaleRow
                     : sp;
          const uint32_t d = dst + C::kRawNib + kr * C::kScaleRow;
#pragma unroll
          for (int c = 0; c < C::kScaleRow / 4; ++c)
            cp_async_16(d + 16 * c, src + (in > 0 ? 16 * c : 0),
                        static_cast<uint32_t>(max(0, min(16, in * C::kScaleRow - 16 * c))));
          cp_async_mbar_arrive_noinc(bar(pbRawFull + s));
          ++rt;
        }
        ++n;
      };

      int sidx = 0;
      for (; w.t < w.t_end && ok; ++sidx) {
        // the unit's segment of this run
        const int tokA = min(args.tile_tok, w.s.nq - w.tok);
        const int tokB = max(0, min(args.tile_tok, w.s.nq - w.tok - args.tile_tok));
        const int j0 = w.j0(plan), j1 = w.j1(plan);
        if (lane == 0 && sidx >= kSegQ)
          ok = mbar_wait(bar(pbSegEmpty + sidx % kSegQ), ((sidx / kSegQ) - 1) & 1, abort_flag,
                         &g_prefill_paged_error);
        if (lane == 0 && ok) {
          PSeg* s = seg_at(sidx);
          s->row0 = w.s.start + w.tok;
          s->g = w.g;
          s->tokA = tokA;
          s->tokB = tokB;
          s->pos0 = w.s.len - w.s.nq + w.tok;
          s->len = w.s.len;
          s->nbA = plan.blocks(w.s, w.tok + args.tile_tok);
          s->nbB = tokB > 0 ? w.nb : 0;
          s->j0 = j0;
          s->j1 = j1;
          int c_first, c_last, slot_first;
          w.pieces(plan, cta, c_first, c_last, slot_first);
          s->c_first = c_first;
          s->c_last = c_last;
          s->slot_first = slot_first;
          s->own_slot = c_first == cta ? slot_first : 0;
          mbar_arrive(bar(pbSegFull + sidx % kSegQ));
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
        // the segment's Q tiles, once the previous segment's last QK has read the previous ones
        auto load_q = [&]() {
          if (lane == 0) {
            if (sidx > 0)
              ok = mbar_wait(bar(pbQEmpty), (sidx - 1) & 1, abort_flag, &g_prefill_paged_error);
            if (ok) {
              const uint32_t bytes = kChunks * args.tile_tok * args.G * 128;
              mbar_arrive_expect_tx(bar(pbQFull), (tokB > 0 ? 2 : 1) * bytes);
              for (int ti = 0; ti < (tokB > 0 ? 2 : 1); ++ti)
                for (int c = 0; c < kChunks; ++c)
                  tma_load_3d(sbase + C::kOffQ + ti * C::kQBytes + c * (kBM * 128), &tm_q,
                              bar(pbQFull), c * 64, w.g * args.G,
                              w.s.start + w.tok + ti * args.tile_tok);
              ++qn;
            }
          }
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        };
        // block j's boxes, and the pages of block j + 1, looked up while block j is waited for.  A
        // later segment's first K tile goes ahead of its Q tiles: it waits for a ring slot only.
        if (sidx == 0) load_q();
        int at = box_at(j0, page0), row = box_row(j0);
        int next = j0 + 1 < j1 ? look_up(j0 + 1) : -1;
        if constexpr (C::kPaired) {
          if (ok) produce_pair(true, at, row, false, 0, -1, 0);
          if (sidx > 0 && ok) load_q();
          for (int j = j0; j < j1 && ok; ++j) {
            const int at_v = at, row_v = row;
            const bool more = j + 1 < j1;
            if (more) {
              at = box_at(j + 1, next);
              row = box_row(j + 1);
              if (j + 2 < j1) next = look_up(j + 2);
            }
            produce_pair(more, at, row, true, j, at_v, row_v);
          }
        } else {
          // K0 V0 K1 V1 ..., or, where a lone tile's blocks alternate, K0 K1 V0 K2 V1 ...
          const bool ahead = kAlt && tokB == 0;
          produce(false, j0, at, row);
          if (sidx > 0 && ok) load_q();
          for (int j = j0; j < j1 && ok; ++j) {
            const int at_v = at, row_v = row;
            if (!ahead) produce(true, j, at_v, row_v);
            if (j + 1 < j1) {
              at = box_at(j + 1, next);
              row = box_row(j + 1);
              if (j + 2 < j1) next = look_up(j + 2);
              produce(false, j + 1, at, row);
            }
            if (ahead) produce(true, j, at_v, row_v);
          }
        }
        w.next(plan);
        if (w.t < w.t_end) page0 = look_up(0);
      }
      if (ok && run && lane == 0) {
        // end of the run
        if (sidx >= kSegQ)
          ok = mbar_wait(bar(pbSegEmpty + sidx % kSegQ), ((sidx / kSegQ) - 1) & 1, abort_flag,
                         &g_prefill_paged_error);
        if (ok) {
          seg_at(sidx)->j1 = -1;
          mbar_arrive(bar(pbSegFull + sidx % kSegQ));
        }
      }
      if constexpr (C::kAnyQ4) {
        // the dequant warps learn of the end as of one more raw tile
        if (ok && run) {
          const int s = rt % C::kRawStages;
          if (lane == 0 && rt >= C::kRawStages)
            ok = mbar_wait(bar(pbRawEmpty + s), ((rt / C::kRawStages) - 1) & 1, abort_flag,
                           &g_prefill_paged_error);
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (lane == 0) {
            *raw_end = rt;
            if (ok) mbar_arrive(bar(pbRawFull + s));
          }
          __syncwarp();
          if (ok) mbar_arrive(bar(pbRawFull + s));
        }
      }
      if (!ok && lane == 0) {
        // let copies already issued land before the CTA's shared memory goes away
        volatile int never = 0;
        if (qn > 0) mbar_wait(bar(pbQFull), (qn - 1) & 1, &never, nullptr, kWaitLimitNs);
        if (tail_out) mbar_wait(bar(pbTail), tails & 1, &never, nullptr, kWaitLimitNs);
        if constexpr (C::kPaired) {
          for (int i = max(0, pg - C::kSlots); i < pg; ++i)
            mbar_wait(bar(pbRingFull + i % C::kSlots), (i / C::kSlots) & 1, &never, nullptr,
                      kWaitLimitNs);
        }
        for (int i = max(0, n - C::kStages); i < n; ++i)
          if (!((i & 1) ? VQ4 : KQ4))
            mbar_wait(bar(pbRingFull + i % C::kStages), (i / C::kStages) & 1, &never, nullptr,
                      kWaitLimitNs);
        if constexpr (C::kAnyQ4) {
          for (int i = max(0, rt - C::kRawStages); i < rt; ++i)
            mbar_wait(bar(pbRawFull + i % C::kRawStages), (i / C::kRawStages) & 1, &never,
                      nullptr, kWaitLimitNs);
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA issuer
      if (lane == 0 && run) {
        constexpr uint32_t idesc_qk = make_idesc_f16(kBM, kBN, BF16, false);
        constexpr uint32_t idesc_pv = make_idesc_f16(kBM, D, BF16, true);
        bool ok = true;
        int n = 0, gn = 0;       // ring tiles / paired slots taken
        int prA = 0, prB = 0, prAlt = 0;  // P-ready waits before this segment (barrier phases)
        int actA = 0, actB = 0;  // earlier segments in which the tile had blocks
        auto acquire_g = [&]() -> int {
          const int p = gn % C::kSlots;
          if (ok) ok = mbar_wait(bar(pbRingFull + p), (gn / C::kSlots) & 1, abort_flag,
                                 &g_prefill_paged_error);
          tc_fence_after();
          ++gn;
          return p;
        };
        auto acquire = [&]() -> int {
          const int s = n % C::kStages;
          if (ok) ok = mbar_wait(bar(pbRingFull + s), (n / C::kStages) & 1, abort_flag,
                                 &g_prefill_paged_error);
          tc_fence_after();
          ++n;
          return s;
        };
        auto release = [&](int s) { mma_commit(bar(pbRingEmpty + s)); };
        // QK of tile t into S buffer sb (its own, or either for a lone tile A)
        auto issue_qk = [&](int t, int s, int sb, int full) {
          const uint32_t qaddr = sbase + C::kOffQ + t * C::kQBytes;
          const uint32_t kaddr = sbase + C::kOffRing + s * C::kTileBytes;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * (kBM * 128) + (kk & 3) * 32;
            mma_ss(tmem + col_s(sb), make_sdesc_sw128(qaddr + off, 16, 1024),
                   make_sdesc_sw128(kaddr + off, 16, 1024), idesc_qk, kk > 0 ? 1u : 0u);
          }
          mma_commit(bar(full));
        };
        auto issue_pv = [&](int t, int j, int s, int j0, int e_t, int pb) {
          ok = ok && mbar_wait(bar(pbPReady + t), (pb + j) & 1, abort_flag,
                               &g_prefill_paged_error);
          if (!ok) return;
          tc_fence_after();
          const uint32_t vaddr = sbase + C::kOffRing + s * C::kTileBytes;
          const uint32_t ocol = t ? C::kColO1 : C::kColO0;
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)
            mma_ts(tmem + ocol, tmem + col_s(t) + kk * 8,
                   make_sdesc_sw128(vaddr + kk * (16 * 128), kBN * 128, 1024), idesc_pv,
                   (j > j0 || kk > 0) ? 1u : 0u);
          if (j == e_t - 1) mma_commit(bar(pbODone + t));
        };
        // per segment: QK_A(j0) QK_B(j0) | PV_A(j) QK_A(j+1) PV_B(j) QK_B(j+1) | ...
        for (int sidx = 0; ok; ++sidx) {
          ok = mbar_wait(bar(pbSegFull + sidx % kSegQ), (sidx / kSegQ) & 1, abort_flag,
                         &g_prefill_paged_error);
          if (!ok) break;
          const PSeg sg = read_seg(segs + (sidx % kSegQ) * 64);
          const int j0 = sg.j0, j1 = sg.j1;
          if (j1 < 0) break;
          const int eA = min(j1, sg.nbA), eB = min(j1, sg.nbB);
          const bool sp_lone = sg.tokB == 0;
          mbar_arrive(bar(pbSegEmpty + sidx % kSegQ));
          ok = mbar_wait(bar(pbQFull), sidx & 1, abort_flag, &g_prefill_paged_error);
          tc_fence_after();
          if (!ok) break;
          const int pbA = prA - j0, pbB = prB - j0;
          if (kAlt && sp_lone) {
            // a lone tile A: its blocks alternate between the two S buffers, so that QK(j + 1) is
            // done while the softmax is at block j: QK(j0) QK(j0+1) | PV(j) QK(j+2) | ...
            auto take = [&]() -> int {  // the next K (paired ring: with the V before it)
              return C::kPaired ? 2 * acquire_g() : acquire();
            };
            auto qk = [&](int j, int s) {
              const int sb = (j - j0) & 1;
              issue_qk(0, s, sb, sb ? pbSAlt : pbSFull);
              if (j + 1 == j1) mma_commit(bar(pbQEmpty));
            };
            int s = take();
            if (!ok) break;
            qk(j0, s);
            release(C::kPaired ? s / 2 : s);
            if (C::kPaired || j0 + 1 < j1) {
              s = take();  // paired: V(j0) and K(j0 + 1)
              if (!ok) break;
              if (j0 + 1 < j1) qk(j0 + 1, s);
              if (!C::kPaired) release(s);
            }
            if (actA > 0)
              ok = ok && mbar_wait(bar(pbOFree + 0), (actA - 1) & 1, abort_flag,
                                   &g_prefill_paged_error);
            for (int j = j0; j < j1 && ok; ++j) {
              const int sb = (j - j0) & 1;
              if (!C::kPaired) s = acquire();
              ok = ok && mbar_wait(bar(sb ? pbPAlt : pbPReady), (sb ? prAlt++ : prA++) & 1,
                                   abort_flag, &g_prefill_paged_error);
              if (!ok) break;
              tc_fence_after();
              const uint32_t vaddr =
                  sbase + C::kOffRing + (C::kPaired ? s + 1 : s) * C::kTileBytes;
#pragma unroll
              for (int kk = 0; kk < kBN / 16; ++kk)
                mma_ts(tmem + C::kColO0, tmem + col_s(sb) + kk * 8,
                       make_sdesc_sw128(vaddr + kk * (16 * 128), kBN * 128, 1024), idesc_pv,
                       (j > j0 || kk > 0) ? 1u : 0u);
              mma_commit(bar(pbPvAlt));
              if (j == j1 - 1) mma_commit(bar(pbODone));
              release(C::kPaired ? s / 2 : s);
              if (C::kPaired ? j + 1 < j1 : j + 2 < j1) {
                s = take();
                if (!ok) break;
                if (j + 2 < j1) qk(j + 2, s);
                if (!C::kPaired) release(s);
              }
            }
            ++actA;
            continue;
          }
          if constexpr (C::kPaired) {
            {
              const int p = acquire_g();
              if (!ok) break;
              if (j0 < eA) issue_qk(0, 2 * p, 0, pbSFull);
              if (j0 < eB)
                issue_qk(1, 2 * p, 1, pbSFull + 1);  // tile B's softmax releases the slot
              else
                release(p);
              if (j0 + 1 == j1) mma_commit(bar(pbQEmpty));
            }
            if (j0 < eA && actA > 0)
              ok = ok && mbar_wait(bar(pbOFree + 0), (actA - 1) & 1, abort_flag,
                                   &g_prefill_paged_error);
            if (j0 < eB && actB > 0)
              ok = ok && mbar_wait(bar(pbOFree + 1), (actB - 1) & 1, abort_flag,
                                   &g_prefill_paged_error);
            for (int j = j0; j < j1 && ok; ++j) {
              const int p = acquire_g();
              const bool next = j + 1 < j1;
              if (!ok) break;
              if (j < eA) issue_pv(0, j, 2 * p + 1, j0, eA, pbA);
              if (!ok) break;
              if (next && j + 1 < eA) issue_qk(0, 2 * p, 0, pbSFull);
              if (j < eB) issue_pv(1, j, 2 * p + 1, j0, eB, pbB);
              if (!ok) break;
              if (next && j + 1 < eB)
                issue_qk(1, 2 * p, 1, pbSFull + 1);
              else
                release(p);
              if (next && j + 2 == j1) mma_commit(bar(pbQEmpty));
            }
          } else {
            {
              const int sK = acquire();
              if (!ok) break;
              if (j0 < eA) issue_qk(0, sK, 0, pbSFull);
              if (j0 < eB) issue_qk(1, sK, 1, pbSFull + 1);
              release(sK);
              if (j0 + 1 == j1) mma_commit(bar(pbQEmpty));
            }
            if (j0 < eA && actA > 0)
              ok = ok && mbar_wait(bar(pbOFree + 0), (actA - 1) & 1, abort_flag,
                                   &g_prefill_paged_error);
            if (j0 < eB && actB > 0)
              ok = ok && mbar_wait(bar(pbOFree + 1), (actB - 1) & 1, abort_flag,
                                   &g_prefill_paged_error);
            for (int j = j0; j < j1 && ok; ++j) {
              const int sV = acquire();
              const bool next = j + 1 < j1;
              const int sK = next ? acquire() : 0;
              if (!ok) break;
              if (j < eA) issue_pv(0, j, sV, j0, eA, pbA);
              if (!ok) break;
              if (next && j + 1 < eA) issue_qk(0, sK, 0, pbSFull);
              if (j < eB) issue_pv(1, j, sV, j0, eB, pbB);
              if (!ok) break;
              release(sV);
              if (next) {
                if (j + 1 < eB) issue_qk(1, sK, 1, pbSFull + 1);
                release(sK);
                if (j + 2 == j1) mma_commit(bar(pbQEmpty));
              }
            }
          }
          if (j0 < eA) {
            ++actA;
            prA += eA - j0;
          }
          if (j0 < eB) {
            ++actB;
            prB += eB - j0;
          }
        }
        if (!ok) {
          // wait until every MMA issued so far has finished before TMEM is released
          volatile int never = 0;
          mma_commit(bar(pbDrain));
          mbar_wait(bar(pbDrain), 0, &never, nullptr, kWaitLimitNs);
        }
      }
    } else if constexpr (C::kAnyQ4) {
      if (C::is_dq_warp(warp)) {
        // -------------------------------------------------------------- q4_0 dequant
        const int u = C::dq_index(warp, lane);
        const uint32_t mg = opaque_u32(BF16 ? 0x43004300u : 0x64006400u);
        bool ok = true;
        int r = 0;  // raw q4_0 tiles consumed
        for (int n = 0; run; ++n) {
          if (!((n & 1) ? VQ4 : KQ4)) continue;  // a dense tile: the producer's TMA fills it
          const int rs = r % C::kRawStages;
          const int s = n % C::kStages;
          ok = mbar_wait(bar(pbRawFull + rs), (r / C::kRawStages) & 1, abort_flag,
                         &g_prefill_paged_error);
          if (!ok || r >= *raw_end) break;
          if (n >= C::kStages)
            ok = mbar_wait(bar(pbRingEmpty + s), ((n / C::kStages) - 1) & 1, abort_flag,
                           &g_prefill_paged_error);
          if (!ok) break;
          const uint8_t* raw = sgen + C::kOffRaw + rs * C::kRawBytes;
          uint8_t* dst = sgen + C::kOffRing + s * C::kTileBytes;
          constexpr int kItems = kBN * (D / 32);
#pragma unroll
          for (int k = 0; k < (kItems + C::kDqThreads - 1) / C::kDqThreads; ++k) {
            const int it = u + k * C::kDqThreads;
            if (kItems % C::kDqThreads == 0 || it < kItems)
              dequant_item<D, BF16, C::kNibRow, C::kScaleRow, C::kRawNib,
                           typename DqOf<BF16>::type>(raw, dst, it % kBN, it / kBN, mg);
          }
          // generic-proxy writes must be visible to the tensor core's async proxy
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(pbRingFull + s));
            mbar_arrive(bar(pbRawEmpty + rs));
          }
          ++r;
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax rows
    // Registers: a block's 128 scores (with a q4_0 side 64, and 64 as P) and little else.  Nothing but
    // the two words below is carried from one segment to the next, and what follows from the thread's
    // number or the segment is formed again where it is used: values kept across the block loop, or
    // across the call that ends a cut segment, would be spilled inside it (measured: 343 -> 383 us on
    // the 2048-token chunk at 16384 f16 keys).
    enum : uint32_t {
      kPhS = 1,       // barrier phases: S-full,
      kPhAlt = 2,     // S-full of the second buffer,
      kPhPv = 4,      // PVs of a lone tile,
      kPhO = 8,       // O-done
      kLone = 16,     // the segment: its tile is alone (its blocks alternate),
      kLive = 32,     // some row of the warp is in use,
      kLater = 64,    // O holds earlier blocks,
      kSecond = 128,  // the block uses the second buffer,
      kTileB = 256,
      kFirstCut = 512  // the run's first segment was a piece
    };
    uint32_t st = 0;
    int ks = 0;  // paired ring: the slot that holds the block's K
    const uint32_t stop = bar0 + kOffAbort;
    volatile uint32_t* decisions = reinterpret_cast<volatile uint32_t*>(bgen + kOffMerge);
    bool open = false;    // the loop was left with a segment whose rows are still in tensor memory
    int sidx = 0;
    uint32_t tm = 0;      // this warp's TMEM lanes
    float f = -INFINITY;  // frame, base-2 units of the scaled score
    float l = 0.f;
    for (; run; ++sidx) {
      bool ok = wait_bounded(bar(pbSegFull + sidx % kSegQ), (sidx / kSegQ) & 1, stop);
      if (!__all_sync(0xffffffffu, ok)) break;
      int left;      // blocks of this tile still to come
      int rel;       // last key that this thread's row sees, relative to the block
      f = -INFINITY;
      l = 0.f;
      {
        const PSeg sg = read_seg(segs + (sidx % kSegQ) * 64);
        const int j0 = sg.j0, j1 = sg.j1;
        if (j1 < 0) break;
        const int tid = opaque_tid();
        const int t = tid >= 256 ? 1 : 0, row = tid & 127;
        const int ntok = t ? sg.tokB : sg.tokA;
        left = ntok > 0 ? max(0, min(j1, t ? sg.nbB : sg.nbA) - j0) : 0;
        const int last = sg.len - 1;
        rel = (plan.causal ? min(last, sg.pos0 + t * args.tile_tok + row / args.G) : last) -
              j0 * kBN;
        st = (st & (kPhS | kPhAlt | kPhPv | kPhO | kFirstCut)) | (t ? kTileB : 0) |
             ((row & ~31) < ntok * args.G ? kLive : 0) | (kAlt && sg.tokB == 0 ? kLone : 0);
        tm = *reinterpret_cast<volatile uint32_t*>(tmem_slot) +
             (static_cast<uint32_t>(row & ~31) << 16);
      }
      for (; left > 0; --left) {
        const int t = st & kTileB ? 1 : 0;
        ok = wait_bounded(bar(st & kSecond ? pbSAlt : pbSFull + t),
                          st & kSecond ? (st >> 1) & 1 : st & 1, stop);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        st ^= st & kSecond ? kPhAlt : kPhS;
        tc_fence_after();
        if constexpr (C::kPaired) {
          // QK_B of the block done: release the ring slot holding its K
          if (opaque_tid() == 256) mbar_arrive(bar(pbRingEmpty + ks));
          if (++ks == C::kSlots) ks = 0;
        }
        if (st & kLive) {
          // a lone tile's PV of the block before may still be adding to O when this block moves the
          // frame; its own PV cannot have started, so the PVs done are all but one or all
          auto wait_pv = [&]() {
            if (st & kLone) {
              wait_bounded(bar(pbPvAlt), ((st >> 2) & 1) ^ 1, stop);
              tc_fence_after();
            }
          };
          const uint32_t scol = tm + (st & (kSecond | kTileB) ? col_s(1) : col_s(0));
          const uint32_t ocol = tm + (st & kTileB ? C::kColO1 : C::kColO0);
          const bool mask = __any_sync(0xffffffffu, rel < kBN - 1);
          if constexpr (C::kWide) {
            softmax_block_lean<D, BF16>(scol, ocol, mask, rel, args.scale_log2, (st & kLater) != 0,
                                        f, l, wait_pv);
          } else {
            int moves = 0;
            float top = 0.f;
            softmax_block<D, BF16>(scol, ocol, mask, rel, args.scale_log2, (st & kLater) != 0, f,
                                   l, moves, top, wait_pv);
          }
          tmem_wait_st();
        }
        rel -= kBN;
        tc_fence_before();
        mbar_arrive(bar(st & kSecond ? pbPAlt : pbPReady + (st & kTileB ? 1 : 0)));
        st |= kLater;
        if (st & kLone) st ^= kSecond | kPhPv;
      }
      if (!ok) break;
      open = true;
      const PSeg sg = read_seg(segs + (sidx % kSegQ) * 64);
      const int tid = opaque_tid();
      const int t = tid >= 256 ? 1 : 0, row = tid & 127;  // query tile, this thread's row
      const int rtok = row / args.G;                      // the row's token within the tile
      const int ntok = t ? sg.tokB : sg.tokA;
      const uint32_t ocol = tm + (t ? C::kColO1 : C::kColO0);
      if constexpr (C::kPaired) {
        const int j0 = sg.j0, j1 = sg.j1;
        const int n = ntok > 0 ? max(0, min(j1, t ? sg.nbB : sg.nbA) - j0) : 0;
        ks = (ks + j1 - j0 - n + 1) % C::kSlots;
      }
      if (sg.c_last != cta) break;  // the run ends inside the unit: below
      const bool cut = sg.c_first != cta;
      if (st & kLater) {  // the tile had key blocks in this segment
        ok = wait_bounded(bar(pbODone + t), (st >> 3) & 1, stop);
        st ^= kPhO;
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
      }
      const bool valid = rtok < ntok && row < args.G * args.tile_tok;
      // (its first key is in the segment's first block if any is; f alone does not say: a row of NaN
      // scores leaves it at -inf)
      const bool sees = last_key(sg, plan.causal, t * args.tile_tok + rtok) >= sg.j0 * kBN;
      if (cut) {  // the last piece of a unit that other CTAs began
        if (st & kLive)
          store_piece<D>(args, 0, t, row, ocol, (st & kLater) != 0, valid, piece_frame(sees, f, l), l);
      } else if ((st & kLater) && (st & kLive)) {
        const bool none = !sees;
        const float inv_l = 1.f / l;
        uint8_t* orow = args.o + (sg.row0 + t * args.tile_tok + rtok) * args.o_row_stride +
                        (sg.g * args.G + (row - rtok * args.G)) * args.o_head_stride;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld32(ocol + 32 * c, r);
          tmem_wait_ld();
          reg_fence32(r);
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            pk[i] = none ? 0u
                         : pack2<BF16>(__uint_as_float(r[2 * i]) * inv_l,
                                       __uint_as_float(r[2 * i + 1]) * inv_l);
          if (valid) {
            uint4* dst = reinterpret_cast<uint4*>(orow + c * 64);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dst[i] = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
          }
        }
      }
      if (st & kLater) {
        // O has been read out of tensor memory: the next segment's PV may overwrite it
        tc_fence_before();
        mbar_arrive(bar(pbOFree + t));
      }
      if (cut) {
        // published at once; if the others were there before it, its merge waits for the run's end
        mbar_arrive(bar(pbPiece));
        if (tid >= 352) {  // (a warp of tile B: of a lone tile's segment, one with nothing else to do)
          const bool all = publish_piece(args, sg, bar(pbPiece), stop);
          if (lane == 0) {
            *reinterpret_cast<PSeg*>(bgen + kOffFirst) = sg;
            decisions[0] = all ? 1u : 0u;
            mbar_arrive(bar(pbDecided));
          }
        }
        st |= kFirstCut;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(pbSegEmpty + sidx % kSegQ));
      open = false;
    }
    // The run's last segment, if others go on with its unit.  Where all their pieces are published by
    // now, nobody else can merge: this CTA does, without publishing its own -- from tensor memory
    // where the pieces are few.  Else the piece is stored and published, and merged if all are
    // there then.
    if (open && run) {
      const PSeg sg = read_seg(segs + (sidx % kSegQ) * 64);
      const int t = warp >= 8 ? 1 : 0, row = threadIdx.x & 127;
      const int ntok = t ? sg.tokB : sg.tokA;
      const bool active = (st & kLater) != 0;
      const bool valid = row / args.G < ntok && row < args.G * args.tile_tok;
      const uint32_t ocol = tm + (t ? C::kColO1 : C::kColO0);
      f = piece_frame(active && last_key(sg, plan.causal, t * args.tile_tok + row / args.G) >=
                                    sg.j0 * kBN,
                      f, l);
      bool ok = true;
      if (warp == 4) {
        const bool early = pieces_there(args, sg, cta);
        if (lane == 0) {
          decisions[2] = early ? 1u : 0u;
          mbar_arrive(bar(pbEarly));
        }
      }
      if (active) {
        ok = wait_bounded(bar(pbODone + t), (st >> 3) & 1, stop);
        tc_fence_after();
      }
      ok = wait_bounded(bar(pbEarly), 0, stop) && ok;
      if (__all_sync(0xffffffffu, ok)) {
        const bool early = decisions[2] != 0u;
        if (early && sg.c_last - sg.c_first == 1) {
          if (st & kLive)
            merge_with_own<D, BF16, C::kWide ? 64 : D>(args, sg, t, row, ocol, active, valid, f, l);
          if (warp == 4) clear_flags(args, sg);
        } else {
          if (st & kLive) store_piece<D>(args, sg.own_slot, t, row, ocol, active, valid, f, l);
          mbar_arrive(bar(pbPiece + 1));
          if (warp == 4) {
            const bool all = early ? __all_sync(0xffffffffu, wait_bounded(bar(pbPiece + 1), 0, stop))
                                   : publish_piece(args, sg, bar(pbPiece + 1), stop);
            if (lane == 0) {
              decisions[1] = all ? 1u : 0u;
              mbar_arrive(bar(pbDecided + 1));
            }
          }
          ok = wait_bounded(bar(pbDecided + 1), 0, stop);
          if (__all_sync(0xffffffffu, ok) && decisions[1] != 0u) {
            merge_pieces<D, BF16>(args, sg);
            if (warp == 4) clear_flags(args, sg);
          }
        }
      }
    }
    // the first segment's unit, if its other pieces were there before this CTA's
    if (st & kFirstCut) {
      const bool ok = wait_bounded(bar(pbDecided), 0, stop);
      if (__all_sync(0xffffffffu, ok) && decisions[0] != 0u) {
        const PSeg sg = read_seg(bar0 + kOffFirst);
        merge_pieces<D, BF16>(args, sg);
        if (warp == 4) clear_flags(args, sg);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_flag) st_relaxed_gpu(abandoned_tag(args), args.tag);
}

size_t flag_bytes(int num_sms) {
  return (static_cast<size_t>(num_sms) * 2 + 1) * sizeof(uint32_t);
}

template <int D, bool BF16, bool KQ4, bool VQ4>
cudaError_t launch_t(const PagedPrefillLaunch& L, cudaStream_t stream) {
  using C = Cfg<D, KQ4, VQ4, true>;
  static_assert(C::kSmemBytes <= 227 * 1024, "shared memory budget");
  auto kern = prefill_paged_kernel<D, BF16, KQ4, VQ4>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             C::kSmemBytes);
  if (e != cudaSuccess) return e;
  PArgs a;
  a.o = static_cast<uint8_t*>(L.o);
  a.o_row_stride = 2 * L.o_row_stride;
  a.o_head_stride = 2 * L.o_head_stride;
  a.k_scale = static_cast<const uint8_t*>(L.k_scale);
  a.v_scale = static_cast<const uint8_t*>(L.v_scale);
  a.G = L.Hq / L.Hkv;
  a.tile_tok = kBM / a.G;
  a.plan = PagedPlan{L.batch, DivBy(L.batch.page_size), L.Hkv, L.causal, 2 * a.tile_tok};
  a.box = L.box;
  a.box_bits = L.box_bits;
  a.scale_log2 = L.scale * kLog2e;
  a.pflags = static_cast<uint32_t*>(L.workspace);
  // the pieces' columns are whole 128-byte lines: from a 256-byte boundary on
  a.part = reinterpret_cast<float*>(
      (reinterpret_cast<uintptr_t>(L.workspace) + flag_bytes(L.num_sms) + 255) / 256 * 256);
  a.tag = L.tag;
  kern<<<L.num_sms, C::kThreads, C::kSmemBytes, stream>>>(L.tm_q, L.tm_k, L.tm_v, a);
  return cudaGetLastError();
}

template <int D, bool BF16>
cudaError_t launch_fmt(const PagedPrefillLaunch& L, cudaStream_t stream) {
  if (L.kq4) return L.vq4 ? launch_t<D, BF16, true, true>(L, stream)
                          : launch_t<D, BF16, true, false>(L, stream);
  return L.vq4 ? launch_t<D, BF16, false, true>(L, stream)
               : launch_t<D, BF16, false, false>(L, stream);
}

}  // namespace

// publication flags and the word behind them, then the partial rows: two slots of two tiles for every CTA
size_t paged_prefill_workspace(int D, int num_sms) {
  const size_t n = static_cast<size_t>(num_sms);
  return flag_bytes(num_sms) + 255 + n * 4 * (D + 2) * kBM * sizeof(float);
}

cudaError_t paged_prefill_launch(const PagedPrefillLaunch& L, cudaStream_t stream) {
  if (L.D == 128)
    return L.bf16 ? launch_fmt<128, true>(L, stream) : launch_fmt<128, false>(L, stream);
  return L.bf16 ? launch_fmt<64, true>(L, stream) : launch_fmt<64, false>(L, stream);
}

uint32_t paged_prefill_take_error() {
  uint32_t v = 0;
  if (cudaMemcpyFromSymbol(&v, g_prefill_paged_error, sizeof(v)) != cudaSuccess)
    return 0xffffffffu;
  const uint32_t z = 0;
  cudaMemcpyToSymbol(g_prefill_paged_error, &z, sizeof(z));
  return v;
}

}  // namespace fa
