// Writing new tokens into page pools (fa_append_paged) and reading tokens back out of them
// (fa_read_paged), each pool dense or q4_0.  This is the paged form of the step that keeps the cache
// quantized ("FlashAttention on gfx90a: Why It's Broken and How to Fix It", Impact of the V Dequant
// Patch, -ctk q4_0 -ctv q4_0).
//
// Both move every byte once and are bound by HBM bandwidth when there are many rows, by the latency
// of their dependent loads (batch description, then page table, then data) when there are few.  A CTA
// takes 16 packed rows of K or of V at a time: its threads first find the rows' places in the pool
// together (an append's first loads, which do not depend on them, are already under way), then
// walk the rows head by head, so that the 16 rows of a head, neighbours in a page, are stored as
// one run: 16 x 64 bytes of nibbles and 16 x 8 bytes of scales at D = 128.  A thread keeps its row
// and its part of the head for all of them.
//
// Measured (one GB300, 8 kv heads, D = 128, K and V): 4 x 16384 rows read out of f16 pools 82 us (6.5
// TB/s), out of q4_0 pools 56 us (6.1 TB/s); 4 x 2048 bf16 rows appended to q4_0 pools and read back
// 25 us, the append alone 15.4, into dense pools 14.7; 64 rows appended and read back 6.0 us.  With 16
// bytes of the dense row a thread, integer conversions and run-time divisions in the loop the first
// three and the last took 86, 87, 31 and 11 us.
#include <algorithm>

#include "fa_internal.h"
#include "fa_paged.cuh"
#include "fa_ptx.cuh"
#include "fa_quant.cuh"

namespace fa {

__device__ uint32_t g_paged_error;

namespace {

constexpr int kTok = 16;        // packed rows that the threads of a CTA cover at once
constexpr int kThreads = 256;
constexpr int kGroups = 8;      // most groups of kTok rows per CTA
constexpr int kDeep = 2;        // passes whose loads are in flight together (4: 25.7 for 23.8 us of
                                // the 4 x 2048 rows above, for the registers they take)
constexpr int kSmemSeqs = 1024; // batches up to this size keep starts and lens in shared memory

// Places of the n rows from t0 on in the pool: row_of[i] = the pool row (of D elements) of kv
// head 0, head h's being h * page_size further, or -1 for a row that belongs to no sequence or
// whose place is out of range (recorded).  False, with nothing to do, when starts is not a rising
// run within the tensors (recorded).  Ends with a barrier.
__device__ __forceinline__ bool locate_rows(const PagedBatch& b, int Hkv, int t0, int n,
                                            int64_t* row_of) {
  __shared__ int32_t s_starts[kSmemSeqs + 1];
  __shared__ int32_t s_lens[kSmemSeqs];
  const int tid = threadIdx.x;
  const bool small = b.B <= kSmemSeqs;
  const int64_t cap = static_cast<int64_t>(b.page_size) * b.pages_per_seq;
  int bad = 0;
  for (int i = tid; i < b.B; i += kThreads) {
    const int v = __ldg(b.starts + i), next = __ldg(b.starts + i + 1);
    if (small) s_lens[i] = __ldg(b.lens + i);
    bad |= bad_start(v, next, b.rows);
    if (small) {
      s_starts[i] = v;
      if (i == b.B - 1) s_starts[b.B] = next;
    }
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) atomicCAS(&g_paged_error, kErrNone, kErrBadIndex);
    return false;
  }
  const int32_t* starts = small ? s_starts : b.starts;
  const int32_t* lens = small ? s_lens : b.lens;
  if (tid < n) {
    const int t = t0 + tid;
    int64_t row = -1;
    if (t >= starts[0] && t < starts[b.B]) {
      int lo = 0, hi = b.B;  // the last sequence that starts at or before row t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= t) lo = mid; else hi = mid;
      }
      const int pos = row_position(lens[lo], cap, starts[lo + 1] - t);
      if (pos >= 0) {
        const int lp = pos / b.page_size;
        const int page = __ldg(b.table + static_cast<int64_t>(lo) * b.pages_per_seq + lp);
        if (page >= 0 && page < b.num_pages)
          row = static_cast<int64_t>(page) * Hkv * b.page_size + (pos - lp * b.page_size);
      }
      if (row < 0) atomicCAS(&g_paged_error, kErrNone, kErrBadIndex);
    }
    row_of[tid] = row;
  } else if (tid >= kTok * kGroups && (blockIdx.x | blockIdx.y | blockIdx.z) == 0) {
    // meanwhile one CTA's other threads record bad lengths, of sequences without rows too
    for (int i = tid - kTok * kGroups; i < b.B; i += kThreads - kTok * kGroups)
      if (bad_length(lens[i], cap)) atomicCAS(&g_paged_error, kErrNone, kErrBadIndex);
  }
  __syncthreads();
  return true;
}

// The two values of codes in the low nibbles of bytes 0 and 1 of w: (code - 8) d, exact before the
// one rounding to the type.  A code becomes a float in the low mantissa bits of 2^10 (f16) or 2^23
// (f32, for bf16: its product with an f16 scale needs more bits than bf16 holds); conversions from
// integers run at a quarter of the rate.
template <bool BF16>
__device__ __forceinline__ uint32_t q4_pair(uint32_t w, __half d) {
  if constexpr (BF16) {
    const float f = __half2float(d);
    const float x0 = __uint_as_float((w & 15u) | 0x4B000000u) - 8388616.f;
    const float x1 = __uint_as_float(((w >> 8) & 15u) | 0x4B000000u) - 8388616.f;
    return pack2<true>(__fmul_rn(x0, f), __fmul_rn(x1, f));
  } else {
    const uint32_t bits = __byte_perm(w & 0x0F0Fu, 0x64u, 0x4140);
    const __half2 x = __hsub2(reinterpret_cast<const __half2&>(bits), __float2half2_rn(1032.f));
    const __half2 o = __hmul2_rn(x, __half2half2(d));
    return reinterpret_cast<const uint32_t&>(o);
  }
}

// Quantization of a block by two neighbouring lanes: lane 0 of the pair holds elements 0-7 (lo) and
// 16-23 (hi), lane 1 the 8 after each, so that a lane's codes share its 8 bytes of nibbles.  The
// arithmetic of q4_quantize_block: m / -8 and 1 / d are the same correctly rounded values by a
// product and a reciprocal, and a code's truncation is that of an addition rounded to zero (a NaN
// gives code 0 in both).
template <bool BF16>
__device__ __forceinline__ uint2 q4_quantize_half(uint4 lo, uint4 hi, bool second, __half& scale) {
  const uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  float v[16];
  float m[2];  // the first of largest magnitude of each half
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    m[x] = 0.f;
#pragma unroll
    for (int j = 8 * x; j < 8 * x + 8; ++j) {
      v[j] = q4_to_f32<BF16>(static_cast<uint16_t>(u[j >> 1] >> (16 * (j & 1))));
      if (fabsf(v[j]) > fabsf(m[x])) m[x] = v[j];
    }
    const float o = __shfl_xor_sync(0xffffffffu, m[x], 1);
    if (second ? fabsf(o) >= fabsf(m[x]) : fabsf(o) > fabsf(m[x])) m[x] = o;
  }
  const float d = __fmul_rn(fabsf(m[1]) > fabsf(m[0]) ? m[1] : m[0], -0.125f);
  const float id = d != 0.f ? __frcp_rn(d) : 0.f;
  uint32_t q[16];  // a code in the low byte
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float t = __fadd_rn(__fmul_rn(v[j], id), 8.5f);
    q[j] = __float_as_uint(__fadd_rz(fminf(fmaxf(t, 0.f), 15.f), 8388608.f));
  }
  auto bytes = [&](int j) {
    return __byte_perm(__byte_perm(q[j], q[j + 1], 0x0040), __byte_perm(q[j + 2], q[j + 3], 0x0040),
                       0x5410);
  };
  scale = __float2half_rn(d);
  return make_uint2(bytes(0) | (bytes(8) << 4), bytes(4) | (bytes(12) << 4));
}

// A head's row is moved in pieces of W elements, nv to a row (one where D is 64 or 128, else W =
// 32).  A CTA moves `groups` x kTok rows from blockIdx.x * groups * kTok on, of `span` of the
// Hkv * nv pieces of a row.  A thread keeps its row of a group and its part of a piece, and passes
// over the groups and pieces.  The part is 16 bytes of a dense row, or, with a q4_0 pool, the 16
// elements of 8 bytes of nibbles.
struct Split {
  int Hkv, groups, span;
  DivBy nv;
};

template <bool APPEND, bool Q4, int W, bool BF16>
__device__ __forceinline__ void move_rows(const PagedBatch& b, const PagedSide& s,
                                          const Split& sp) {
  __shared__ int64_t row_of[kTok * kGroups];
  constexpr int kParts = W / (Q4 ? 16 : 8);             // of a piece
  constexpr int kPieces = kThreads / (kTok * kParts);   // of a pass
  const int nv = W == 32 ? static_cast<int>(sp.nv.d) : 1;
  const int c = threadIdx.x % kParts, i = threadIdx.x / kParts % kTok;
  const int t0 = blockIdx.x * sp.groups * kTok;
  const int first = blockIdx.z * sp.span, end = min(sp.Hkv * nv, first + sp.span);
  const int passes = sp.groups * ((end - first + kPieces - 1) / kPieces);
  // (q4_0: elements 8 (c mod 2) .. of block c / 2, and those 16 further)
  uint16_t* const x0 = static_cast<uint16_t*>(s.x) + (t0 + i) * s.row_stride +
                       (Q4 ? (c >> 1) * 32 + (c & 1) * 8 : c * 8);
  int g = 0, at = first;  // of the next pass: its group, its first piece
  struct Place {
    uint16_t* x;
    int row, h, v;  // row within the CTA's (-1: none), head, piece of the head
  };
  auto next = [&]() -> Place {
    Place p;
    const int piece = at + threadIdx.x / (kTok * kParts);
    p.h = W == 32 ? sp.nv(piece) : piece;
    p.v = W == 32 ? piece - p.h * nv : 0;
    p.x = x0 + static_cast<int64_t>(g) * kTok * s.row_stride + p.h * s.head_stride + p.v * W;
    p.row = g < sp.groups && piece < end && t0 + g * kTok + i < b.rows ? g * kTok + i : -1;
    if ((at += kPieces) >= end) {
      at = first;
      ++g;
    }
    return p;
  };
  auto pool_piece = [&](const Place& p) -> int64_t {  // -1: no place
    const int64_t r = p.row < 0 ? -1 : row_of[p.row];
    return r < 0 ? r : (r + static_cast<int64_t>(p.h) * b.page_size) * nv + p.v;
  };
  Place p[kDeep];
  if constexpr (APPEND) {
    uint4 lo[kDeep], hi[Q4 ? kDeep : 1];
    auto load = [&]() {
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        p[u] = next();
        const uint4* src = reinterpret_cast<const uint4*>(p[u].x);
        lo[u] = p[u].row >= 0 ? __ldg(src) : make_uint4(0, 0, 0, 0);
        if constexpr (Q4) hi[u] = p[u].row >= 0 ? __ldg(src + 2) : make_uint4(0, 0, 0, 0);
      }
    };
    load();  // before the rows' places are known
    if (!locate_rows(b, sp.Hkv, t0, sp.groups * kTok, row_of)) return;
    for (int n = 0;;) {
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        if (n + u >= passes) break;
        const int64_t piece = pool_piece(p[u]);
        if constexpr (Q4) {
          __half sc;
          const uint2 nib = q4_quantize_half<BF16>(lo[u], hi[u], c & 1, sc);
          if (piece >= 0) {
            static_cast<uint2*>(s.pages)[piece * kParts + c] = nib;
            if ((c & 1) == 0) static_cast<__half*>(s.scale)[piece * (W / 32) + (c >> 1)] = sc;
          }
        } else {
          if (piece >= 0) static_cast<uint4*>(s.pages)[piece * kParts + c] = lo[u];
        }
      }
      n += kDeep;
      if (n >= passes) break;
      load();
    }
  } else {
    if (!locate_rows(b, sp.Hkv, t0, sp.groups * kTok, row_of)) return;
    for (int n = 0; n < passes; n += kDeep) {
      int64_t piece[kDeep];
      if constexpr (Q4) {
        uint2 w[kDeep];
        __half sc[kDeep];
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
          p[u] = next();
          piece[u] = pool_piece(p[u]);
          if (piece[u] >= 0) {
            w[u] = __ldg(static_cast<const uint2*>(s.pages) + piece[u] * kParts + c);
            sc[u] = __ldg(static_cast<const __half*>(s.scale) + piece[u] * (W / 32) + (c >> 1));
          }
        }
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
          if (piece[u] < 0) continue;
          uint4* dst = reinterpret_cast<uint4*>(p[u].x);
#pragma unroll
          for (int hi = 0; hi < 2; ++hi) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              o[j] = q4_pair<BF16>(((j & 2) ? w[u].y : w[u].x) >> (16 * (j & 1) + 4 * hi), sc[u]);
            dst[2 * hi] = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      } else {
        uint4 w[kDeep];
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
          p[u] = next();
          piece[u] = pool_piece(p[u]);
          if (piece[u] >= 0) w[u] = __ldg(static_cast<const uint4*>(s.pages) + piece[u] * kParts + c);
        }
#pragma unroll
        for (int u = 0; u < kDeep; ++u)
          if (piece[u] >= 0) *reinterpret_cast<uint4*>(p[u].x) = w[u];
      }
    }
  }
}

template <bool APPEND, int W, bool BF16>
__global__ void __launch_bounds__(kThreads)
    rows_kernel(PagedBatch b, PagedSide k, PagedSide v, Split sp) {
  const PagedSide& s = blockIdx.y ? v : k;
  if (s.q4)
    move_rows<APPEND, true, W, BF16>(b, s, sp);
  else
    move_rows<APPEND, false, W, BF16>(b, s, sp);
}

template <bool APPEND, int W>
void rows_launch(dim3 grid, cudaStream_t stream, bool bf16, const PagedBatch& b,
                 const PagedSide& k, const PagedSide& v, const Split& sp) {
  auto kern = bf16 ? rows_kernel<APPEND, W, true> : rows_kernel<APPEND, W, false>;
  kern<<<grid, kThreads, 0, stream>>>(b, k, v, sp);
}

}  // namespace

cudaError_t paged_rows_launch(bool append, const PagedBatch& b, const PagedSide& k,
                              const PagedSide& v, int Hkv, int D, bool bf16, int num_sms,
                              cudaStream_t stream) {
  if (b.rows == 0) return cudaSuccess;
  const int tiles = (b.rows + kTok - 1) / kTok, sides = v.x ? 2 : 1;
  const int W = D == 64 || D == 128 ? D : 32;
  const int pieces = Hkv * (D / W);  // of a row
  const int64_t items = static_cast<int64_t>(tiles) * pieces * sides;
  // Work per CTA: kMost pieces of 16 rows, fewer where the SMs would not all have a CTA.  (4 x 16384
  // rows, f16 and q4_0: 82 and 72 us with 4 pieces, 81 and 55 with 8, 83 and 55 with 16, 88 and 62
  // with 64; 64 rows appended and read back: 5.7 us, 11.2 with all 8 heads in one CTA.)
  constexpr int kMost = 8;
  const int per = static_cast<int>(std::max<int64_t>(
      pieces / 65535 + 1, std::min<int64_t>(kMost, items / num_sms)));
  const int parts = (pieces + std::min(pieces, per) - 1) / std::min(pieces, per);
  const Split sp = {Hkv, parts > 1 ? 1 : std::max(1, std::min(kGroups, per / pieces)),
                    (pieces + parts - 1) / parts, DivBy(D / W)};
  const dim3 grid((tiles + sp.groups - 1) / sp.groups, sides, (pieces + sp.span - 1) / sp.span);
  auto go = append ? (W == 128  ? rows_launch<true, 128>
                      : W == 64 ? rows_launch<true, 64>
                                : rows_launch<true, 32>)
                   : (W == 128  ? rows_launch<false, 128>
                      : W == 64 ? rows_launch<false, 64>
                                : rows_launch<false, 32>);
  go(grid, stream, bf16, b, k, v, sp);
  return cudaGetLastError();
}

uint32_t paged_take_error() {
  uint32_t v = 0;
  if (cudaMemcpyFromSymbol(&v, g_paged_error, sizeof(v)) != cudaSuccess) return 0xffffffffu;
  const uint32_t z = 0;
  cudaMemcpyToSymbol(g_paged_error, &z, sizeof(z));
  return v;
}

}  // namespace fa
