// Writing new tokens into page pools (fa_append_paged) and reading tokens back out of them
// (fa_read_paged), each pool dense or q4_0.  This is the paged form of the step that keeps the cache
// quantized ("FlashAttention on gfx90a: Why It's Broken and How to Fix It", Impact of the V Dequant
// Patch, -ctk q4_0 -ctv q4_0).
//
// Both are bound by HBM bandwidth when there are many rows and by the latency of their dependent
// loads (batch description, then page table, then data) when there are few.  One CTA takes 16
// packed rows of K or of V, all heads: its threads first find the 16 rows' places in the pool
// together (the data loads that do not depend on them are already under way when appending), then
// walk the rows head by head, so that the 16 rows of a head, neighbours in a page, are stored as
// one run: 16 x 64 bytes of nibbles and 16 x 8 bytes of scales at D = 128.
#include <algorithm>

#include "fa_internal.h"
#include "fa_paged.cuh"
#include "fa_ptx.cuh"
#include "fa_quant.cuh"

namespace fa {

__device__ uint32_t g_paged_error;

namespace {

constexpr int kTok = 16;        // packed rows per CTA
constexpr int kThreads = 256;
constexpr int kSmemSeqs = 1024; // batches up to this size keep starts and lens in shared memory

// Places of rows t0 .. t0 + kTok - 1 in the pool: row_of[i] = the pool row (of D elements) of kv
// head 0, head h's being h * page_size further, or -1 for a row that belongs to no sequence or
// whose place is out of range (recorded).  False, with nothing to do, when starts is not a rising
// run within the tensors (recorded).  Ends with a barrier.
__device__ __forceinline__ bool locate_rows(const PagedBatch& b, int Hkv, int t0,
                                            int64_t (&row_of)[kTok]) {
  __shared__ int32_t s_starts[kSmemSeqs + 1];
  __shared__ int32_t s_lens[kSmemSeqs];
  const int tid = threadIdx.x;
  const bool small = b.B <= kSmemSeqs;
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
  if (tid < kTok) {
    const int t = t0 + tid;
    int64_t row = -1;
    if (t >= starts[0] && t < starts[b.B]) {
      int lo = 0, hi = b.B;  // the last sequence that starts at or before row t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= t) lo = mid; else hi = mid;
      }
      const int len = lens[lo];
      const int64_t cap = static_cast<int64_t>(b.page_size) * b.pages_per_seq;
      const int pos = len - (starts[lo + 1] - t);
      if (pos >= 0 && len <= cap) {
        const int lp = pos / b.page_size;
        const int page = __ldg(b.table + static_cast<int64_t>(lo) * b.pages_per_seq + lp);
        if (page >= 0 && page < b.num_pages)
          row = static_cast<int64_t>(page) * Hkv * b.page_size + (pos - lp * b.page_size);
      }
      if (row < 0) atomicCAS(&g_paged_error, kErrNone, kErrBadIndex);
    }
    row_of[tid] = row;
  }
  __syncthreads();
  return true;
}

// item idx of a tile: chunk fastest, then row, then head, so that a warp's items are neighbours
// in the page
struct Item {
  int h, i, c;
};
__device__ __forceinline__ Item item_of(int idx, int chunks) {
  Item it;
  const int r = idx / chunks;
  it.c = idx - r * chunks;
  it.i = r % kTok;
  it.h = r / kTok;
  return it;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) append_kernel(PagedBatch b, PagedSide k, PagedSide v,
                                                          int Hkv, int D) {
  __shared__ int64_t row_of[kTok];
  const PagedSide s = blockIdx.y ? v : k;
  const int t0 = blockIdx.x * kTok;
  const uint16_t* x = static_cast<const uint16_t*>(s.x);
  if (s.q4) {
    // one thread per 32-element block
    const int nb = D / 32, total = Hkv * kTok * nb;
    auto load = [&](int idx, uint4(&w)[4]) {
      const Item it = item_of(idx, nb);
      if (idx < total && t0 + it.i < b.rows) {
        const uint4* src = reinterpret_cast<const uint4*>(x + (t0 + it.i) * s.row_stride +
                                                          it.h * s.head_stride + it.c * 32);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __ldg(src + j);
      }
    };
    uint4 w[4] = {};
    load(threadIdx.x, w);  // before the rows' places are known
    if (!locate_rows(b, Hkv, t0, row_of)) return;
    for (int idx = threadIdx.x; idx < total; idx += kThreads) {
      uint4 next[4] = {};
      load(idx + kThreads, next);
      const Item it = item_of(idx, nb);
      if (row_of[it.i] >= 0) {
        uint4 nib;
        __half sc;
        q4_quantize_block<BF16>(w, nib, sc);
        const int64_t row = row_of[it.i] + static_cast<int64_t>(it.h) * b.page_size;
        static_cast<uint4*>(s.pages)[row * nb + it.c] = nib;
        static_cast<__half*>(s.scale)[row * nb + it.c] = sc;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = next[j];
    }
  } else {
    const int nc = D / 8, total = Hkv * kTok * nc;  // 16-byte chunks
    if (!locate_rows(b, Hkv, t0, row_of)) return;
    for (int idx = threadIdx.x; idx < total; idx += kThreads) {
      const Item it = item_of(idx, nc);
      if (row_of[it.i] < 0) continue;
      const int64_t row = row_of[it.i] + static_cast<int64_t>(it.h) * b.page_size;
      static_cast<uint4*>(s.pages)[row * nc + it.c] = __ldg(reinterpret_cast<const uint4*>(
          x + (t0 + it.i) * s.row_stride + it.h * s.head_stride + it.c * 8));
    }
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) read_kernel(PagedBatch b, PagedSide k, PagedSide v,
                                                        int Hkv, int D) {
  __shared__ int64_t row_of[kTok];
  const PagedSide s = blockIdx.y ? v : k;
  const int t0 = blockIdx.x * kTok;
  uint16_t* x = static_cast<uint16_t*>(s.x);
  if (!locate_rows(b, Hkv, t0, row_of)) return;
  const int nc = D / 8, total = Hkv * kTok * nc;  // 16-byte chunks of the output
  for (int idx = threadIdx.x; idx < total; idx += kThreads) {
    const Item it = item_of(idx, nc);
    if (row_of[it.i] < 0) continue;
    const int64_t row = row_of[it.i] + static_cast<int64_t>(it.h) * b.page_size;
    uint4 out;
    if (s.q4) {
      // chunk c of a block: elements 8c .. 8c + 7, the low (c < 2) or high nibbles of 8 bytes
      const int blk = it.c >> 2, c = it.c & 3;
      const uint2 n = __ldg(static_cast<const uint2*>(s.pages) + (row * (D / 32) + blk) * 2 +
                            (c & 1));
      const float d = __half2float(static_cast<const __half*>(s.scale)[row * (D / 32) + blk]);
      const uint32_t w[2] = {(c & 2) ? n.x >> 4 : n.x, (c & 2) ? n.y >> 4 : n.y};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t u = w[j >> 1] >> (16 * (j & 1));
        // (code - 8) * d is exact in f32 and rounded once here
        o[j] = pack2<BF16>((static_cast<int>(u & 15u) - 8) * d,
                           (static_cast<int>((u >> 8) & 15u) - 8) * d);
      }
      out = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      out = __ldg(static_cast<const uint4*>(s.pages) + row * nc + it.c);
    }
    *reinterpret_cast<uint4*>(x + (t0 + it.i) * s.row_stride + it.h * s.head_stride + it.c * 8) =
        out;
  }
}

}  // namespace

cudaError_t paged_rows_launch(bool append, const PagedBatch& b, const PagedSide& k,
                              const PagedSide& v, int Hkv, int D, bool bf16,
                              cudaStream_t stream) {
  if (b.rows == 0) return cudaSuccess;
  const dim3 grid((b.rows + kTok - 1) / kTok, v.x ? 2u : 1u);
  auto kern = append ? (bf16 ? append_kernel<true> : append_kernel<false>)
                     : (bf16 ? read_kernel<true> : read_kernel<false>);
  kern<<<grid, kThreads, 0, stream>>>(b, k, v, Hkv, D);
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
