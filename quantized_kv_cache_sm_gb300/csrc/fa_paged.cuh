// A ragged batch over page pools, as the paged operators see it.
//
// Sequence b owns packed rows starts[b] .. starts[b + 1] - 1; they are its last tokens, at positions
// lens[b] - n_b .. lens[b] - 1 (n_b rows).  Position p lives in page table[b][p / page_size], slot
// p % page_size, of a pool [num_pages][Hkv][page_size][D].  All three arrays are device memory: the
// same captured launch serves other batches by rewriting them.
#pragma once

#include <stdint.h>

namespace fa {

struct PagedBatch {
  const int32_t* table;   // [B][pages_per_seq]
  const int32_t* starts;  // [B + 1]
  const int32_t* lens;    // [B]
  int B, rows;            // rows: packed rows the tensors hold; rows from starts[B] on are padding
  int num_pages, page_size, pages_per_seq;
};

// starts must rise from a non-negative first entry and end within the tensors: entry i against
// the next one
__host__ __device__ __forceinline__ bool bad_start(int v, int next, int rows) {
  return v < 0 || next < v || next > rows;
}

// a length of a sequence that the block table cannot hold
__host__ __device__ __forceinline__ bool bad_length(int len, int64_t cap) {
  return len < 0 || len > cap;
}
// position of the row that is `back` rows before its sequence's end (1: the last row); negative
// where it has none: a bad length, or more rows than tokens.  (The length is looked at first: near
// -2^31 the difference would overflow to a large position.)
__host__ __device__ __forceinline__ int row_position(int len, int64_t cap, int back) {
  return bad_length(len, cap) ? -1 : len - back;
}

// x / d for 0 <= x < 2^31 by a multiplication and a shift: with s = ceil(log2 d) and m =
// floor(2^32 (2^s - d) / d) + 1, x / d = (mulhi(m, x) + x) >> s (Granlund and Montgomery, "Division
// by invariant integers using multiplication", PLDI 1994)
struct DivBy {
  uint32_t d, m, s;
  DivBy() = default;
  explicit DivBy(uint32_t divisor) : d(divisor), m(0), s(0) {
    while ((1ull << s) < d) ++s;
    m = static_cast<uint32_t>((((1ull << s) - d) << 32) / d + 1);
  }
  __device__ __forceinline__ int operator()(int x) const {
    return static_cast<int>((__umulhi(m, static_cast<uint32_t>(x)) + static_cast<uint32_t>(x)) >>
                            s);
  }
};

// ------------------------------------------------------------------------------------------
// The ragged prefill's schedule.  A work unit is `unit_tok` consecutive new tokens of a sequence
// for one kv head; its steps are the 128-key blocks that its last token sees, at least one.  In
// the schedule a unit counts `over` steps more, at its beginning, for what it costs whatever its
// length (loading its queries, storing its rows).  The counts of all units -- ordered by sequence,
// then tokens, then kv head -- are concatenated and cut evenly over the CTAs.  Lengths live on the
// device, so every CTA finds its own run.  Counts fit 32 bits (the host checks).
// ------------------------------------------------------------------------------------------
struct PagedSeq {
  int start, nq, len;  // first packed row, new tokens, keys
};

// W counts cut over n CTAs: the first W mod n of them take one more
struct PagedCut {
  int q = 1, rem = 0;
  __device__ __forceinline__ int start(int c) const { return c * q + min(c, rem); }
  // the CTA that holds count t
  __device__ __forceinline__ int of(int t) const {
    const int wide = rem * (q + 1);
    return t < wide ? t / (q + 1) : rem + (t - wide) / q;
  }
};

struct PagedPlan {
  PagedBatch bt;
  DivBy page;         // by page_size
  int Hkv, causal;
  int unit_tok;
  // A unit's start and end (first scores, last products, epilogue) count as two of its blocks.  (1,
  // 2 or 4: the same within 1 % from one token a sequence to the 2048-token chunk; 0 leaves runs of
  // many short units late.)
  static constexpr int kOver = 2;
  // A cut costs its pieces' round trip through memory and their merge: units of up to so many blocks
  // stay whole (a run's end inside one moves to the nearer end of it), longer ones are cut anywhere.
  // Measured, D = 64, f16 K and q4_0 V, prompts of up to 1000 tokens: 19.2 us with 8 or 16, 20.8
  // with 0 or 4; 16 sequences of mixed lengths, bf16 at D = 128: 52.5 us with 0 or 8, 67.0 with 16
  // (these before later steps took the calls themselves to other times).
  // A limit of 32 for units of one 32-row quarter of a tile alone took 16 sequences of a few q4_0
  // draft tokens from 48.0 to 45.8 us, and the mixed batch from 52.5 to 58.5.
  static constexpr int kWhole = 8;

  __device__ __forceinline__ int cap() const { return bt.page_size * bt.pages_per_seq; }
  __device__ __forceinline__ PagedSeq seq(int b) const {
    PagedSeq s = {0, 0, 0};
    if (b < bt.B) {
      s.start = __ldg(bt.starts + b);
      s.nq = __ldg(bt.starts + b + 1) - s.start;
      s.len = max(0, min(__ldg(bt.lens + b), cap()));
    }
    return s;
  }
  // blocks that the tokens before tok_end see, at least one
  __device__ __forceinline__ int blocks(const PagedSeq& s, int tok_end) const {
    const int last = causal ? s.len - s.nq + min(tok_end, s.nq) : s.len;
    return max(1, (max(0, min(s.len, last)) + 127) >> 7);
  }
  // counts of a sequence's units for one kv head
  __device__ __forceinline__ int counts(const PagedSeq& s) const {
    int n = 0;
    for (int t = 0; t < s.nq; t += unit_tok) n += kOver + blocks(s, t + unit_tok);
    return n;
  }
};

// One CTA's walk through its run, by one warp (every member is the same in all lanes)
struct PagedWalk {
  PagedCut cut;
  int t = 0, t_end = 0;       // the next count and the end of the run
  int u0 = 0;                 // the unit's first count (block 0 is count u0 + over)
  int b = 0, tok = 0, g = 0;  // the unit: sequence, first token, kv head
  int nb = 1;                 // its blocks
  bool whole = false;         // the unit is not cut
  PagedSeq s = {0, 0, 0};

  // CTA `cta`'s run out of `grid` CTAs.  Bad starts or lengths are recorded in *err by CTA 0; bad
  // starts leave nothing to anybody.
  __device__ __forceinline__ void find(const PagedPlan& p, int cta, int grid, uint32_t* err,
                                       uint32_t bad_index) {
    const int lane = threadIdx.x & 31;
    int W = 0, own = 0;  // own: the counts of sequence `lane`
    bool bad = false;
    for (int b0 = 0; b0 < p.bt.B; b0 += 32) {
      const int i = b0 + lane;
      if (i < p.bt.B) {
        const int v = __ldg(p.bt.starts + i), next = __ldg(p.bt.starts + i + 1);
        const int len = __ldg(p.bt.lens + i);
        if (bad_start(v, next, p.bt.rows)) {
          bad = true;
        } else {
          if (cta == 0 && (len < 0 || len > p.cap())) atomicCAS(err, 0u, bad_index);
          const int n = p.counts(p.seq(i)) * p.Hkv;
          if (b0 == 0) own = n;
          W += n;
        }
      }
    }
    if (__any_sync(0xffffffffu, bad)) {
      if (cta == 0 && lane == 0) atomicCAS(err, 0u, bad_index);
      return;
    }
    W = __reduce_add_sync(0xffffffffu, W);
    const int n = min(grid, W);
    if (cta >= n) return;
    cut.q = W / n;
    cut.rem = W - cut.q * n;
    t = cut.start(cta);
    t_end = cut.start(cta + 1);
    for (int b0 = 0; b0 < p.bt.B; b0 += 32) {
      if (b0 > 0) own = p.counts(p.seq(b0 + lane)) * p.Hkv;
      int end = own;  // inclusive scan over the lanes
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, end, off);
        if (lane >= off) end += x;
      }
      const unsigned past = __ballot_sync(0xffffffffu, u0 + end > t);
      if (past) {
        const int who = __ffs(past) - 1;
        u0 += __shfl_sync(0xffffffffu, end - own, who);
        b = b0 + who;
        break;
      }
      u0 += __shfl_sync(0xffffffffu, end, 31);
    }
    s = p.seq(b);
    nb = p.blocks(s, p.unit_tok);
    while (tok < s.nq && t >= u0 + (p.kOver + nb) * p.Hkv) {
      u0 += (p.kOver + nb) * p.Hkv;
      tok += p.unit_tok;
      nb = p.blocks(s, tok + p.unit_tok);
    }
    g = (t - u0) / (p.kOver + nb);
    u0 += g * (p.kOver + nb);
    settle(p);
    if (whole && t > u0) {
      if (2 * (t - u0) >= p.kOver + nb) {
        next(p);
        return;
      }
      t = u0;
    }
    stop_before(p);
  }
  __device__ __forceinline__ void settle(const PagedPlan& p) {
    whole = nb <= p.kWhole;
  }
  // ends the run at a unit that it has no blocks of: it ends before block 0, or in the first half of
  // a unit that is not cut
  __device__ __forceinline__ void stop_before(const PagedPlan& p) {
    if (whole ? 2 * (t_end - u0) < p.kOver + nb : t_end <= u0 + p.kOver) t = t_end;
  }

  // the blocks [j0, j1) of the unit that belong to the run
  __device__ __forceinline__ int j0(const PagedPlan& p) const { return max(0, t - u0 - p.kOver); }
  __device__ __forceinline__ int j1(const PagedPlan& p) const {
    return whole ? nb : min(nb, t_end - u0 - p.kOver);
  }
  // past those; the next unit if the run has blocks of it
  __device__ __forceinline__ void next(const PagedPlan& p) {
    u0 += p.kOver + nb;
    t = u0;
    if (t >= t_end) return;
    if (++g == p.Hkv) {
      g = 0;
      tok += p.unit_tok;
      while (tok >= s.nq && b + 1 < p.bt.B) {
        s = p.seq(++b);
        tok = 0;
      }
      nb = p.blocks(s, tok + p.unit_tok);
      settle(p);
    }
    stop_before(p);
  }
  // the CTAs of the unit's first and last block, and the first one's partial slot: 1 where it
  // reaches the unit after others, 0 where its run begins in the unit (all other pieces' slot)
  __device__ __forceinline__ void pieces(const PagedPlan& p, int cta, int& c_first, int& c_last,
                                         int& slot_first) const {
    c_first = t > u0 + p.kOver ? cut.of(u0 + p.kOver) : cta;
    c_last = !whole && t_end < u0 + p.kOver + nb ? cut.of(u0 + p.kOver + nb - 1) : cta;
    slot_first = cut.start(c_first) < u0 ? 1 : 0;
  }
  // the page that holds keys [key, ...) of the sequence, -1 where there are none (not checked: the
  // value is not waited for here)
  __device__ __forceinline__ int look_up(const PagedPlan& p, int key) const {
    if (key >= s.len) return -1;
    return __ldg(p.bt.table + static_cast<int64_t>(b) * p.bt.pages_per_seq + p.page(key));
  }
  // a key's row in its page
  static __device__ __forceinline__ int page_row(const PagedPlan& p, int key) {
    return key - p.page(key) * p.bt.page_size;
  }
  // the tensor map's third coordinate (page, kv head) of a looked-up page; -1, where TMA fills with
  // zeros without reading memory, for none and for one outside the pool (recorded)
  __device__ __forceinline__ int block_of(const PagedPlan& p, int key, int page, uint32_t* err,
                                          uint32_t bad_index) const {
    if (key >= s.len) return -1;
    if (page < 0 || page >= p.bt.num_pages) {
      atomicCAS(err, 0u, bad_index);
      return -1;
    }
    return page * p.Hkv + g;
  }
};

}  // namespace fa
