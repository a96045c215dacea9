// PagedWalk (csrc/fa_paged.cuh) on the host: a warp's 32 lanes are run in turn, each up to its next
// exchange with the others, so that the header's own code runs as it stands.
//
// Input: B Hkv causal unit_tok num_pages page_size pages_per_seq rows grid, then starts[B + 1], lens[B].
// Output: the error word, then a line a segment: cta b tok g j0 j1 c_first c_last slot_first.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <ucontext.h>
#include <vector>

#define __host__
#define __device__
#define __forceinline__ inline
using std::max;
using std::min;

namespace {
constexpr int kLanes = 32;
struct Lane {
  ucontext_t ctx;
  std::vector<char> stack;
  bool done;
} lanes[kLanes];
ucontext_t scheduler;
int current;            // the lane that runs
int exchanged[kLanes];  // how many exchanges each has come to
uint32_t slots[2][kLanes];

// the lanes' values, once all have come to this exchange (read before the next one's are written)
const uint32_t* exchange(uint32_t v) {
  const int me = current, turn = exchanged[me]++ & 1;
  slots[turn][me] = v;
  swapcontext(&lanes[me].ctx, &scheduler);
  for (int i = 0; i < kLanes; ++i)  // (those before this one may be at the next already)
    if (exchanged[i] != exchanged[me] && (i > me || exchanged[i] != exchanged[me] + 1)) {
      std::fprintf(stderr, "lanes %d and %d apart\n", i, me);
      std::exit(3);
    }
  return slots[turn];
}
}  // namespace

struct Index {
  operator int() const { return current; }
};
struct {
  Index x;
} threadIdx;

template <class T>
T __ldg(const T* p) { return *p; }
uint32_t __umulhi(uint32_t a, uint32_t b) { return static_cast<uint64_t>(a) * b >> 32; }
uint32_t atomicCAS(uint32_t* p, uint32_t expect, uint32_t v) {
  const uint32_t old = *p;
  if (old == expect) *p = v;
  return old;
}
int __ffs(unsigned v) { return __builtin_ffs(static_cast<int>(v)); }
unsigned __ballot_sync(unsigned, bool p) {
  const uint32_t* v = exchange(p);
  unsigned r = 0;
  for (int i = 0; i < kLanes; ++i) r |= static_cast<unsigned>(v[i] != 0) << i;
  return r;
}
bool __any_sync(unsigned m, bool p) { return __ballot_sync(m, p) != 0; }
int __reduce_add_sync(unsigned, int x) {
  const uint32_t* v = exchange(static_cast<uint32_t>(x));
  int64_t r = 0;
  for (int i = 0; i < kLanes; ++i) r += static_cast<int>(v[i]);
  if (r < 0 || r > INT32_MAX) std::exit(4);
  return static_cast<int>(r);
}
int __shfl_sync(unsigned, int x, int from) { return static_cast<int>(exchange(static_cast<uint32_t>(x))[from]); }
int __shfl_up_sync(unsigned, int x, int by) {
  const int me = current;
  const uint32_t* v = exchange(static_cast<uint32_t>(x));
  return static_cast<int>(v[me >= by ? me - by : me]);
}

#include "fa_paged.cuh"

namespace {
fa::PagedPlan plan;
fa::PagedWalk walks[kLanes];
uint32_t error;
int cta, grid;

void lane_main() {
  walks[current] = fa::PagedWalk();
  walks[current].find(plan, cta, grid, &error, 2u);
  lanes[current].done = true;
}

int number() {
  int v;
  if (std::scanf("%d", &v) != 1) std::exit(5);
  return v;
}
}  // namespace

int main() {
  const int B = number(), Hkv = number(), causal = number(), unit_tok = number();
  const int pages = number(), page = number(), pps = number(), rows = number();
  grid = number();
  std::vector<int32_t> starts(B + 1), lens(B);
  for (int32_t& v : starts) v = number();
  for (int32_t& v : lens) v = number();
  plan.bt = fa::PagedBatch{nullptr, starts.data(), lens.data(), B, rows, pages, page, pps};
  plan.page = fa::DivBy(page);
  plan.Hkv = Hkv;
  plan.causal = causal;
  plan.unit_tok = unit_tok;
  std::vector<std::vector<int>> out;
  for (cta = 0; cta < grid; ++cta) {
    for (int i = 0; i < kLanes; ++i) {
      lanes[i].stack.resize(1 << 16);
      lanes[i].done = false;
      exchanged[i] = 0;
      getcontext(&lanes[i].ctx);
      lanes[i].ctx.uc_stack.ss_sp = lanes[i].stack.data();
      lanes[i].ctx.uc_stack.ss_size = lanes[i].stack.size();
      lanes[i].ctx.uc_link = &scheduler;
      makecontext(&lanes[i].ctx, lane_main, 0);
    }
    while (!lanes[0].done)
      for (current = 0; current < kLanes; ++current) swapcontext(&scheduler, &lanes[current].ctx);
    current = 0;
    fa::PagedWalk w = walks[0];
    for (int i = 1; i < kLanes; ++i) {
      const fa::PagedWalk& x = walks[i];
      if (x.t != w.t || x.t_end != w.t_end || x.u0 != w.u0 || x.b != w.b || x.tok != w.tok || x.g != w.g ||
          x.nb != w.nb || x.whole != w.whole || x.s.start != w.s.start || x.s.nq != w.s.nq ||
          x.s.len != w.s.len) {
        std::fprintf(stderr, "cta %d: lane %d differs\n", cta, i);
        return 6;
      }
    }
    while (w.t < w.t_end) {
      int first, last, slot;
      w.pieces(plan, cta, first, last, slot);
      out.push_back({cta, w.b, w.tok, w.g, w.j0(plan), w.j1(plan), first, last, slot});
      w.next(plan);
    }
  }
  std::printf("%u\n", error);
  for (const auto& r : out) {
    for (int v : r) std::printf("%d ", v);
    std::printf("\n");
  }
}
