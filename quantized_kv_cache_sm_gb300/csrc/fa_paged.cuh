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

}  // namespace fa
