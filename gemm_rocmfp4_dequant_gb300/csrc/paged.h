// The paged ROCmFP4 K/V cache as the kernels see it.
#pragma once
#include <cstdint>

namespace rocmfp4 {

// K and V: [num_pages][Hkv][page_size] rows of D / 32 blocks.  Sequence b
// holds lens[b] tokens, token t of it in page table[b * ldt + t / page_size];
// rows cu[b] .. cu[b + 1] - 1 of a call are its last tokens.
struct PagedArgs {
  uint8_t* K;
  uint8_t* V;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu;
  int64_t ldt;
  int B, width;  // sequences; page numbers per sequence
  int num_pages, page_size, Hkv, D;
  uint32_t* err;
};

}  // namespace rocmfp4
