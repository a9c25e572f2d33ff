// paged_dev.h -- the paged cache's device arrays and its host handle, shared by
// libbeamstep.so (which owns them) and libbeamattn.so (whose 8-bit reorder
// follows the step's copy list).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

struct bs_state;

namespace {

struct PagedDev {
  int* table;     // [B*W][mb] global block ids, -1 = none
  int* refc;      // [B*bpi] live-row references of each block
  int* freel;     // [B][bpi] stack of free global block ids
  int* nfree;     // [B]
  int* overflow;  // [1]
  int* cpy;       // [B*W][3] copy list of the step: source block, destination block, positions
  int* ncpy;      // [2] entries of the list, by step parity
};

}  // namespace

struct bs_kv_paged {
  bs_state* h;          // null once the handle is destroyed (the cache is orphaned)
  bs_kv_paged* next;    // the handle's next cache
  hipStream_t stream;   // the handle's stream
  int device;           // the handle's device
  int rows;             // B*W: the capacity of the step's copy list
  int blocks;           // B*blocks_per_item: the blocks every pool holds at least
  int bs, bpi, mb;
  int last_t;   // the step last reordered (0: none since the reset)
  int table_t;  // the step whose table update has run (0: none since the reset)
  void* block;
  PagedDev pg;
};
