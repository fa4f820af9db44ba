// kap_tma.h - tensor maps of the KV pool for tiled TMA loads (internal to the library).
#pragma once

#include <cuda.h>

namespace kap {

// 2-D view [num_pages * Hkv * 16 rows][128 columns] of a bf16 pool; boxes of 64 columns x 16 rows, 128-byte swizzle.
bool make_pool_map(CUtensorMap *map, const void *base, int num_pages, int hkv);
// The pool as [groups of 8 rows][column halves of 64][8 rows][64 columns]: a box is one page of a head, so one request
// brings it, with its 8 x 64 blocks one after the other (1 KB each, 128-byte swizzle).
bool make_page_map(CUtensorMap *map, const void *base, int num_pages, int hkv, int d);

}  // namespace kap
