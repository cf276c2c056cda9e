// layer.cuh — device helpers of the decode-layer kernels: the cache's element types and the
// translation of a sequence's position to its place in the paged cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace spax {

// Element offset of (position, head 0) in the pools, or -1 for a page outside the cache. row is a
// row of the page table; the caller keeps pos within [0, max_pages * page_size).
__device__ __forceinline__ long long cache_row(const spax_kv_cache& c, const int32_t* row,
                                               int pos) {
  const int at = pos / c.page_size;
  const int page = row[at];
  if (page < 0 || page >= c.n_pages) return -1;
  return page * c.page_stride + (long long)(pos - at * c.page_size) * c.token_stride;
}

// One value in the bf16 cache's type.
__device__ __forceinline__ uint16_t to_bf16(float v) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

}  // namespace spax
