// The tokens of a step and the keys that they see, for the kernels over a paged cache.
#pragma once
#include "common.cuh"

namespace ds4a {

struct PagedItem {
  uint32_t first, cnt, pos0;   // packed index of a sequence's first token, tokens, its position
  uint32_t lo, hi;             // positions lo .. hi - 1 are seen by some of them
};

__device__ __forceinline__ PagedItem paged_item(const PagedArgs &a, uint32_t b) {
  PagedItem it;
  it.first = a.cu_len ? __ldg(a.cu_len + b) : b * a.max_new;
  const uint32_t n = a.cu_len ? __ldg(a.cu_len + b + 1) - it.first : a.max_new;
  it.cnt = n < 0x80000000u ? min(n, a.max_new) : 0u;
  it.pos0 = __ldg(a.seq_pos + b);
  const uint64_t end = (uint64_t)it.pos0 + it.cnt, room = (uint64_t)a.max_blocks * 256u;
  it.hi = (uint32_t)(end < room ? end : room);
  it.lo = a.window && it.pos0 + 1 > a.window ? it.pos0 + 1 - a.window : 0u;
  if (it.lo > it.hi) it.lo = it.hi;
  return it;
}

}  // namespace ds4a
