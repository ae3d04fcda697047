// kv_cache.h -- what the append to the paged 8-bit cache and the attention over it share: the sequences of
// a call, read and checked on the device.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace hq {

// New tokens and length of one sequence; n = 0 where there is nothing to do or the sequence is left out.
struct KvSeq {
  int first, n, len;
};

__device__ __forceinline__ KvSeq kv_sequence(const KvCall& c, int b) {
  KvSeq q{c.cu[b], 0, c.kv_lens[b]};
  const int end = c.cu[b + 1];
  if (q.first >= 0 && end > q.first && end <= c.T && end - q.first <= c.max_new && q.len >= 0 && q.len <= c.capacity) q.n = end - q.first;
  return q;
}

}  // namespace hq
