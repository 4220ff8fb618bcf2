// Device helpers shared by the attention kernels.
#pragma once

#include "attn.h"

namespace moe {

__device__ __forceinline__ void raise_bad_index(WsHeader* hdr) {
  atomicOr(&hdr->status, status_bit(MOE_ERR_BAD_INDEX));
}

// Raises MOE_ERR_BAD_INDEX unless the offsets cu[0..n] ascend from 0 to total; `threads` threads call it.
__device__ __forceinline__ void check_offsets(const int32_t* cu, int n, int total, WsHeader* hdr, int thread,
                                              int threads) {
  bool bad = false;
  for (int i = thread; i <= n; i += threads) {
    const int x = __ldg(cu + i), next = i < n ? __ldg(cu + i + 1) : total;
    bad |= x > next || (i == 0 && x != 0) || (i == n && x != total);
  }
  if (bad) raise_bad_index(hdr);
}

}  // namespace moe
