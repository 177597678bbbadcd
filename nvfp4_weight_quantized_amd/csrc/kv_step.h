// A step's requests on the device: which request, and which part of it, a workgroup belongs to.
#pragma once

#include "device_util.h"

namespace moe {
namespace {

struct StepRequest {
  int r;       // request
  int row0;    // first token row
  int n;       // token rows
  int len;     // positions held once the rows are in; the rows are the last n
};

// Tokens past the last row have no row, and the positions from theirs on are not looked at.
__device__ __forceinline__ StepRequest step_request(const KvStep& s, int r) {
  StepRequest q;
  const int b0 = min(max(s.offsets[r], 0), s.T), end = max(s.offsets[r + 1], b0), b1 = min(end, s.T);
  q.r = r;
  q.row0 = b0;
  q.n = b1 - b0;
  q.len = (int)max(min((long long)s.lens[r], 0x7FFFF000ll) - (end - b1), 0ll);
  return q;
}

// Item `index` of the step, the requests in order with count(request) items each: its request and place there.  One
// whole wave; false past the last.  256 requests a round, so that the loads of 4096 lengths wait 16 times.
template <typename Count>
__device__ __forceinline__ bool step_find(const KvStep& s, int index, Count&& count, StepRequest* out, int* within) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int r0 = 0; r0 < s.R; r0 += 256) {
    int own[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 4 * lane + i;
      own[i] = 0;
      if (r < s.R) own[i] = count(step_request(s, r));
      sum += own[i];
    }
    const int scan = wave_inclusive_scan(sum), excl = base + scan - sum;
    const uint64_t hit = __ballot(excl <= index && index < excl + sum);
    if (hit) {
      const int src = __ffsll((unsigned long long)hit) - 1;
      int at = index - __builtin_amdgcn_readlane(excl, src), r = r0 + 4 * src;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int c = __builtin_amdgcn_readlane(own[i], src);
        if (r == r0 + 4 * src + i && at >= c) {
          at -= c;
          ++r;
        }
      }
      *out = step_request(s, r);
      *within = at;
      return true;
    }
    base += __builtin_amdgcn_readlane(scan, 63);
  }
  return false;
}

}  // namespace
}  // namespace moe
