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

// From the request's entries of the offsets and lengths.  Tokens past the last row have no row, and the positions from
// theirs on are not looked at.
__device__ __forceinline__ StepRequest step_request(const KvStep& s, int r, int from, int to, int len) {
  StepRequest q;
  const int b0 = min(max(from, 0), s.T), end = max(to, b0), b1 = min(end, s.T);
  q.r = r;
  q.row0 = b0;
  q.n = b1 - b0;
  q.len = (int)max(min((long long)len, 0x7FFFF000ll) - (end - b1), 0ll);
  return q;
}

// Item `index` of the step, the requests in order with count(request) items each: its request and place there.  One
// whole wave; false past the last.  A lane per request, 256 a round whose loads are in flight together (4096 lengths
// wait 16 times).
template <typename Count>
__device__ __forceinline__ bool step_find(const KvStep& s, int index, Count&& count, StepRequest* out, int* within) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int r0 = 0; r0 < s.R; r0 += 256) {
    int from[4], to[4], len[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i > 0 && r0 + 64 * i >= s.R) break;
      const int r = min(r0 + 64 * i + lane, s.R - 1);
      from[i] = s.offsets[r];
      to[i] = s.offsets[r + 1];
      len[i] = s.lens[r];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 64 * i + lane;
      if (r - lane >= s.R) break;
      const int own = r < s.R ? count(step_request(s, r, from[i], to[i], len[i])) : 0;
      const int scan = wave_inclusive_scan(own), excl = base + scan - own;
      const uint64_t hit = __ballot(excl <= index && index < excl + own);
      if (hit) {
        const int src = __ffsll((unsigned long long)hit) - 1;
        *within = index - __builtin_amdgcn_readlane(excl, src);
        *out = step_request(s, r0 + 64 * i + src, __builtin_amdgcn_readlane(from[i], src),
                            __builtin_amdgcn_readlane(to[i], src), __builtin_amdgcn_readlane(len[i], src));
        return true;
      }
      base += __builtin_amdgcn_readlane(scan, 63);
    }
  }
  return false;
}

}  // namespace
}  // namespace moe
