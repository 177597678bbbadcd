// Work items of the attention over the paged cache, found on the device from the request lengths.
//
// A request r with n query tokens has n * G rows per kv head (row = token * G + head of the group), cut
// into tiles of BM rows, and the units (32 positions) [lo, hi) that its rows see.  The units are cut
// into splits of C units, C chosen so that the items of one kv head number about `target`:
//   C = max(min_chunk, ceil(sum_r tiles_r * units_r / target)).
// Items are ordered by request, tile, split; a tile of a request with one split writes its rows, the
// others leave partial sums in `slots` numbered the same way, which the combine launch adds in split
// order.  Every workgroup finds its own item with two passes over the lengths (no host knowledge, no
// list in memory, no atomics).
#pragma once

#include "common.h"

namespace moe {
namespace {

struct KvRequest {
  int n;        // query tokens
  int row0;     // first token row
  int len;      // positions held
  int tiles;    // row tiles (0: not of this launch)
  int lo, hi;   // units seen
};

struct KvItem {
  KvRequest q;
  int r;        // request
  int tile;     // row tile
  int split;    // index of the split (of splits)
  int splits;
  int chunk;    // units per split
  int slot;     // partial slot of this tile's split 0
};

struct KvSchedule {
  int bm;          // rows per tile
  int target;      // items aimed at, per kv head
  int min_chunk;   // units
  int min_rows, max_rows;   // requests of this launch: min_rows < rows <= max_rows
};

__device__ __forceinline__ KvRequest kv_request(const KvAttentionProblem& a, const KvSchedule& s, int r) {
  KvRequest q{};
  const int b0 = min(max(a.offsets[r], 0), a.T), b1 = min(max(a.offsets[r + 1], b0), a.T);
  q.row0 = b0;
  q.n = b1 - b0;
  q.len = max(a.lens[r], 0);
  const int rows = q.n * a.G;
  if (rows <= s.min_rows || rows > s.max_rows) return q;
  q.tiles = (rows + s.bm - 1) / s.bm;
  // first position that the first row sees
  const long long first = a.window > 0 ? (long long)q.len - q.n - a.window + 1 : 0;
  q.lo = (int)(max(first, 0ll) / kKvUnit);
  q.hi = max(q.lo, (int)(((long long)q.len + kKvUnit - 1) / kKvUnit));
  return q;
}

__device__ __forceinline__ long long wave_sum_i64(long long v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// Item `index` (BY_TILE: all splits of tile `index`); false past the last.  One whole wave.
template <bool BY_TILE>
__device__ __forceinline__ bool kv_find(const KvAttentionProblem& a, const KvSchedule& s, int index, KvItem* out) {
  const int lane = threadIdx.x & 63;
  long long work = 0;
  for (int r = lane; r < a.R; r += 64) {
    const KvRequest q = kv_request(a, s, r);
    work += (long long)q.tiles * (q.hi - q.lo);
  }
  work = wave_sum_i64(work);
  const int chunk = (int)max((long long)s.min_chunk, (work + s.target - 1) / s.target);
  int base = 0, slots = 0;
  for (int r0 = 0; r0 < a.R; r0 += 64) {
    const int r = r0 + lane;
    KvRequest q{};
    if (r < a.R) q = kv_request(a, s, r);
    const int splits = max(1, (int)(((long long)(q.hi - q.lo) + chunk - 1) / chunk));
    const int items = q.tiles * splits, count = BY_TILE ? q.tiles : items;
    const int part = splits > 1 ? items : 0;
    int ic = count, ip = part;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int x = __shfl_up(ic, off), y = __shfl_up(ip, off);
      if (lane >= off) {
        ic += x;
        ip += y;
      }
    }
    const int excl = base + ic - count;
    const uint64_t hit = __ballot(excl <= index && index < excl + count);
    if (hit) {
      const int src = __ffsll((unsigned long long)hit) - 1;
      const int within = index - __builtin_amdgcn_readlane(excl, src);
      out->r = r0 + src;
      out->q.n = __builtin_amdgcn_readlane(q.n, src);
      out->q.row0 = __builtin_amdgcn_readlane(q.row0, src);
      out->q.len = __builtin_amdgcn_readlane(q.len, src);
      out->q.tiles = __builtin_amdgcn_readlane(q.tiles, src);
      out->q.lo = __builtin_amdgcn_readlane(q.lo, src);
      out->q.hi = __builtin_amdgcn_readlane(q.hi, src);
      out->splits = __builtin_amdgcn_readlane(splits, src);
      out->chunk = chunk;
      out->tile = BY_TILE ? within : within / out->splits;
      out->split = BY_TILE ? 0 : within % out->splits;
      out->slot = slots + __builtin_amdgcn_readlane(ip - part, src) + out->tile * out->splits;
      return true;
    }
    base += __builtin_amdgcn_readlane(ic, 63);
    slots += __builtin_amdgcn_readlane(ip, 63);
  }
  return false;
}

}  // namespace
}  // namespace moe
