// Work of the attention over the paged cache, divided on the device from the request lengths: equal
// shares of a linear order (few rows per request, kv_locate), or items (many rows, kv_find).
//
// Items:
// A request r with n query tokens has n * G rows per kv head (row = token * G + head of the group), cut
// into tiles of BM rows, each of which sees at most `units` units (32 positions): all of them, or with a
// window those that its rows' windows reach.  A tile's units, counted from the first one it sees, are cut
// into equal splits of about C units, C chosen so that the items of one kv head number about `target`:
//   C = max(min_chunk, ceil(sum_r tiles_r * units_r / target)).
// What exceeds a multiple of C by less than a quarter of it makes no further split: a tile cut for a few
// units pays for the partial sums and their joining (2 prompts of 900, 16/8 heads, dimension 64:
// 43.4 against 28.7 us).
// Items are ordered by request, tile, split; a tile of a request with one split writes its rows, the
// others leave partial sums in `slots` numbered the same way, which the combine launch adds in split
// order.  Every workgroup finds its own item with two passes over the lengths (no host knowledge, no
// list in memory, no atomics).
#pragma once

#include <type_traits>

#include "device_util.h"
#include "kv_launch.h"

namespace moe {
namespace {

struct KvRequest {
  int n;        // query tokens
  int row0;     // first token row
  int len;      // positions held
  int tiles;    // row tiles (0: not of this launch)
  int units;    // units a tile sees at most
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

__device__ __forceinline__ KvRequest kv_request(const KvAttentionProblem& a, const KvSchedule& s, int r) {
  KvRequest q{};
  const int b0 = min(max(a.offsets[r], 0), a.T), end = max(a.offsets[r + 1], b0), b1 = min(end, a.T);
  q.row0 = b0;
  q.n = b1 - b0;
  // Tokens past the last row have no row, and the positions from theirs on are seen by none.  Below 2^31 by
  // more than any unit that a kernel looks at ahead.
  q.len = (int)max(min((long long)a.lens[r], 0x7FFFF000ll) - (end - b1), 0ll);
  const int rows = q.n * a.G;
  if (rows <= s.min_rows || rows > s.max_rows) return q;
  q.tiles = (rows + s.bm - 1) / s.bm;
  const int span = (s.bm - 1) / a.G + 1;      // the last row of a tile is at most so many positions behind the first
  long long units = ((long long)q.len + kKvUnit - 1) / kKvUnit;
  if (a.window > 0) units = min(units, ((long long)span + a.window + 2 * kKvUnit - 2) / kKvUnit);
  // Behind the table every unit is bad, and a row that sees one is NaN: a tile needs none past those that
  // hold the first position behind the table or the first one seen, whichever is later, of each of its rows.
  // So a length far beyond the table costs no more than one that fills it.
  units = min(units, (long long)a.width * (a.cache.page_size / kKvUnit) + span / kKvUnit + 2);
  q.units = (int)units;
  return q;
}

// Inclusive wave scan (lane order) of 64-bit integers, and a quotient that is a 32-bit one where it can be.
__device__ __forceinline__ long long wave_scan_i64(long long v) {
  auto step = [&](auto dpp) { v += dpp(v); };
  auto move = [](long long x, auto ctrl, auto mask) {
    constexpr int C = decltype(ctrl)::value, M = decltype(mask)::value;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)x, C, M, 0xF, M == 0xF);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)((uint64_t)x >> 32), C, M, 0xF, M == 0xF);
    return (long long)(((uint64_t)hi << 32) | lo);
  };
  using All = std::integral_constant<int, 0xF>;
  step([&](long long x) { return move(x, std::integral_constant<int, 0x111>{}, All{}); });   // row_shr:1
  step([&](long long x) { return move(x, std::integral_constant<int, 0x112>{}, All{}); });
  step([&](long long x) { return move(x, std::integral_constant<int, 0x114>{}, All{}); });
  step([&](long long x) { return move(x, std::integral_constant<int, 0x118>{}, All{}); });
  step([&](long long x) { return move(x, std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{}); });
  step([&](long long x) { return move(x, std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{}); });
  return v;
}
__device__ __forceinline__ long long lane_i64(long long v, int src) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, src);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)v >> 32), src);
  return (long long)(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ long long wave_sum_i64(long long v) { return lane_i64(wave_scan_i64(v), 63); }
__device__ __forceinline__ long long div_i64(long long x, long long y) {
  return ((x | y) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
}

// Linear order of a launch's work: requests in order, in each its kv heads, row tiles and units
// (at least one unit per tile, so that a row that sees nothing is written too).  Workgroup i of `target`
// takes [i * chunk, (i + 1) * chunk) of that order: an equal share, whatever the lengths.
// A tile cut between workgroups leaves one partial sum per workgroup; a workgroup has at most two
// unfinished tiles, the one it begins with (slot 2i) and the one it ends with (slot 2i + 1).
// Beginning a tile costs a workgroup about as much as kSwitch units (the rows, the table and the first
// units arrive one after the other), so every tile's units are preceded by kSwitch empty places in the
// order: without them a share of many short tiles ended 15 us after the others (64 requests of 90 to
// 8100 positions, 77 us).
// Aligned: no empty places, each tile's units padded to whole chunks, so that no workgroup crosses from
// one tile into the next.  Taken where the chunks this needs, work / (target - tiles), are no longer than
// the shares: with few tiles, that is.
struct KvShare {
  long long total, chunk;
  bool aligned;
};
struct KvWhere {
  int r;
  KvRequest q;
  long long base;    // order position of the request's first unit
};
// units of a tile, its length in the order, and a request's per kv head
__device__ __forceinline__ long long kv_step(const KvRequest& q, const KvShare& sh) {
  const int units = max(1, q.units);
  return sh.aligned ? div_i64(units + sh.chunk - 1, sh.chunk) * sh.chunk : units + kSwitch;
}
__device__ __forceinline__ long long kv_units(const KvRequest& q, const KvShare& sh) {
  return q.tiles * kv_step(q, sh);
}

__device__ __forceinline__ KvRequest lane_request(const KvRequest& q, int src) {
  KvRequest o;
  o.n = __builtin_amdgcn_readlane(q.n, src);
  o.row0 = __builtin_amdgcn_readlane(q.row0, src);
  o.len = __builtin_amdgcn_readlane(q.len, src);
  o.tiles = __builtin_amdgcn_readlane(q.tiles, src);
  o.units = __builtin_amdgcn_readlane(q.units, src);
  return o;
}

__device__ __forceinline__ int wave_scan(int v) { return wave_inclusive_scan(v); }
__device__ __forceinline__ long long wave_scan(long long v) { return wave_scan_i64(v); }
__device__ __forceinline__ int lane_value(int v, int src) { return __builtin_amdgcn_readlane(v, src); }
__device__ __forceinline__ long long lane_value(long long v, int src) { return lane_i64(v, src); }

// kv_locate in integers of type I, which hold the whole work; `q` is lane r's request when R <= 64.
template <bool BY_TILE, typename I>
__device__ __forceinline__ bool kv_locate_in(const KvAttentionProblem& a, const KvSchedule& s, int index, KvRequest q,
                                             I work, I all_tiles, KvShare* sh, KvWhere* out, long long* within) {
  const int lane = threadIdx.x & 63, hkv = a.cache.kv_heads;
  auto quot = [](I x, I y) { return (I)(sizeof(I) == 4 ? (uint32_t)x / (uint32_t)y : div_i64(x, y)); };
  // whole rounds of the four waves
  auto chunk_of = [&](I all, I workgroups) {
    return max((I)s.min_chunk, (quot(all + workgroups - 1, workgroups) + 3) & ~(I)3);
  };
  I chunk = chunk_of(work + kSwitch * all_tiles, s.target);
  bool aligned = false;
  if (all_tiles < s.target) {
    const I padded = chunk_of(work, s.target - all_tiles);
    aligned = padded <= chunk;
    if (aligned) chunk = padded;
  }
  sh->chunk = chunk;
  sh->aligned = aligned;
  const long long at = BY_TILE ? index : (long long)index * sh->chunk;
  I base = 0, tiles = 0;
  bool found = false;
  for (int r0 = 0; r0 < a.R; r0 += 64) {
    if (a.R > 64) {
      q = KvRequest{};
      if (r0 + lane < a.R) q = kv_request(a, s, r0 + lane);
    }
    const I units = max(1, q.units), step = aligned ? quot(units + chunk - 1, chunk) * chunk : units + kSwitch;
    const I mine = step * q.tiles * hkv, scan = wave_scan(mine);
    I key = scan, own = mine, first = base;
    if (BY_TILE) {
      own = (I)q.tiles * hkv;
      key = wave_scan(own);
      first = tiles;
    }
    const I excl = first + key - own;
    const uint64_t hit = found ? 0 : __ballot(excl <= at && at < excl + own);
    if (hit) {
      const int src = __ffsll((unsigned long long)hit) - 1;
      out->r = r0 + src;
      out->q = lane_request(q, src);
      out->base = base + lane_value(scan - mine, src);
      *within = at - lane_value(excl, src);
      found = true;
      if (BY_TILE) return true;      // the total is not needed
    }
    base += lane_value(scan, 63);
    if (BY_TILE) tiles += lane_value(key, 63);
  }
  sh->total = base;
  return found;
}

// The shares, and the request that holds order position index * chunk (BY_TILE: tile `index` of the
// launch, counted over requests, heads and tiles), with the place in it.  One whole wave; false past the
// end.  Up to 64 requests of less than 2^23 units and 2^18 tiles each go the short way, in 32 bits (padding
// to chunks at most doubles the work).
template <bool BY_TILE>
__device__ __forceinline__ bool kv_locate(const KvAttentionProblem& a, const KvSchedule& s, int index, KvShare* sh,
                                          KvWhere* out, long long* within) {
  const int lane = threadIdx.x & 63, hkv = a.cache.kv_heads;
  KvRequest q{};
  long long work = 0, all_tiles = 0;
  for (int r0 = 0; r0 < a.R; r0 += 64) {
    q = KvRequest{};
    if (r0 + lane < a.R) q = kv_request(a, s, r0 + lane);
    work += (long long)q.tiles * max(1, q.units);
    all_tiles += q.tiles;
  }
  work *= hkv;
  all_tiles *= hkv;
  if (a.R <= 64 && !__any(work >= (1 << 23) || all_tiles >= (1 << 18)))
    return kv_locate_in<BY_TILE, int>(a, s, index, q, lane_value(wave_scan((int)work), 63),
                                      lane_value(wave_scan((int)all_tiles), 63), sh, out, within);
  return kv_locate_in<BY_TILE, long long>(a, s, index, q, wave_sum_i64(work), wave_sum_i64(all_tiles), sh, out, within);
}

// kv_find in integers of type I, which hold the whole work; `q` is lane r's request when R <= 64.
template <bool CUT_TILE, typename I>
__device__ __forceinline__ bool kv_find_in(const KvAttentionProblem& a, const KvSchedule& s, int index, KvRequest q,
                                           I work, KvItem* out) {
  const int lane = threadIdx.x & 63;
  auto quot = [](I x, I y) { return (I)(sizeof(I) == 4 ? (uint32_t)x / (uint32_t)y : div_i64(x, y)); };
  const int chunk = (int)min((I)(1 << 27), max((I)s.min_chunk, quot(work + s.target - 1, s.target)));   // units < 2^27
  int base = 0, slots = 0;
  for (int r0 = 0; r0 < a.R; r0 += 64) {
    if (a.R > 64) {
      q = KvRequest{};
      if (r0 + lane < a.R) q = kv_request(a, s, r0 + lane);
    }
    const int splits = (int)((uint32_t)(max(0, q.units - 1 - chunk / 4)) / (uint32_t)chunk) + 1;
    const int items = q.tiles * splits, count = CUT_TILE ? (splits > 1 ? q.tiles : 0) : items;
    const int part = splits > 1 ? items : 0;
    const int ic = wave_scan(count), ip = wave_scan(part);
    const int excl = base + ic - count;
    const uint64_t hit = __ballot(excl <= index && index < excl + count);
    if (hit) {
      const int src = __ffsll((unsigned long long)hit) - 1;
      const int within = index - lane_value(excl, src);
      out->r = r0 + src;
      out->q = lane_request(q, src);
      out->splits = lane_value(splits, src);
      out->chunk = (int)((uint32_t)(out->q.units + out->splits - 1) / (uint32_t)out->splits);
      out->tile = CUT_TILE ? within : within / out->splits;
      out->split = CUT_TILE ? 0 : within % out->splits;
      out->slot = slots + lane_value(ip - part, src) + out->tile * out->splits;
      return true;
    }
    base += lane_value(ic, 63);
    slots += lane_value(ip, 63);
  }
  return false;
}

// Item `index` (CUT_TILE: all splits of the tile `index`, counted over those of two splits or more); false past the
// last.  One whole wave.
template <bool CUT_TILE>
__device__ __forceinline__ bool kv_find(const KvAttentionProblem& a, const KvSchedule& s, int index, KvItem* out) {
  const int lane = threadIdx.x & 63;
  KvRequest q{};
  long long work = 0;
  for (int r0 = 0; r0 < a.R; r0 += 64) {
    q = KvRequest{};
    if (r0 + lane < a.R) q = kv_request(a, s, r0 + lane);
    work += (long long)q.tiles * q.units;
  }
  if (a.R <= 64 && !__any(work >= (1 << 24)))
    return kv_find_in<CUT_TILE, int>(a, s, index, q, lane_value(wave_scan((int)work), 63), out);
  return kv_find_in<CUT_TILE, long long>(a, s, index, q, wave_sum_i64(work), out);
}

}  // namespace
}  // namespace moe
