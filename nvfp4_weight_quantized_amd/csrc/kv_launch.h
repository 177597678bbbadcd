// Host side of the attention over the paged cache: which kernels a call launches, their grids and workspace, from
// what the host knows (rows, requests, the table's width; not the lengths).  No HIP: it is tested on its own.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "kv_limits.h"

namespace moe {

namespace {

struct KvSchedule {
  int bm;          // rows per tile
  int target;      // items aimed at, per kv head
  int min_chunk;   // units
  int min_rows, max_rows;   // requests of this launch: min_rows < rows <= max_rows
};

// Waves per SIMD the few-row kernel is built for (registers, ring), and so its resident workgroups per compute unit.
template <int D, int MI, int NW = 4>
constexpr int rows_occupancy() {
  if (NW > 4) return NW / 4;      // one workgroup
  return D == 256 ? (MI == 2 ? 1 : 2) : D == 128 ? (MI == 2 ? 2 : 4) : (MI == 2 ? 3 : 4);
}

// One launch: schedule, grid and workspace.
struct Launch {
  bool shares;        // few-row kernel (equal shares) or tile kernel (items)
  bool whole;         // tiles are not cut: no partial sums, no combine launch
  int rs;             // tile kernel: rows per wave
  KvSchedule s;
  int64_t grid;       // workgroups
  int64_t tiles;      // bound on the row tiles over all heads
  int64_t join;       // tiles to join: of shares, all (== tiles) or those cut at the end of each but the last; of items,
                      // the cut ones over all heads
  size_t o_bytes, bytes;
};

constexpr int kCus = 256;              // compute units of the card
constexpr int kRowsMinChunk = 4;       // units: one per wave
constexpr int kSwitch = 8;             // empty places before a tile's units in the order of the shares (KvShare)
// Few rows, block tables of at most so many units and at most so many tiles: a workgroup of 8 waves takes a
// tile whole.  These are bound by latency, and whole tiles save the combine launch and its gap (one request
// of 1024 positions, 32/4 heads, dimension 128: 11.1 us on the GPU, 10.8 us a call, against 12.1 and 13.8 us; 16 waves
// took 1.9 us longer than 8).
constexpr int kWholeUnits = 64, kWholeTiles = 256;
constexpr int kTilesTarget = kCus;     // one workgroup is resident per compute unit
constexpr int kTilesMinChunk = 8;      // units: four steps
// Many rows, block tables of at most so many steps: tiles are not cut, for the same reason (3 requests of 243 to
// 337 tokens, 4/2 heads, dimension 64, 17 units: 13.2 against 16.2 us; 2 requests of 921, 8 heads, 29 units:
// 20.7 against 24.4 us; 5 of 527 to 763, 24 units, 8 heads on 1 of dimension 128: 25.3 against 35.3 us; but 3 of 140 to
// 439, 3 heads, dimension 128, 26 units: 24.9 against 21.9 us).  Past that it goes by the number of tiles, which the
// host does not know well: 4 chunks of 100 on up to 900 positions, 30 units, dimension 128, 29.5 against 36.9 us with
// 32/8 heads, 28.4 against 20.5 us with 8/1; 300 tokens and 3 single ones on 1000, 32 units, 29.4 against 18.3 us.
constexpr int kTilesWholeSteps = 12;
constexpr int64_t kWideWork = 32768;   // tiles * units of the table from which 32-row waves are taken
// Requests of more rows go to the tile kernel where both run.  32 requests on 4000 positions, 32/8 heads,
// dimension 128: 64 rows each 96 us, in the tile kernel 145 us; 128 rows each 149 us, in the few-row kernel
// 144 us, but then 12 short prompts of up to 32 tokens take 14.2 instead of 7.9 us (two more launches).
constexpr int kRowsSplit = 64;
// Requests * heads * units of the table up to which the tile kernel takes requests of few rows too, and two
// launches are saved (5 prompts of 527 to 763 tokens, 4/2 heads, dimension 64: 17.5 against 21.3 us; 4 chunks of 100
// on up to 900 positions, 32/8 heads, dimension 128: 36.9 against 41.3 us; 300 tokens and 3 single ones on 1000: 18.3
// against 30.8 us).  A request of one row and a long context takes several times longer there.
constexpr int64_t kAloneWork = 2048;

// Query rows, over all heads, beyond one token per request, from which a long request is taken to be among many short
// ones and the tile kernel is launched beside the few-row kernel.  The few-row kernel alone against both:
// 32/8 heads, dimension 128: 1000 single tokens and a chunk of 500 (16k rows) 246 against 408 us, 300 and 900 (29k)
// 185 / 220, 200 requests of 6 tokens (32k) 129 / 153, 400 and 1500 on 4000 positions (48k) 513 / 417, 400 and 6000
// (192k) 1418 / 592; 8/2 heads, dimension 64: 400 and 3000 (24k) 125 / 139, 400 and 6000 (48k) 245 / 210.
// Where the tile kernel takes all requests (kAloneWork) from 1024 tokens on: 60 prompts of 1 to 59 tokens, 4/4 heads,
// dimension 64, 14.8 / 7.0 us, 90 of 1 to 30, 32/8 heads, dimension 128, 44.3 / 24.4 us.
constexpr int64_t kLikelyRows = 40960;

int rows_resident(int D, int bm) {
  if (D == 64) return bm == 16 ? rows_occupancy<64, 1>() : rows_occupancy<64, 2>();
  if (D == 128) return bm == 16 ? rows_occupancy<128, 1>() : rows_occupancy<128, 2>();
  return bm == 16 ? rows_occupancy<256, 1>() : rows_occupancy<256, 2>();
}

// Most requests of more than min_rows rows that a step of T tokens can hold.  (A padded batch of 1000 single tokens,
// T = 1024, once also launched the tile kernel: with R in place of this bound its workgroups, each with a search of all
// lengths, made 384 us 1220 us.)
int64_t requests_of(int min_rows, int32_t T, int32_t R, int32_t G) {
  return std::min({(int64_t)R, (int64_t)T, (int64_t)T * G / (min_rows + 1)});
}

// Requests with min_rows < rows <= max_rows in tiles of bm rows.  Few rows: as many shares as workgroups
// are resident at once.  Many rows: with chunk >= sum(tiles * units) / target the items are
// sum tiles * ceil(units / chunk) <= tiles + target per kv head; those of requests with two splits or
// more number at most twice target, and so their tiles at most target.
Launch plan_launch(bool shares, int bm, int min_rows, int max_rows, int32_t T, int32_t R, int32_t G, int32_t hkv,
                   int32_t D, int64_t table_units) {
  Launch p{};
  p.shares = shares;
  const int64_t with_rows = requests_of(min_rows, T, R, G);
  const int64_t tiles = std::min(with_rows + (int64_t)T * G / bm, with_rows * (((int64_t)max_rows + bm - 1) / bm));
  p.tiles = tiles * hkv;
  size_t slots;
  p.whole = shares && bm == 16 && table_units <= kWholeUnits && p.tiles <= kWholeTiles;
  if (p.whole) {
    p.s = KvSchedule{bm, 1, 1, min_rows, max_rows};
    p.grid = p.tiles;
    slots = 0;
  } else if (shares) {
    p.s = KvSchedule{bm, kCus * rows_resident(D, bm), kRowsMinChunk, min_rows, max_rows};
    // no more than the shares of least length that the table's units make (kv_request)
    const int64_t most = std::min(table_units, (int64_t)1 << 32) + (bm + kKvUnit) / kKvUnit + 2 + kSwitch;
    p.grid = std::min((int64_t)p.s.target, p.tiles * ((most + kRowsMinChunk - 1) / kRowsMinChunk));
    p.join = std::min(p.tiles, p.grid - 1);
    slots = 2 * (size_t)p.s.target;
  } else {
    p.whole = table_units <= kTilesWholeSteps * (D == 256 ? 1 : 2);
    p.s = KvSchedule{bm, std::max(1, kTilesTarget / hkv), p.whole ? 1 << 20 : kTilesMinChunk, min_rows, max_rows};
    p.grid = (tiles + (p.whole ? 0 : p.s.target)) * hkv;
    p.join = p.whole ? 0 : std::min(tiles, (int64_t)p.s.target) * hkv;      // a cut tile has two items or more
    slots = p.whole ? 0 : 2 * (size_t)p.s.target * hkv;
  }
  p.o_bytes = slots * bm * D * 4;
  p.bytes = p.o_bytes + slots * 2 * bm * 4;
  return p;
}

// The launches of a call: the few-row kernel, the tile kernel, or both, each on its requests.
struct Launches {
  int n;
  Launch l[2];
};

Launches plan_launches(int32_t T, int32_t R, int32_t G, int32_t hkv, int32_t D, int64_t table_units) {
  Launches x{};
  const int64_t rows = (int64_t)T * G;
  // Requests of more than kRowsSplit rows are certain, or likely.
  const bool alone = R == 1 || (int64_t)R * hkv * std::min(table_units, (int64_t)1 << 32) <= kAloneWork;
  const bool likely = T > R && (alone ? T >= 1024 : ((int64_t)T - R) * G * hkv >= kLikelyRows);
  const bool tiles = rows > (int64_t)kRowsSplit * R || likely;
  const bool few = !tiles || !alone;
  if (tiles) {
    // 32 rows per wave (256 per tile) at twice the rate, 16 rows (128) with twice the tiles.  Measured, 32/8
    // heads, dimension 128: prompt of 8192 (264k units over all tiles) 572 against 849 us, 512 tokens on
    // 20000 positions (46k) 211 against 275 us, prompt of 2000 (17k) 105 against 75 us.  The host knows the
    // table's width, not the lengths; a wide table only means the slower of the two for a short step.
    const int min_rows = few ? kRowsSplit : 0;
    const int64_t wide = requests_of(min_rows, T, R, G) + rows / 256;
    const int rs = D != 256 && wide * hkv * std::min(table_units, (int64_t)1 << 26) >= kWideWork ? 32 : 16;
    x.l[x.n] = plan_launch(false, 8 * rs, min_rows, 0x7FFFFFFF, T, R, G, hkv, D, table_units);
    x.l[x.n++].rs = rs;
  }
  if (few) {
    const int bm = tiles || rows > 16 * (int64_t)R ? 32 : 16;
    x.l[x.n++] = plan_launch(true, bm, 0, tiles ? kRowsSplit : 0x7FFFFFFF, T, R, G, hkv, D, table_units);
  }
  return x;
}

// A launch holds fewer than 2^32 work-items (512 per workgroup, those that fill rows included).
bool launchable(const Launches& x) {
  for (int i = 0; i < x.n; ++i)
    if ((x.l[i].grid + kCus) * 512 >= (int64_t)1 << 32) return false;
  return true;
}

}  // namespace
}  // namespace moe
