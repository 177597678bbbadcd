// Host side of the rotary kernels: tokens of a workgroup, and how many workgroups a call takes.  No HIP: it is tested on
// its own.
#pragma once

#include <algorithm>
#include <cstdint>

#include "kv_limits.h"

namespace moe {

constexpr int kRotaryEntries = 1024;      // cosines and sines that a workgroup holds in LDS, 8 KB
constexpr int kRotaryThreads = 256;

namespace {

struct RotaryLaunch {
  int pieces;         // of a head, one thread each: a pair of chunks of eight elements (halves), or one chunk (neighbours, and
                      // what lies behind the rotated elements)
  int per_block;      // tokens
  int64_t blocks;
};

// Tokens per workgroup: about `items` pieces of `per` a token, within what LDS holds of angles.
int rotary_tokens(int64_t T, int pairs, int64_t per, int64_t items) {
  const int64_t most = std::min((int64_t)kRotaryEntries / pairs, std::max((int64_t)1, items / per));
  // small steps: a workgroup per token until the card is full
  return (int)std::max((int64_t)1, std::min(most, T / 1024));
}

int64_t rotary_blocks(int64_t n, int64_t per_block) { return (n + per_block - 1) / per_block; }

RotaryLaunch plan_rotary(int64_t T, int heads, int head_dim, int pairs, bool interleaved) {
  RotaryLaunch x;
  x.pieces = (interleaved ? pairs / 4 : pairs / 8) + (head_dim - 2 * pairs) / 8;
  x.per_block = rotary_tokens(T, pairs, (int64_t)heads * x.pieces, 2048);
  x.blocks = rotary_blocks(T, x.per_block);
  return x;
}

// The rotating append: workgroups of the queries, of the keys and of the values, an eighth of each kind per XCD.
struct AppendRotaryLaunch {
  RotaryLaunch rows;      // of the queries
  bool quads;             // half rows of keys and quads of values, as the append's rule has them
  int k_per, k_tokens;    // threads of the keys per token: groups, or half rows; tokens per workgroup
  int64_t q, k, v;        // an eighth of the workgroups of each kind
  int64_t blocks;
};

AppendRotaryLaunch plan_append_rotary(int64_t T, int heads, int kv_heads, int head_dim, int pairs, bool interleaved) {
  AppendRotaryLaunch x;
  const int64_t per = (int64_t)kv_heads * (head_dim / 16);
  x.rows = plan_rotary(T, heads, head_dim, pairs, interleaved);
  x.quads = 2 * T * per >= kKvAppendQuadThreads;
  x.k_per = (int)(x.quads ? 2 * kv_heads : per);
  x.k_tokens = rotary_tokens(T, pairs, x.k_per, x.quads ? 256 : 512);
  x.q = (x.rows.blocks + 7) / 8;
  x.k = (rotary_blocks(T, x.k_tokens) + 7) / 8;
  x.v = (rotary_blocks((x.quads ? (T + 3) / 4 : T) * per, kRotaryThreads) + 7) / 8;
  x.blocks = 8 * (x.q + x.k + x.v);
  return x;
}

// A launch holds fewer than 2^32 work-items.  Within the limits of the arguments every call does (the rows take a
// workgroup per token at most, of less than 2^24; the append comes to 0.78 * 2^32), which a change of the constants above
// could undo.
bool rotary_fits(int64_t blocks) { return blocks * kRotaryThreads < (int64_t)1 << 32; }

}  // namespace
}  // namespace moe
