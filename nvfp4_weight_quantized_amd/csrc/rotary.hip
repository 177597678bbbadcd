// Rotary positions: rows rotated on their own, and rows on their way into the paged key/value cache.
#include "kv_append.h"
#include "rotary.h"

namespace moe {
namespace {

// Pieces of a head that one thread takes: a pair of chunks of eight elements (halves), or one chunk (neighbours, and
// what lies behind the rotated elements).
__host__ __device__ inline int rotary_pieces(const moe_rotary_t& r) {
  return (r.interleaved ? r.pairs / 4 : r.pairs / 8) + (r.head_dim - 2 * r.pairs) / 8;
}

// The rows of the tokens [t0, t0 + count) of x, rotated into out (which may be x).
__device__ __forceinline__ void rotate_rows(const RotaryProblem& p, int t0, int count, const float2* table) {
  const moe_rotary_t& r = p.r;
  const int pieces = rotary_pieces(r), turned = r.interleaved ? r.pairs / 4 : r.pairs / 8;
  const bool in_place = p.out == p.x;
  for (int i = threadIdx.x; i < count * p.heads * pieces; i += blockDim.x) {
    const int row = i / pieces, piece = i - row * pieces, t = row / p.heads, h = row - t * p.heads;
    const uint16_t* src = p.x + (int64_t)(t0 + t) * p.x_stride + (size_t)h * r.head_dim;
    uint16_t* dst = p.out + (int64_t)(t0 + t) * p.out_stride + (size_t)h * r.head_dim;
    if (piece >= turned) {
      const int at = 2 * r.pairs + 8 * (piece - turned);
      if (!in_place) *reinterpret_cast<uint4*>(dst + at) = *reinterpret_cast<const uint4*>(src + at);
    } else if (r.interleaved) {
      Chunk a = load_chunk(src + 8 * piece);
      rotate_neighbours(table + t * r.pairs + 4 * piece, a);
      store_chunk(dst + 8 * piece, a);
    } else {
      Chunk a = load_chunk(src + 8 * piece), b = load_chunk(src + r.pairs + 8 * piece);
      rotate_halves(table + t * r.pairs + 8 * piece, a, b);
      store_chunk(dst + 8 * piece, a);
      store_chunk(dst + r.pairs + 8 * piece, b);
    }
  }
}

__global__ __launch_bounds__(256) void rotary_kernel(RotaryProblem p, int per_block) {
  __shared__ float2 table[kRotaryEntries];
  const int t0 = blockIdx.x * per_block, count = min(per_block, p.T - t0);
  rotary_table(p.r, p.positions, p.position_stride, t0, count, table);
  __syncthreads();
  rotate_rows(p, t0, count, table);
}

// Elements [16g, 16g + 16) of a key row at src, rotated and rounded to bf16, as the cache's quantizer takes them.
__device__ __forceinline__ void load_rotated_group(const moe_rotary_t& r, const uint16_t* src, int g,
                                                   const float2* turn, float (&x)[16]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int at = 16 * g + 8 * e;
    Chunk a = load_chunk(src + at);
    if (at < 2 * r.pairs) {
      if (r.interleaved) {
        rotate_neighbours(turn + at / 2, a);
      } else if (at < r.pairs) {
        Chunk b = load_chunk(src + at + r.pairs);
        rotate_halves(turn + at, a, b);
      } else {
        Chunk b = load_chunk(src + at - r.pairs);
        rotate_halves(turn + at - r.pairs, b, a);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[8 * e + i] = bf16_to_f32(f32_to_bf16(a.v[i]));
  }
}

// Blocks of the queries move memory, those of the keys and values keep the vector unit busy: a compute unit should hold
// both, so they take turns, `run` blocks of the queries after each of the others for as long as both last.
struct AppendRotaryBlocks {
  int q_tokens, k_tokens;      // per block
  unsigned q, k, v;            // blocks of the queries, of the keys, of the values
  unsigned run, turns;
};

// Three kinds of workgroups in one launch: tokens of the queries, of the keys, and windows of the values as kv_append
// takes them.
template <int D, int W>
__global__ __launch_bounds__(256) void kv_append_rotary_kernel(moe_nvfp4_kv_cache_t c, RotaryProblem q,
                                                               const uint16_t* __restrict__ k,
                                                               const uint16_t* __restrict__ v, int64_t k_stride,
                                                               int64_t v_stride, const int32_t* __restrict__ slots,
                                                               AppendRotaryBlocks blocks) {
  constexpr int NG = D / 16;
  __shared__ float2 table[kRotaryEntries];
  // block: first the keys', then the values', from there on the queries'
  unsigned block = blockIdx.x;
  const unsigned period = blocks.run + 1, mixed = blocks.turns * period, others = blocks.k + blocks.v;
  if (block < mixed) {
    const unsigned turn = block / period, place = block - turn * period;
    block = place == 0 ? turn : others + turn * blocks.run + place - 1;
  } else if (blocks.turns == others) {
    block = others + (block - mixed) + blocks.turns * blocks.run;
  } else {      // every query is taken
    block = blocks.turns + (block - mixed);
  }
  if (block < blocks.k) {
    const int t0 = block * blocks.k_tokens, count = min(blocks.k_tokens, q.T - t0);
    rotary_table(q.r, q.positions, q.position_stride, t0, count, table);
    __syncthreads();
    const int per = c.kv_heads * NG;
    for (int i = threadIdx.x; i < count * per; i += 256) {
      const int t = i / per, rest = i - t * per, h = rest / NG, g = rest % NG;
      append_window<D, 1>(c, [&](int row, float(&x)[16]) {
        load_rotated_group(q.r, k + (int64_t)row * k_stride + h * D, g, table + t * q.r.pairs, x);
      }, c.k_gscale, false, h, g, t0 + t, slots, q.T);
    }
    return;
  }
  if (block >= others) {
    const int t0 = (block - others) * blocks.q_tokens, count = min(blocks.q_tokens, q.T - t0);
    rotary_table(q.r, q.positions, q.position_stride, t0, count, table);
    __syncthreads();
    rotate_rows(q, t0, count, table);
    return;
  }
  const long long i = (long long)(block - blocks.k) * 256 + threadIdx.x;
  const int per = c.kv_heads * NG;
  const long long wl = i / per;
  if (wl * W >= q.T) return;
  const int rest = (int)(i % per), g = rest % NG, h = rest / NG;
  const uint16_t* src = v + h * D + g * 16;
  append_window<D, W>(c, [&](int row, float(&x)[16]) { load_group16(src + (int64_t)row * v_stride, x); }, c.v_gscale,
                      true, h, g, (int)wl * W, slots, q.T);
}

// Tokens per block: about `items` pieces of `per` a token, within what LDS holds of angles.
int tokens_per_block(int64_t T, int pairs, int64_t per, int64_t items) {
  const int64_t most = std::min((int64_t)kRotaryEntries / pairs, std::max((int64_t)1, items / per));
  // small steps: a block per token until the card is full
  return (int)std::max((int64_t)1, std::min(most, T / 1024));
}

unsigned blocks_for(int64_t T, int per_block) { return (unsigned)((T + per_block - 1) / per_block); }

}  // namespace

moe_status_t launch_rotary(const RotaryProblem& p, hipStream_t stream) {
  const int per_block = tokens_per_block(p.T, p.r.pairs, (int64_t)p.heads * rotary_pieces(p.r), 2048);
  hipLaunchKernelGGL(rotary_kernel, dim3(blocks_for(p.T, per_block)), dim3(256), 0, stream, p, per_block);
  return launch_status();
}

moe_status_t launch_kv_append_rotary(const moe_nvfp4_kv_cache_t& c, const RotaryProblem& q, const uint16_t* k,
                                     const uint16_t* v, int64_t k_stride, int64_t v_stride, const int32_t* slots,
                                     hipStream_t stream) {
  const int64_t per = (int64_t)c.kv_heads * (c.head_dim / 16), T = q.T;
  const bool quads = 2 * T * per >= kAppendQuadThreads;
  AppendRotaryBlocks b;
  b.q_tokens = tokens_per_block(T, q.r.pairs, (int64_t)q.heads * rotary_pieces(q.r), 2048);
  b.k_tokens = tokens_per_block(T, q.r.pairs, per, 512);
  b.q = blocks_for(T, b.q_tokens);
  b.k = blocks_for(T, b.k_tokens);
  b.v = (unsigned)(((quads ? (T + 3) / 4 : T) * per + 255) / 256);
  const unsigned others = b.k + b.v;
  b.run = std::max(1u, b.q / others);
  b.turns = std::min(others, b.q / b.run);
  const dim3 grid(b.q + others);
  with_head_dim(c.head_dim, [&](auto tag) {
    constexpr int D = decltype(tag)::value;
    if (quads)
      hipLaunchKernelGGL((kv_append_rotary_kernel<D, 4>), grid, dim3(256), 0, stream, c, q, k, v, k_stride, v_stride,
                         slots, b);
    else
      hipLaunchKernelGGL((kv_append_rotary_kernel<D, 1>), grid, dim3(256), 0, stream, c, q, k, v, k_stride, v_stride,
                         slots, b);
  });
  return launch_status();
}

}  // namespace moe
