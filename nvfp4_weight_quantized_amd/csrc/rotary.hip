// Rotary positions: rows rotated on their own, and rows on their way into the paged key/value cache.
#include "kv_append.h"
#include "rotary.h"

namespace moe {
namespace {

static_assert(kRotaryThreads == 256, "the kernels below");

struct RotaryShape {
  int per_block;            // tokens
  Divider pieces, heads;
};

// The rows of the tokens [t0, t0 + count) of x, rotated into out (which may be x).  A thread asks for kAhead pieces
// before it turns the first; the table is made meanwhile.  Bound by memory: 8192 rows of 32 heads of 128 (134 MB) in 25.6
// to 26.9 us, 5.0 TB/s, the rate of a copy; one row in 3.3 us.
constexpr int kAhead = 2;

__device__ __forceinline__ void rotate_rows(const RotaryProblem& p, const RotaryShape& sh, int t0, int count,
                                            RotaryTable& table) {
  const moe_rotary_t& r = p.r;
  const int pieces = sh.pieces.divisor, turned = r.interleaved ? r.pairs / 4 : r.pairs / 8;
  const int items = count * p.heads * pieces, second = r.interleaved ? 0 : r.pairs;
  const bool in_place = p.out == p.x;
  struct Item {
    int t, piece, at;      // at: first element
    uint16_t* dst;
    uint4 a, b;
  };
  auto fetch = [&](int i, Item& x) {
    if (i >= items) return;
    const int row = sh.pieces(i), t = sh.heads(row), h = row - t * p.heads;
    x.t = t;
    x.piece = i - row * pieces;
    x.at = x.piece < turned ? 8 * x.piece : 2 * r.pairs + 8 * (x.piece - turned);
    const uint16_t* src = p.x + (int64_t)(t0 + t) * p.x_stride + (size_t)h * r.head_dim + x.at;
    x.dst = p.out + (int64_t)(t0 + t) * p.out_stride + (size_t)h * r.head_dim + x.at;
    x.a = *reinterpret_cast<const uint4*>(src);
    if (second) x.b = *reinterpret_cast<const uint4*>(src + (x.piece < turned ? second : 0));
  };
  auto turn = [&](int i, Item& x) {
    if (i >= items) return;
    if (x.piece >= turned) {
      if (!in_place) *reinterpret_cast<uint4*>(x.dst) = x.a;
    } else if (r.interleaved) {
      Chunk a = chunk_of(x.a);
      rotate_neighbours(table, x.t * r.pairs + x.at / 2, a);
      *reinterpret_cast<uint4*>(x.dst) = bits_of(a);
    } else {
      Chunk a = chunk_of(x.a), b = chunk_of(x.b);
      rotate_halves(table, x.t * r.pairs + x.at, a, b);
      *reinterpret_cast<uint4*>(x.dst) = bits_of(a);
      *reinterpret_cast<uint4*>(x.dst + r.pairs) = bits_of(b);
    }
  };
  Item x[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) fetch(threadIdx.x + 256 * k, x[k]);
  rotary_table(r, p.positions, p.position_stride, t0, count, table);
  __syncthreads();
  for (int i = threadIdx.x; i < items; i += 256 * kAhead) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) turn(i + 256 * k, x[k]);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) fetch(i + 256 * (kAhead + k), x[k]);
  }
}

__global__ __launch_bounds__(256) void rotary_kernel(RotaryProblem p, RotaryShape sh) {
  __shared__ RotaryTable table;
  const int t0 = blockIdx.x * sh.per_block;
  rotate_rows(p, sh, t0, min(sh.per_block, p.T - t0), table);
}

// Elements [16g, 16g + 16) of a key row at src, rotated and rounded to bf16, as the cache's quantizer takes them; the
// row's entries begin at `entry`.
__device__ __forceinline__ void load_rotated_group(const moe_rotary_t& r, const uint16_t* src, int g,
                                                   const RotaryTable& table, int entry, float (&x)[16]) {
  uint4 w[2], other[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int at = 16 * g + 8 * e, to = r.interleaved || at >= 2 * r.pairs ? at : at < r.pairs ? at + r.pairs : at - r.pairs;
    w[e] = *reinterpret_cast<const uint4*>(src + at);
    other[e] = *reinterpret_cast<const uint4*>(src + to);
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int at = 16 * g + 8 * e;
    if (at < 2 * r.pairs) {
      Chunk a = chunk_of(w[e]);
      if (r.interleaved) {
        rotate_neighbours(table, entry + at / 2, a);
      } else {
        Chunk b = chunk_of(other[e]);
        if (at < r.pairs) rotate_halves(table, entry + at, a, b);
        else rotate_halves(table, entry + at - r.pairs, b, a);
      }
      w[e] = bits_of(a);
    }
    const Chunk y = chunk_of(w[e]);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[8 * e + i] = y.v[i];
  }
}

// Half of a key row, the groups 2s + z of all ranges s of 32 elements, into the cache: what lies there together.  The
// codes of elements [32s + 8u, +8) of all s fill 16 bytes (8 of dimension 64, twice 16 of 256), so a thread stores two
// words of 16 bytes and one of scales where a thread per group stores two dwords and a byte each time: a quarter of the
// requests.  With every element rotated it also holds both elements of its pairs.  For long steps (8192 rows of 128 with
// the gather that reads them back: 8/8 heads 28.9 against 30.5 us, 32/8 58.7 against 59.5); short ones need the threads.
template <int D>
__device__ __forceinline__ void append_key_half(const moe_nvfp4_kv_cache_t& c, const moe_rotary_t& r,
                                                const uint16_t* __restrict__ src, int h, int z, int slot,
                                                const RotaryTable& table, int entry) {
  using U = KvUnit<D>;
  constexpr int NS = D / 32;
  uint32_t code[2][NS], scale[NS];
  auto quantize = [&](int s, const float(&x)[16]) {
    quantize_group16_fast(x, c.k_gscale, &code[0][s], &code[1][s], &scale[s]);
  };
  if (!r.interleaved && 2 * r.pairs == D) {
    uint4 w[NS][2];
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int e = 0; e < 2; ++e) w[s][e] = *reinterpret_cast<const uint4*>(src + 32 * s + 16 * z + 8 * e);
#pragma unroll
    for (int s = 0; s < NS / 2; ++s) {
      float x[16], y[16];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        Chunk a = chunk_of(w[s][e]), b = chunk_of(w[s + NS / 2][e]);
        rotate_halves(table, entry + 32 * s + 16 * z + 8 * e, a, b);
        a = chunk_of(bits_of(a));
        b = chunk_of(bits_of(b));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[8 * e + i] = a.v[i], y[8 * e + i] = b.v[i];
      }
      quantize(s, x);
      quantize(s + NS / 2, y);
    }
  } else {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      float x[16];
      load_rotated_group(r, src, 2 * s + z, table, entry, x);
      quantize(s, x);
    }
  }
  uint8_t* unit = c.pages + kv_unit_offset<D>(c, slot, h);
  const int p = slot % kKvUnit;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    uint8_t* dst = unit + U::k_word(p, 2 * z + e);
    if (NS == 2) {
      *reinterpret_cast<uint2*>(dst) = uint2{code[e][0], code[e][1]};
    } else {
#pragma unroll
      for (int j = 0; j < NS / 4; ++j)
        *reinterpret_cast<uint4*>(dst + 1024 * j) =
            uint4{code[e][4 * j], code[e][4 * j + 1], code[e][4 * j + 2], code[e][4 * j + 3]};
    }
  }
  uint8_t* dst = unit + U::k_scale(p, z);
  if (NS == 2) {
    *reinterpret_cast<uint16_t*>(dst) = (uint16_t)(scale[0] | scale[1] << 8);
  } else {
#pragma unroll
    for (int j = 0; j < NS / 4; ++j)
      reinterpret_cast<uint32_t*>(dst)[j] =
          scale[4 * j] | scale[4 * j + 1] << 8 | scale[4 * j + 2] << 16 | scale[4 * j + 3] << 24;
  }
}

struct AppendRotaryBlocks {
  RotaryShape rows;            // of the queries
  int k_tokens;                // per block
  Divider k_per;               // threads of the keys per token: groups, or half rows with W > 1
  unsigned q, k, v;            // an eighth of the blocks of the queries, of the keys, of the values
};

// Three kinds of workgroups in one launch: tokens of the queries, of the keys, and windows of the values as kv_append
// takes them.  Bound by memory: 8192 rows of 32/8 heads of 128 (177 MB) in 41.5 us, 4.3 TB/s, where the queries alone run
// at the rate of a copy (25.6 us) and what is left is the vector unit and the scattered stores of keys and values.
template <int D, int W>
__global__ __launch_bounds__(256) void kv_append_rotary_kernel(moe_nvfp4_kv_cache_t c, RotaryProblem q,
                                                               const uint16_t* __restrict__ k,
                                                               const uint16_t* __restrict__ v, int64_t k_stride,
                                                               int64_t v_stride, const int32_t* __restrict__ slots,
                                                               AppendRotaryBlocks blocks) {
  constexpr int NG = D / 16;
  __shared__ RotaryTable table;
  // Workgroups go round the eight XCDs: each takes an eighth of the tokens in one run, so that the positions of a unit meet
  // in one of the caches, whose lines then reach the memory whole (8192 rows of 128 with the gather: 8/8 heads 32.4 ->
  // 28.9 us, 32/1 45.1 -> 36.0, 32/8 64.4 -> 58.7).  The kinds follow one another: mixed by groups of tokens, the queries'
  // stream drives the half-filled lines out (8192 rows of 32/8 heads alone: 41.5 against 45.2 us).
  const unsigned turn = blockIdx.x >> 3, xcd = blockIdx.x & 7;
  if (turn < blocks.k) {
    const int t0 = (xcd * blocks.k + turn) * blocks.k_tokens, count = min(blocks.k_tokens, q.T - t0);
    rotary_table(q.r, q.positions, q.position_stride, t0, count, table);
    __syncthreads();
    const int per = blocks.k_per.divisor;
    if (W > 1) {
      const int cap = c.num_pages * c.page_size;
      for (int i = threadIdx.x; i < count * per; i += 256) {
        const int t = blocks.k_per(i), rest = i - t * per, h = rest >> 1, slot = slots[t0 + t];
        if (slot >= 0 && slot < cap)
          append_key_half<D>(c, q.r, k + (int64_t)(t0 + t) * k_stride + h * D, h, rest & 1, slot, table, t * q.r.pairs);
      }
      return;
    }
    for (int i = threadIdx.x; i < count * per; i += 256) {
      const int t = blocks.k_per(i), rest = i - t * per, h = rest / NG, g = rest % NG;
      append_window<D, 1>(c, [&](int row, float(&x)[16]) {
        load_rotated_group(q.r, k + (int64_t)row * k_stride + h * D, g, table, t * q.r.pairs, x);
      }, c.k_gscale, false, h, g, t0 + t, slots, q.T);
    }
    return;
  }
  if (turn >= blocks.k + blocks.v) {
    const int t0 = (xcd * blocks.q + turn - blocks.k - blocks.v) * blocks.rows.per_block;
    if (t0 < q.T) rotate_rows(q, blocks.rows, t0, min(blocks.rows.per_block, q.T - t0), table);
    return;
  }
  const long long i = ((long long)xcd * blocks.v + turn - blocks.k) * 256 + threadIdx.x;
  const int per = c.kv_heads * NG;
  const long long wl = i / per;
  if (wl * W >= q.T) return;
  const int rest = (int)(i % per), g = rest % NG, h = rest / NG;
  const uint16_t* src = v + h * D + g * 16;
  append_window<D, W>(c, [&](int row, float(&x)[16]) { load_group16(src + (int64_t)row * v_stride, x); }, c.v_gscale,
                      true, h, g, (int)wl * W, slots, q.T);
}

RotaryLaunch plan(const RotaryProblem& p) {
  return plan_rotary(p.T, p.heads, p.r.head_dim, p.r.pairs, p.r.interleaved);
}

AppendRotaryLaunch plan(const moe_nvfp4_kv_cache_t& c, const RotaryProblem& q) {
  return plan_append_rotary(q.T, q.heads, c.kv_heads, c.head_dim, q.r.pairs, q.r.interleaved);
}

RotaryShape shape_of(const RotaryLaunch& x, int heads) {
  return RotaryShape{x.per_block, Divider::of(x.pieces), Divider::of(heads)};
}

}  // namespace

bool rotary_launchable(const RotaryProblem& p) { return rotary_fits(plan(p).blocks); }

bool kv_append_rotary_launchable(const moe_nvfp4_kv_cache_t& c, const RotaryProblem& q) {
  return rotary_fits(plan(c, q).blocks);
}

moe_status_t launch_rotary(const RotaryProblem& p, hipStream_t stream) {
  const RotaryLaunch x = plan(p);
  hipLaunchKernelGGL(rotary_kernel, dim3((unsigned)x.blocks), dim3(kRotaryThreads), 0, stream, p, shape_of(x, p.heads));
  return launch_status();
}

moe_status_t launch_kv_append_rotary(const moe_nvfp4_kv_cache_t& c, const RotaryProblem& q, const uint16_t* k,
                                     const uint16_t* v, int64_t k_stride, int64_t v_stride, const int32_t* slots,
                                     hipStream_t stream) {
  const AppendRotaryLaunch x = plan(c, q);
  const AppendRotaryBlocks b{shape_of(x.rows, q.heads), x.k_tokens,    Divider::of((uint32_t)x.k_per),
                             (unsigned)x.q,             (unsigned)x.k, (unsigned)x.v};
  const dim3 grid((unsigned)x.blocks), block(kRotaryThreads);
  with_head_dim(c.head_dim, [&](auto tag) {
    constexpr int D = decltype(tag)::value;
    if (x.quads)
      hipLaunchKernelGGL((kv_append_rotary_kernel<D, 4>), grid, block, 0, stream, c, q, k, v, k_stride, v_stride,
                         slots, b);
    else
      hipLaunchKernelGGL((kv_append_rotary_kernel<D, 1>), grid, block, 0, stream, c, q, k, v, k_stride, v_stride,
                         slots, b);
  });
  return launch_status();
}

}  // namespace moe
