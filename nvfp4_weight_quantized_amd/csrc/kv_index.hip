// Which pages of the key/value cache a query row reads: 8-bit means of the pages' keys (the index), and the choice of
// pages by the products of the rows with them.
//
// Index of a page and head, from the keys K_p = d_k * e2m1 * e4m3 of the n positions it holds:
//   S_d = sum_p K_p,d / (2^-10 d_k), a whole number (e2m1 is a multiple of 2^-1, e4m3 of 2^-9), summed exactly,
//   A = max_d |S_d|, code_d = rint(127 S_d / A), scale = fp32(A / (127 * 1024 n)): code * scale * d_k is the mean.
// Score of a page for a row of the kv head, with x the row of one head of its group, a = max_d |x_d|,
// x8 = rint(x * fp32(127 / a)):
//   score = fp32(max over the group of fp32((x8 . code) * a) * scale), x8 . code a whole number below 2^24.
// Nothing here depends on the order of a sum, so equal inputs choose equal pages everywhere, and a row's choice does not
// depend on its neighbours; a row's factors that are the same for all pages are left out.
#include "kv_layout.h"
#include "kv_step.h"

namespace moe {
namespace {

// ------------------------------------------------------------------------------------ index
// Pages that hold a request's new rows, as far as the table reaches.
__device__ __forceinline__ int first_page(const KvStep& s, const StepRequest& q) {
  return max(q.len - q.n, 0) / s.page_size;
}
__device__ __forceinline__ int touched_pages(const KvStep& s, const StepRequest& q) {
  if (q.n == 0 || q.len == 0) return 0;
  return max(min((q.len - 1) / s.page_size, s.width - 1) - first_page(s, q) + 1, 0);
}

// Sum over the 16 lanes of a row, in all of them.
__device__ __forceinline__ int row_sum(int v) {
  v += dpp_i<kDppQuad1032>(v, v);
  v += dpp_i<kDppQuad2301>(v, v);
  v += dpp_i<kDppRowHalfMirror>(v, v);
  v += dpp_i<kDppRowMirror>(v, v);
  return v;
}

// A workgroup per touched page and head, its four waves every fourth unit each.  A lane holds one position (of 16) and
// the elements [8u, 8u + 8) of every 32, as the unit's 16-byte pieces give them; 16 units are summed in 32 bits (|S| of
// 512 positions is below 2^31), what lies beyond in 64.
template <int D>
__global__ __launch_bounds__(256) void kv_index_kernel(moe_nvfp4_kv_cache_t c, int8_t* __restrict__ codes,
                                                       float* __restrict__ scales, KvStep s) {
  using U = KvUnit<D>;
  constexpr int NS = D / 32, NL = NS / 2, kFlush = 16;
  __shared__ long long sums[D], tops[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, u4 = lane >> 4, n16 = lane & 15, h = blockIdx.y;
  StepRequest q;
  int within;
  if (!step_find(s, blockIdx.x, [&](const StepRequest& x) { return touched_pages(s, x); }, &q, &within)) return;
  const int b = first_page(s, q) + within, page = s.table[(size_t)q.r * s.width + b];
  if (page < 0 || page >= c.num_pages) return;
  const int held = min(c.page_size, q.len - b * c.page_size), units = (held + kKvUnit - 1) / kKvUnit;
  if (tid < D) sums[tid] = 0;
  __syncthreads();
  const uint8_t* first = c.pages + kv_unit_offset<D>(c, page * c.page_size, h);
  for (int u0 = wave; u0 < units; u0 += 4 * kFlush) {
    int acc[NS][8];
#pragma unroll
    for (int k = 0; k < NS; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[k][e] = 0;
    for (int u = u0; u < min(units, u0 + 4 * kFlush); u += 4) {
      const uint8_t* unit = first + (size_t)u * U::kBytes;
      uint32_t w[2 * NS], sc[NS / 2];
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const uint4 x = *reinterpret_cast<const uint4*>(unit + 1024 * j + 16 * lane);
        w[4 * j] = x.x, w[4 * j + 1] = x.y, w[4 * j + 2] = x.z, w[4 * j + 3] = x.w;
      }
#pragma unroll
      for (int j = 0; j < NS / 2; ++j)
        sc[j] = *reinterpret_cast<const uint32_t*>(unit + U::kKScales + (16 * (u4 >> 1) + n16) * 2 * NS + 4 * j);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const bool seen = kKvUnit * u + 16 * half + n16 < held;
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          const int word = half * NS + k, byte = word & 3;
          const int bits = (int)sc[word >> 2];
          const float f = 1024.f * (byte == 0   ? __builtin_amdgcn_cvt_f32_fp8(bits, 0)
                                    : byte == 1 ? __builtin_amdgcn_cvt_f32_fp8(bits, 1)
                                    : byte == 2 ? __builtin_amdgcn_cvt_f32_fp8(bits, 2)
                                                : __builtin_amdgcn_cvt_f32_fp8(bits, 3));
          const f32x2 e[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[word], 1.0f, 0),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[word], 1.0f, 1),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[word], 1.0f, 2),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[word], 1.0f, 3)};
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[k][i] += seen ? (int)(e[i >> 1][i & 1] * f) : 0;      // exact
        }
      }
    }
#pragma unroll
    for (int k = 0; k < NS; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int v = row_sum(acc[k][i]);
        if (n16 == 0)
          atomicAdd(reinterpret_cast<unsigned long long*>(&sums[32 * k + 8 * u4 + i]), (unsigned long long)(long long)v);
      }
  }
  __syncthreads();
  const long long sum = tid < D ? sums[tid] : 0;
  long long top = sum < 0 ? -sum : sum;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = max(top, (long long)__shfl_xor(top, off));
  if (lane == 0) tops[wave] = top;
  __syncthreads();
  top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
  const size_t at = (size_t)page * c.kv_heads + h;
  // in 64 bits: a quotient half way between two whole numbers is exact, others are further from it than their rounding
  if (tid < D) codes[at * D + tid] = top > 0 ? (int8_t)(int)rint(127.0 * (double)sum / (double)top) : (int8_t)0;
  if (tid == 0) scales[at] = (float)((double)top / (130048.0 * held));
}

// ------------------------------------------------------------------------------------ choice
// A workgroup takes some tokens of a request and one kv head: their rows in 8 bits into LDS as matrix operands, the
// products of all of them with 16 pages at a time on the matrix unit (the rows are the first operand, so a lane holds one
// page's products with four rows), a key per token and page (its score as an ordered integer) into LDS, and then a wave
// per token, or with many pages the whole workgroup, takes the top_k largest keys.
//
// Rows of a 16-row block, so that the heads of a token meet in one lane, without exchange:
//   several tokens: lane quarter q4 holds the rows 4*q4 + i; with HS = 4 these are heads 4*block + i of token q4 of the
//   group (heads past the group's last repeat it), with HS = 2 or 1 (as many heads) two or four tokens';
//   one token (kOne): head 16*block + 4*q4 + i, and the four quarters meet by lane exchange.
typedef int i32x4 __attribute__((ext_vector_type(4)));

struct SelectShape {
  int tokens;      // per workgroup
  int blocks;      // 16-row blocks of a group of tokens
  int groups;      // groups of tokens
  int stride;      // keys per token
  uint32_t work_groups;
};

constexpr int kOne = 0;
constexpr int group_tokens(int HS) { return HS == kOne ? 1 : 16 / HS; }

// The rows of the workgroup's tokens in 8 bits: operand bytes codes[block][step][lane][16] and tops[block][row].
template <int D, int HS>
__device__ __forceinline__ void select_rows(const KvSelectProblem& p, const StepRequest& q, int h, int tok0,
                                            const SelectShape& sh, int8_t* codes, float* tops) {
  constexpr int LPR = D / 16;      // lanes per row, 16 elements each
  const int part = threadIdx.x % LPR, rows = 16 * sh.blocks * sh.groups;
  for (int row = threadIdx.x / LPR; row < rows; row += blockDim.x / LPR) {
    const int block = row / 16, r16 = row & 15;
    int t, g;
    if (HS == kOne) {
      t = 0;
      g = row;
    } else {
      const int grp = block / sh.blocks, hb = block - grp * sh.blocks;
      t = grp * (16 / HS) + r16 / HS;
      g = hb * 4 + r16 % HS;
    }
    t = min(tok0 + t, q.n - 1);
    g = min(g, p.G - 1);
    const uint4* src = reinterpret_cast<const uint4*>(p.q + (int64_t)(q.row0 + t) * p.q_stride +
                                                      (size_t)(h * p.G + g) * D + 16 * part);
    const uint4 w0 = src[0], w1 = src[1];
    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    float x[16], top = 0.f;
    bool fine = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      fine &= fabsf(x[i]) <= 0x1p100f;
      top = fmaxf(top, fabsf(x[i]));
    }
    if (!fine) top = INFINITY;
    top = fmaxf(top, __int_as_float(dpp_i<kDppQuad1032>(__float_as_int(top), __float_as_int(top))));
    top = fmaxf(top, __int_as_float(dpp_i<kDppQuad2301>(__float_as_int(top), __float_as_int(top))));
    if (LPR > 4) top = fmaxf(top, __int_as_float(dpp_i<kDppRowHalfMirror>(__float_as_int(top), __float_as_int(top))));
    if (LPR > 8) top = fmaxf(top, __int_as_float(dpp_i<kDppRowMirror>(__float_as_int(top), __float_as_int(top))));
    const bool use = top >= 0x1p-100f && top <= 0x1p100f;
    const float inv = use ? __fdiv_rn(127.f, top) : 0.f;
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      out[i] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        out[i] |= (uint32_t)((use ? (int)rintf(x[4 * i + e] * inv) : 0) & 0xFF) << (8 * e);
    }
    // element d of the row: step d / 64, lane 16 * ((d % 64) / 16) + row
    *reinterpret_cast<uint4*>(codes + ((size_t)block * (D / 64) + part / 4) * 1024 + (16 * (part & 3) + r16) * 16) =
        uint4{out[0], out[1], out[2], out[3]};
    if (part == 0) tops[row] = use ? top : 0.f;
  }
}

// Keys of the pages [0, pages) for the workgroup's tokens: keys[token * stride + page], 0 for a page that is not in the
// cache.  A wave takes 64 pages at a time, whose codes are all asked for before the first product.
template <int D, int HS, int NW>
__device__ __forceinline__ void select_scores(const KvSelectProblem& p, const int32_t* __restrict__ table, int h,
                                              int pages, const SelectShape& sh, const int8_t* codes, const float* tops,
                                              uint32_t* keys) {
  constexpr int KS = D / 64, TPL = HS == kOne ? 1 : 4 / HS;      // tokens of a lane
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q4 = lane >> 4, n16 = lane & 15, hkv = p.index.kv_heads;
  for (int j0 = 64 * wave; j0 < pages; j0 += 64 * NW) {
    i32x4 b[4][KS];
    float scale[4];
    bool good[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int j = j0 + 16 * x + n16, page = j < pages ? table[j] : -1;
      good[x] = page >= 0 && page < p.index.num_pages;
      const size_t at = good[x] ? (size_t)page * hkv + h : 0;
      scale[x] = p.index.scales[at];
#pragma unroll
      for (int k = 0; k < KS; ++k)
        b[x][k] = *reinterpret_cast<const i32x4*>(p.index.codes + at * D + 64 * k + 16 * q4);
    }
    for (int grp = 0; grp < sh.groups; ++grp) {
      float best[4][TPL];
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < TPL; ++y) best[x][y] = -INFINITY;
      for (int blk = 0; blk < sh.blocks; ++blk) {
        const int8_t* a = codes + (size_t)(grp * sh.blocks + blk) * KS * 1024 + 16 * lane;
        i32x4 rows[KS];
#pragma unroll
        for (int k = 0; k < KS; ++k) rows[k] = *reinterpret_cast<const i32x4*>(a + 1024 * k);
        const float4 top = *reinterpret_cast<const float4*>(tops + 16 * (grp * sh.blocks + blk) + 4 * q4);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          i32x4 dot = {0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < KS; ++k) dot = __builtin_amdgcn_mfma_i32_16x16x64_i8(rows[k], b[x][k], dot, 0, 0, 0);
          const float s[4] = {(float)dot[0] * top.x, (float)dot[1] * top.y, (float)dot[2] * top.z,
                              (float)dot[3] * top.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) best[x][i * TPL / 4] = fmaxf(best[x][i * TPL / 4], s[i]);
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
#pragma unroll
        for (int y = 0; y < TPL; ++y) {
          float v = best[x][y];
          if (HS == kOne) {
            v = fmaxf(v, __shfl_xor(v, 16));
            v = fmaxf(v, __shfl_xor(v, 32));
          }
          // 1 .. 0xFFFFFFFE
          const uint32_t key = good[x] ? min(max(order_key(v * scale[x]), 1u), 0xFFFFFFFEu) : 0u;
          const int t = HS == kOne ? 0 : grp * (16 / HS) + q4 * TPL + y, j = j0 + 16 * x + n16;
          if ((HS != kOne || q4 == 0) && j < sh.stride) keys[(size_t)t * sh.stride + j] = key;
        }
      }
    }
  }
}

// The top_k largest of a token's keys, by W waves (1 or all of the workgroup's; `me` of them), 64 * W * 32 keys at most:
// the threshold by halving the interval of keys that holds it, from the smallest of the lanes' largest keys (which 64
// keys reach) to the largest; most often some key splits off exactly what is wanted long before the interval is empty.
template <int W>
__device__ __forceinline__ void select_take(const KvSelectProblem& p, const uint32_t* keys, int own, int me, int* meet,
                                            int& turn, int32_t* out) {
  constexpr int VPL = 32, STEP = 8;
  const int lane = threadIdx.x & 63, width = p.step.width, count = min(own + 1, width);
  const int tail = max(own + 1 - p.last, 0), head = min(p.first, count);      // listed always: below head, from tail on
  const int beyond = max(own + 1 - max(width, tail), 0);                       // of them behind the table
  const int room = p.top_k - beyond - head - max(count - max(tail, head), 0);
  uint32_t v[VPL];
#pragma unroll
  for (int s = 0; s < VPL / STEP; ++s) {
    if (64 * W * STEP * s < count) {
#pragma unroll
      for (int i = STEP * s; i < STEP * (s + 1); ++i) {
        const int j = 64 * (W * i + me) + lane;
        v[i] = j >= head && j < tail && j < count ? keys[j] : 0u;
      }
    } else {
#pragma unroll
      for (int i = STEP * s; i < STEP * (s + 1); ++i) v[i] = 0u;
    }
  }
  // over the waves: sums, smallest and largest values
  auto all_waves = [&](int x, auto&& join) {
    if (W == 1) return x;
    int* at = meet + (turn ^= W);      // two sets of W in turn, so that one barrier is enough
    if (lane == 0) at[me] = x;
    __syncthreads();
    int y = at[0];
#pragma unroll
    for (int w = 1; w < W; ++w) y = join(y, at[w]);
    return y;
  };
  auto at_least = [&](uint32_t x) {
    int n = 0;
#pragma unroll
    for (int s = 0; s < VPL / STEP; ++s)
      if (64 * W * STEP * s < count) {
#pragma unroll
        for (int i = STEP * s; i < STEP * (s + 1); ++i) n += __popcll(__ballot(v[i] >= x));
      }
    return all_waves(n, [](int a, int b) { return a + b; });
  };
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) most = max(most, v[i]);
  uint32_t lo = wave_min_u32(most), hi = wave_max_u32(most);
  lo = (uint32_t)all_waves((int)lo, [](int a, int b) { return (int)min((uint32_t)a, (uint32_t)b); });
  hi = (uint32_t)all_waves((int)hi, [](int a, int b) { return (int)max((uint32_t)a, (uint32_t)b); }) + 1;
  // count(lo) >= want > count(hi)
  int at_lo = 64 * W, above = 0;
  const bool short_list = lo == 0 || room > 64 * W;
  if (short_list) {
    lo = 1;
    at_lo = at_least(1);
  }
  const int want = min(room, at_lo);
  if (want <= 0) {
    lo = hi;
  } else if (!short_list || at_lo != want) {
    while (hi - lo > 1) {
      const uint32_t mid = lo + (hi - lo) / 2;
      const int n = at_least(mid);
      if (n >= want) lo = mid;
      else hi = mid, above = n;
      if (n == want) {
        above = want;
        break;
      }
    }
  } else {
    above = want;
  }
  // chosen: keys from lo + 1 on and the first of those equal to lo, or all from lo on
  const uint32_t sure = above == want ? lo : lo + 1;
  int ties = want - above, filled = 0;
  const uint64_t below = lane == 0 ? 0 : ~0ull >> (64 - lane);
  const int total = want + head + max(count - max(tail, head), 0);
  auto take = [&](uint32_t key, int j, int tied_before) {
    const bool tie = key != 0 && key < sure && key >= lo && want > 0;
    const uint64_t tied = __ballot(tie);
    (void)tied;
    return (j < count && (j < head || j >= tail)) || (key != 0 && key >= sure && want > 0) ||
           (tie && tied_before + __popcll(tied & below) < ties);
  };
  if (W == 1) {
#pragma unroll
    for (int s = 0; s < VPL / STEP; ++s) {
      if (64 * STEP * s < count) {
#pragma unroll
        for (int i = STEP * s; i < STEP * (s + 1); ++i) {
          const int j = 64 * i + lane;
          const uint64_t tied = __ballot(v[i] != 0 && v[i] < sure && v[i] >= lo);
          const bool chosen = take(v[i], j, 0);
          const uint64_t taken = __ballot(chosen);
          if (chosen) out[filled + __popcll(taken & below)] = j;
          filled += __popcll(taken);
          ties -= min(ties, (int)__popcll(tied));
        }
      }
    }
  } else {
    // 64 * W keys a round, in order of pages: the waves' counts meet before each writes
    for (int i = 0; i < VPL; ++i) {
      if (64 * W * i >= count) break;
      uint32_t key = 0;
#pragma unroll
      for (int k = 0; k < VPL; ++k) key = k == i ? v[k] : key;
      const int j = 64 * (W * i + me) + lane;
      const int mine = __popcll(__ballot(key != 0 && key < sure && key >= lo));
      int* at = meet + (turn ^= W);
      if (lane == 0) at[me] = mine;
      __syncthreads();
      int before = 0, all_ties = 0;
      for (int w = 0; w < W; ++w) {
        before += w < me ? at[w] : 0;
        all_ties += at[w];
      }
      const bool chosen = take(key, j, before);
      const uint64_t taken = __ballot(chosen);
      at = meet + (turn ^= W);
      if (lane == 0) at[me] = __popcll(taken);
      __syncthreads();
      int start = filled;
      for (int w = 0; w < W; ++w) {
        start += w < me ? at[w] : 0;
        filled += at[w];
      }
      if (chosen) out[start + __popcll(taken & below)] = j;
      ties -= min(ties, all_ties);
    }
  }
  // own pages behind the table are listed all the same: the attention makes such rows NaN
  for (int i = total + 64 * me + lane; i < p.top_k; i += 64 * W)
    out[i] = i - total < beyond ? own + 1 - beyond + (i - total) : -1;
}

template <int D, int HS, bool WIDE>
__global__ __launch_bounds__(WIDE || HS == kOne ? 1024 : 512) void kv_select_kernel(KvSelectProblem p, SelectShape sh) {
  constexpr int NW = WIDE || HS == kOne ? 16 : 8;
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ int meet[2 * NW];
  const KvStep& s = p.step;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), hkv = p.index.kv_heads;
  if (blockIdx.x >= sh.work_groups) {      // rows of no request
    const int before = s.R > 0 ? min(max(s.offsets[0], 0), s.T) : s.T;
    const int after = s.R > 0 ? min(max(s.offsets[s.R], before), s.T) : s.T;
    const int index = blockIdx.x - sh.work_groups, count = gridDim.x - sh.work_groups, row = hkv * p.top_k;
    for (int i = index; i < before + s.T - after; i += count)
      for (int k = tid; k < row; k += 64 * NW) p.selected[(size_t)(i < before ? i : i - before + after) * row + k] = -1;
    return;
  }
  const int h = blockIdx.x % hkv;
  StepRequest q;
  int item;
  if (!step_find(s, blockIdx.x / hkv, [&](const StepRequest& x) { return (x.n + sh.tokens - 1) / sh.tokens; }, &q, &item))
    return;
  const int tok0 = item * sh.tokens, toks = min(sh.tokens, q.n - tok0), pos0 = q.len - q.n + tok0;
  const int last = pos0 + toks - 1, pages = last < 0 ? 0 : min(last / s.page_size + 1, s.width);
  uint32_t* keys = reinterpret_cast<uint32_t*>(lds);
  float* tops = reinterpret_cast<float*>(keys + (size_t)sh.tokens * sh.stride);
  int8_t* codes = reinterpret_cast<int8_t*>(tops + 16 * sh.blocks * sh.groups);
  if (pages > 0) {
    select_rows<D, HS>(p, q, h, tok0, sh, codes, tops);
    __syncthreads();
    select_scores<D, HS, NW>(p, s.table + (size_t)q.r * s.width, h, pages, sh, codes, tops, keys);
    __syncthreads();
  }
  int turn = 0;
  for (int t = WIDE ? 0 : wave; t < toks; t += WIDE ? 1 : NW) {
    const int pos = pos0 + t;
    int32_t* out = p.selected + ((size_t)(q.row0 + tok0 + t) * hkv + h) * p.top_k;
    if (pos < 0) {
      for (int i = WIDE ? tid : tid & 63; i < p.top_k; i += WIDE ? 64 * NW : 64) out[i] = -1;
    } else {
      select_take<WIDE ? NW : 1>(p, keys + (size_t)t * sh.stride, pos / s.page_size, WIDE ? wave : 0, meet, turn, out);
    }
  }
}

// LDS of a workgroup, and what fits: a compute unit holds 160 KB, two workgroups of several tokens are wanted on it.
constexpr int kSelectLds = 150 << 10, kSelectHalf = 76 << 10;

size_t select_lds(const SelectShape& s, int32_t D) {
  return (size_t)s.tokens * s.stride * 4 + (size_t)16 * s.blocks * s.groups * (4 + D);
}

// One token per workgroup where the step may be of single tokens (T <= R); otherwise as many groups of tokens as leave
// 512 workgroups and fit, since all of them share what a workgroup reads of the index.
int select_heads(const KvSelectProblem& p, SelectShape* s) {
  const int64_t T = p.step.T, R = p.step.R;
  const int D = p.index.head_dim, hkv = p.index.kv_heads;
  s->stride = (p.step.width + 63) / 64 * 64 + 16;      // the 64 lanes' keys of four tokens lie in 64 banks
  if (T > R) {
    const int HS = p.G == 1 ? 1 : p.G == 2 ? 2 : 4;
    s->blocks = (p.G + 3) / 4;
    for (int groups = 4; groups >= 1; groups /= 2) {
      s->groups = groups;
      s->tokens = groups * group_tokens(HS);
      const bool fits = select_lds(*s, D) <= (groups > 1 ? kSelectHalf : kSelectLds);
      if (fits && (groups == 1 || T / s->tokens * hkv >= 512)) return HS;
    }
  }
  s->tokens = s->groups = 1;
  s->blocks = (p.G + 15) / 16;
  return kOne;
}

}  // namespace

int64_t kv_index_items(int32_t T, int32_t R, int32_t page_size) {
  const int64_t requests = std::min(T, R);
  return std::min((int64_t)T, T / page_size + 2 * requests);      // n rows lie in at most (n - 2) / page_size + 2 pages
}

moe_status_t launch_kv_index_update(const moe_nvfp4_kv_cache_t& c, const moe_nvfp4_kv_index_t& index, const KvStep& s,
                                    hipStream_t stream) {
  with_head_dim(c.head_dim, [&](auto tag) {
    hipLaunchKernelGGL(kv_index_kernel<decltype(tag)::value>,
                       dim3((unsigned)kv_index_items(s.T, s.R, s.page_size), c.kv_heads), dim3(256), 0, stream, c,
                       index.codes, index.scales, s);
  });
  return launch_status();
}

moe_status_t launch_kv_select(const KvSelectProblem& p, hipStream_t stream) {
  SelectShape s;
  const int HS = select_heads(p, &s);
  const int64_t T = p.step.T, R = p.step.R, fill = std::min((T + 3) / 4, (int64_t)256);
  const int64_t items = R == 0 ? 0 : std::min(T, T / s.tokens + std::min(T, R)) * p.index.kv_heads;
  s.work_groups = (uint32_t)items;
  const dim3 grid((unsigned)(items + fill));
  const size_t bytes = select_lds(s, p.index.head_dim);
  const bool wide = p.step.width > 2048;
  with_head_dim(p.index.head_dim, [&](auto tag) {
    constexpr int D = decltype(tag)::value;
    auto launch = [&](auto heads) {
      constexpr int H = decltype(heads)::value;
      if (wide)
        hipLaunchKernelGGL((kv_select_kernel<D, H, true>), grid, dim3(1024), bytes, stream, p, s);
      else
        hipLaunchKernelGGL((kv_select_kernel<D, H, false>), grid, dim3(H == kOne ? 1024 : 512), bytes, stream, p, s);
    };
    if (HS == kOne) launch(DimC<kOne>{});
    else if (HS == 1) launch(DimC<1>{});
    else if (HS == 2) launch(DimC<2>{});
    else launch(DimC<4>{});
  });
  return launch_status();
}

}  // namespace moe
