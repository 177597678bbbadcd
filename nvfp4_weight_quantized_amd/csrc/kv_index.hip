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

// Sums over the 16 lanes of a row, 16 numbers at once: number i meets in lane i of the row.  Each step pairs lanes and
// halves the numbers each holds, so that all of it takes 15 exchanges where 16 sums would take 64.
template <int CTRL, int BIT, int N>
__device__ __forceinline__ void meet_halves(int (&v)[16]) {
  const bool upper = (threadIdx.x >> BIT) & 1;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const int keep = upper ? v[i + N / 2] : v[i], give = upper ? v[i] : v[i + N / 2];
    v[i] = keep + dpp_i<CTRL>(give, give);
  }
}
__device__ __forceinline__ int row_sums(int (&v)[16]) {
  meet_halves<kDppRowMirror, 3, 16>(v);
  meet_halves<kDppRowHalfMirror, 2, 8>(v);
  meet_halves<kDppQuad2301, 1, 4>(v);
  meet_halves<kDppQuad1032, 0, 2>(v);
  return v[0];
}

// W waves per touched page and head take every W-th unit.  A lane holds one position (of 16) and the elements
// [8u, 8u + 8) of every 32, as the unit's 16-byte pieces give them.  Sums go from fp32 (three units: six positions of a
// lane, below 2^24 in units of 2^-10, so exact) to 32-bit integers over the 16 lanes (96 positions: below 2^29) and to
// 64 bits beyond.  46 MB of keys (3 prompts of up to 30011 positions, 8 heads of 128, pages of 96) in 14.3 us, 3.2 TB/s: a
// wave looks, loads, sums and stores once, and all of them do so together, so the memory idles while they sum.  The last
// pages of 64 requests in 4.3 us, a chain of loads.
template <int D, int W>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void kv_index_kernel(moe_nvfp4_kv_cache_t c,
                                                                         int8_t* __restrict__ codes,
                                                                         float* __restrict__ scales, KvStep s,
                                                                         int items) {
  using U = KvUnit<D>;
  constexpr int NS = D / 32, NL = NS / 2, kUnits = 3;
  const int tid = threadIdx.x, lane = tid & 63, u4 = lane >> 4, n16 = lane & 15, hkv = c.kv_heads;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), me = W == 1 ? 0 : wave;
  // heads of a page in neighbouring waves
  const int at = W == 1 ? 4 * blockIdx.x + wave : blockIdx.x, h = at % hkv;
  StepRequest q;
  int within;
  if (at >= items * hkv ||
      !step_find(s, at / hkv, [&](const StepRequest& x) { return touched_pages(s, x); }, &q, &within))
    return;
  const int b = first_page(s, q) + within, page = s.table[(size_t)q.r * s.width + b];
  if (page < 0 || page >= c.num_pages) return;
  const int held = min(c.page_size, q.len - b * c.page_size), units = (held + kKvUnit - 1) / kKvUnit;
  const uint8_t* first = c.pages + kv_unit_offset<D>(c, page * c.page_size, h);
  // sum[j]: element 32*k + 8*u4 + i, number 16*j + n16 = 8*k + i
  long long sum[NS / 2];
#pragma unroll
  for (int j = 0; j < NS / 2; ++j) sum[j] = 0;
  for (int u0 = me; u0 < units; u0 += kUnits * W) {
    float acc[NS][8];
#pragma unroll
    for (int k = 0; k < NS; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[k][e] = 0.f;
    // all units' loads first
    uint32_t w[kUnits][2 * NS], sc[kUnits][NS / 2];
#pragma unroll
    for (int x = 0; x < kUnits; ++x) {
      if (u0 + x * W >= units) break;
      const uint8_t* unit = first + (size_t)(u0 + x * W) * U::kBytes;
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const uint4 y = *reinterpret_cast<const uint4*>(unit + 1024 * j + 16 * lane);
        w[x][4 * j] = y.x, w[x][4 * j + 1] = y.y, w[x][4 * j + 2] = y.z, w[x][4 * j + 3] = y.w;
      }
#pragma unroll
      for (int j = 0; j < NS / 2; ++j)
        sc[x][j] = *reinterpret_cast<const uint32_t*>(unit + U::kKScales + (16 * (u4 >> 1) + n16) * 2 * NS + 4 * j);
    }
#pragma unroll
    for (int x = 0; x < kUnits; ++x) {
      const int u = u0 + x * W;
      if (u >= units) break;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const bool seen = kKvUnit * u + 16 * half + n16 < held;
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          const int word = half * NS + k, byte = word & 3;
          const int bits = (int)sc[x][word >> 2];
          const float f8 = byte == 0   ? __builtin_amdgcn_cvt_f32_fp8(bits, 0)
                           : byte == 1 ? __builtin_amdgcn_cvt_f32_fp8(bits, 1)
                           : byte == 2 ? __builtin_amdgcn_cvt_f32_fp8(bits, 2)
                                       : __builtin_amdgcn_cvt_f32_fp8(bits, 3);
          const float f = seen ? 1024.f * f8 : 0.f;
          const f32x2 e[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[x][word], 1.0f, 0),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[x][word], 1.0f, 1),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[x][word], 1.0f, 2),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[x][word], 1.0f, 3)};
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[k][i] = __fmaf_rn(e[i >> 1][i & 1], f, acc[k][i]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NS / 2; ++j) {
      int v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = (int)acc[2 * j + (i >> 3)][i & 7];
      sum[j] += row_sums(v);
    }
  }
  if (W > 1) {
    __shared__ long long sums[W][NS / 2][64];
#pragma unroll
    for (int j = 0; j < NS / 2; ++j) sums[wave][j][lane] = sum[j];
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int j = 0; j < NS / 2; ++j)
      for (int w = 1; w < W; ++w) sum[j] += sums[w][j][lane];
  }
  long long top = 0;
#pragma unroll
  for (int j = 0; j < NS / 2; ++j) top = max(top, sum[j] < 0 ? -sum[j] : sum[j]);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = max(top, (long long)__shfl_xor(top, off));
  const size_t out = (size_t)page * hkv + h;
  // in 64 bits: a quotient half way between two whole numbers is exact, others are further from it than their rounding
#pragma unroll
  for (int j = 0; j < NS / 2; ++j) {
    const int d = 32 * (2 * j + (n16 >> 3)) + 8 * u4 + (n16 & 7);
    codes[out * D + d] = top > 0 ? (int8_t)(int)rint(127.0 * (double)sum[j] / (double)top) : (int8_t)0;
  }
  if (lane == 0) scales[out] = (float)((double)top / (130048.0 * held));
}

// ------------------------------------------------------------------------------------ choice
// A workgroup takes some tokens of a request and one kv head: their rows in 8 bits into LDS as matrix operands, the
// products of all of them with 16 pages at a time on the matrix unit (the rows are the first operand, so a lane holds one
// page's products with four rows), a key per token and page (its score as an ordered integer) into LDS, and then a wave
// per token takes the top_k largest keys.  Chunks of 1024 and 748 rows, 32/8 heads of 128, on 44726 and 60000 positions of
// pages of 64, top 32, 40 us, the vector unit 50% busy (the choice), the matrix unit 5%: a wave's choice is one chain of
// ballots and counts.  One row of 32/4 heads on 131072 positions, top 64, 12.6 us on four compute units, of which the
// products of its 2048 pages are 4 and the choice 3; 64 rows of requests of their own on up to 16000, 32/8 heads, 12.7 us.
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

// Bits that stand for no scale (a NaN that no computation gives).
constexpr uint32_t kBadPage = 0xFFFFDEADu;

// Largest value of the lanes 16 and 32 apart.
__device__ __forceinline__ float quarters_max(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// 16 pages' codes in LDS, a line of D bytes each.  Piece x (16 bytes) of page n lies at piece x ^ fold(n): the lanes that
// read the same piece of 16 pages then find it in 16 different sets of four banks.
template <int D>
__device__ __forceinline__ int page_piece(int n, int x) {
  return n * D + 16 * (x ^ ((n / (256 / D)) & (D / 16 - 1)));
}

// Keys of the pages [0, pages) for the workgroup's tokens: keys[token * stride + page], 0 for a page that is not in the
// cache.  A wave takes 64 pages at a time, a lane's page of the table and its scale first, then the codes 16 pages at a
// time straight to LDS, into a place of its own in `stage`: neighbouring lanes ask for pieces of one
// page, where as operands they would each touch another page's line, and the address unit looks up one line a cycle
// (one row on 2048 pages: 11 us of products in that form).
// rows() makes the operands of the rows while the first pages are on their way.
template <int D, int HS, int NW, typename Rows>
__device__ __forceinline__ void select_scores(const KvSelectProblem& p, const int32_t* __restrict__ table, int h,
                                              int pages, const SelectShape& sh, const int8_t* codes, const float* tops,
                                              uint32_t* keys, uint8_t* stage, Rows&& rows) {
  constexpr int KS = D / 64, TPL = HS == kOne ? 1 : 4 / HS;      // tokens of a lane
  constexpr int LPP = D / 16, PPL = 64 / LPP, LOADS = 16 / PPL;  // lanes per page, pages per load, loads per chunk
  using lds_bytes = __attribute__((address_space(3))) uint8_t*;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q4 = lane >> 4, n16 = lane & 15, hkv = p.index.kv_heads;
  const lds_bytes mine = (lds_bytes)stage + wave * 16 * D;
  struct Batch {
    int page;         // of this lane; 0 where it is not in the cache
    uint32_t scale;   // its bits, kBadPage there
  };
  auto load_batch = [&](int j0) {
    Batch x{0, kBadPage};
    if (j0 + lane < pages) {
      const int page = table[j0 + lane];
      if (page >= 0 && page < p.index.num_pages)
        x = Batch{page, __float_as_uint(p.index.scales[(size_t)page * hkv + h])};
    }
    return x;
  };
  const uint8_t* from[LOADS];      // of page 0
#pragma unroll
  for (int t = 0; t < LOADS; ++t) {
    const int n = t * PPL + lane / LPP;
    from[t] = reinterpret_cast<const uint8_t*>(p.index.codes) + (size_t)h * D +
              16 * ((lane % LPP) ^ ((n / (256 / D)) & (LPP - 1)));
  }
  const uint32_t page_bytes = hkv * D;
  // chunk x of a batch
  auto issue = [&](const Batch& b, int x) {
    const uint32_t dst = (uint32_t)(uintptr_t)mine;
#pragma unroll
    for (int t = 0; t < LOADS; ++t)
      direct_load16_from(from[t] + (uint64_t)(uint32_t)__shfl(b.page, 16 * x + t * PPL + lane / LPP) * page_bytes,
                         dst + 1024 * t);
  };
  // 1 .. 0xFFFFFFFE
  auto key_of = [&](float best, uint32_t scale) {
    return scale != kBadPage ? min(max(order_key(best * __uint_as_float(scale)), 1u), 0xFFFFFFFEu) : 0u;
  };
  const int first = 64 * wave, step = 64 * NW;
  Batch now = load_batch(first), next = now;
  if (first < pages) issue(now, 0);
  rows();
  __syncthreads();
  for (int j0 = first; j0 < pages; j0 += step, now = next) {
    const bool more = j0 + step < pages;
    if (more) next = load_batch(j0 + step);
    float score = 0.f;      // one token: of page j0 + lane
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
      i32x4 b[KS];
#pragma unroll
      for (int k = 0; k < KS; ++k)
        b[k] = *reinterpret_cast<const __attribute__((address_space(3))) i32x4*>(mine + page_piece<D>(n16, 4 * k + q4));
      asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");      // the chunk has been read
      if (x < 3) issue(now, x + 1);
      else if (more) issue(next, 0);
      const int j = j0 + 16 * x + n16;
      const uint32_t scale = HS == kOne ? 0u : __shfl(now.scale, 16 * x + n16);
      for (int grp = 0; grp < sh.groups; ++grp) {
        float best[TPL];
#pragma unroll
        for (int y = 0; y < TPL; ++y) best[y] = -INFINITY;
        for (int blk = 0; blk < sh.blocks; ++blk) {
          const int8_t* a = codes + (size_t)(grp * sh.blocks + blk) * KS * 1024 + 16 * lane;
          const float4 top = *reinterpret_cast<const float4*>(tops + 16 * (grp * sh.blocks + blk) + 4 * q4);
          i32x4 dot = {0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < KS; ++k)
            dot = __builtin_amdgcn_mfma_i32_16x16x64_i8(*reinterpret_cast<const i32x4*>(a + 1024 * k), b[k], dot, 0, 0, 0);
          const float s[4] = {(float)dot[0] * top.x, (float)dot[1] * top.y, (float)dot[2] * top.z, (float)dot[3] * top.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) best[e * TPL / 4] = fmaxf(best[e * TPL / 4], s[e]);
        }
        if (HS == kOne) {
          const float v = quarters_max(best[0]);
          score = q4 == x ? v : score;
        } else {
#pragma unroll
          for (int y = 0; y < TPL; ++y) {
            const int t = grp * (16 / (HS == kOne ? 1 : HS)) + q4 * TPL + y;
            if (j < sh.stride) keys[(size_t)t * sh.stride + j] = key_of(best[y], scale);
          }
        }
      }
    }
    if (HS == kOne && j0 + lane < sh.stride) keys[j0 + lane] = key_of(score, now.scale);
  }
}

// The threshold of the `want` largest of some keys, count(lo) >= want > 0 keys from lo on and none from hi on: afterwards
// count(lo) >= want > count(lo + 1), or *above == want and exactly `want` lie from lo on, which most often happens long
// before the interval has been halved 32 times.
template <typename Count>
__device__ __forceinline__ void halve(uint32_t* lo, uint32_t hi, int want, int* above, Count&& at_least) {
  *above = 0;
  while (hi - *lo > 1) {
    const uint32_t mid = *lo + (hi - *lo) / 2;
    const int n = at_least(mid);
    if (n >= want) *lo = mid;
    else hi = mid;
    if (n <= want) *above = n;
    if (n == want) return;
  }
}

// The pages of one token, chosen by one wave: those listed always, and the `room` largest keys of the others.
// The keys are dealt into 64 sets, one per lane (256 of many pages or for room > 64, 1024 of many for more), whose room-th
// largest maximum bounds the threshold from below: it leaves little more than `room` candidates (44 for 32 of many, 177 for
// 128), found by halving over 1, 4 or 16 maxima per lane.  Their pages go to a list of `cap` places, in order, over which the threshold itself is found; where they are
// more (many equal keys, most of the pages wanted), and where there are few pages, over all keys.  HELD: up to so many pages
// the keys stay in registers (0: each pass reads them).  One token: 2048 (2048 pages, a row of 32/4 heads, top 64: 12.6
// against 15.0 us); several: 1024, since 2048 cost a compute unit the third workgroup (chunks of 1024 and 748 rows on
// 44726 and 60000 positions, 32/8 heads, top 32: 40.2 against 46.9 us).
constexpr int kSelectWaves = 16, kManyWaves = 8;      // of a workgroup: one token, several tokens
constexpr int held_pages(int HS) { return HS == kOne ? 2048 : 1024; }

template <int HELD>
__device__ __forceinline__ void select_take(const KvSelectProblem& p, const uint32_t* keys, int own, uint16_t* list,
                                            int cap, int32_t* out) {
  constexpr bool REGS = HELD > 0;
  constexpr int VPL = REGS ? HELD / 64 : 8, STEP = 4, SETS = REGS ? 4 : 16, FEW = 4;
  const int lane = threadIdx.x & 63, width = p.step.width, count = min(own + 1, width);
  const uint64_t below = lane == 0 ? 0 : ~0ull >> (64 - lane);
  const int head = min(p.first, count), tail = min(max(own + 1 - p.last, head), count);      // [head, tail) by score
  const int beyond = max(own + 1 - max(width, max(own + 1 - p.last, 0)), 0);      // listed always, behind the table
  const int room = p.top_k - beyond - head - (count - tail);
  auto key_at = [&](int j) { return j >= head && j < tail ? keys[j] : 0u; };
  uint32_t v[VPL];
  auto load = [&](int j0) {
#pragma unroll
    for (int s = 0; s < VPL; s += STEP) {
      if (j0 + 64 * s < count) {
#pragma unroll
        for (int i = s; i < s + STEP; ++i) v[i] = key_at(j0 + 64 * i + lane);
      } else {
#pragma unroll
        for (int i = s; i < s + STEP; ++i) v[i] = 0u;
      }
    }
  };
  // f(number of the key in its lane, key, page) for every key
  auto each = [&](auto&& f) {
    for (int j0 = 0; j0 < (REGS ? 1 : count); j0 += 64 * VPL) {
      if (!REGS) load(j0);
#pragma unroll
      for (int s = 0; s < VPL; s += STEP)
        if (j0 + 64 * s < count) {
#pragma unroll
          for (int i = s; i < s + STEP; ++i) f(i, v[i], j0 + 64 * i + lane);
        }
    }
  };
  auto at_least = [&](uint32_t x) {
    int n = 0;
    each([&](int, uint32_t key, int) { n += __popcll(__ballot(key >= x)); });
    return n;
  };
  if (REGS) load(0);
  uint32_t most[SETS], top = 0;
#pragma unroll
  for (int i = 0; i < SETS; ++i) most[i] = 0;
  if (REGS) {
    each([&](int i, uint32_t key, int) { most[i % SETS] = max(most[i % SETS], key); });
  } else {
    for (int j0 = 0; j0 < count; j0 += 64 * SETS)
#pragma unroll
      for (int i = 0; i < SETS; ++i) most[i] = max(most[i], key_at(j0 + 64 * i + lane));
  }
  const bool few = room <= 32 * FEW;
  if (few) {
#pragma unroll
    for (int i = FEW; i < SETS; ++i) most[i % FEW] = max(most[i % FEW], most[i]);
  }
#pragma unroll
  for (int i = 0; i < SETS; ++i) top = max(top, most[i]);
  uint32_t lo = 1;
  const uint32_t hi = wave_max_u32(top) + 1;
  int above = 0;
  auto sets = [&](uint32_t x) {
    if (REGS && room <= 64) return (int)__popcll(__ballot(top >= x));
    int n = 0;
#pragma unroll
    for (int i = 0; i < FEW; ++i) n += __popcll(__ballot(most[i] >= x));
    if (!few) {
#pragma unroll
      for (int i = FEW; i < SETS; ++i) n += __popcll(__ballot(most[i] >= x));
    }
    return n;
  };
  const bool bounded = room > 0 && (few || !REGS) && sets(1) >= room, list_them = bounded && count > 256;
  if (bounded) halve(&lo, hi, room, &above, sets);
  int found = 0;      // candidates; all keys where there is no bound
  if (list_them) {
    each([&](int, uint32_t key, int j) {
      const bool in = key >= lo;
      const uint64_t all = __ballot(in);
      const int at = found + __popcll(all & below);
      if (in && at < cap) list[at] = (uint16_t)j;
      found += __popcll(all);
    });
  } else {
    found = at_least(lo);
  }
  const int want = max(min(room, found), 0);      // found >= room, or lo = 1 and these are all
  const bool listed = list_them && found <= min(cap, 256);
  uint32_t u[4];
  int page[4];
  above = found;
  if (listed) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = 64 * i + lane < found;
      page[i] = in ? list[64 * i + lane] : 0;
      u[i] = in ? keys[page[i]] : 0u;
    }
    if (found > want)
      halve(&lo, hi, want, &above, [&](uint32_t x) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) n += __popcll(__ballot(u[i] >= x));
        return n;
      });
  } else if (list_them && !REGS && found <= cap) {
    if (found > want)
      halve(&lo, hi, want, &above, [&](uint32_t x) {
        int n = 0;
        for (int i = lane; i - lane < found; i += 64) n += __popcll(__ballot(i < found && keys[list[min(i, found - 1)]] >= x));
        return n;
      });
  } else if (want > 0 && found > want) {
    halve(&lo, hi, want, &above, at_least);
  }
  // chosen: keys from `sure` on, and the first `ties` of those equal to lo
  int ties = want - above, filled = head;
  const uint32_t sure = ties > 0 ? lo + 1 : lo;
  auto write = [&](uint32_t key, int j) {
    const bool tie = key == lo && ties > 0;
    const uint64_t tied = __ballot(tie);
    const bool chosen = (key != 0 && key >= sure) || (tie && __popcll(tied & below) < ties);
    const uint64_t taken = __ballot(chosen);
    if (chosen) out[filled + __popcll(taken & below)] = j;
    filled += __popcll(taken);
    ties -= min(ties, (int)__popcll(tied));
  };
  if (listed) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (64 * i < found) write(u[i], page[i]);
  } else if (want > 0) {
    each([&](int, uint32_t key, int j) { write(key, j); });
  }
  // own pages behind the table are listed all the same: the attention makes such rows NaN
  for (int i = lane; i < head; i += 64) out[i] = i;
  const int end = head + want + count - tail;
  for (int i = head + want + lane; i < p.top_k; i += 64)
    out[i] = i < end ? tail + (i - head - want) : i - end < beyond ? own + 1 - beyond + (i - end) : -1;
}

template <int D, int HS, bool REGS>
__global__ __launch_bounds__(64 * (HS == kOne ? kSelectWaves : kManyWaves)) void kv_select_kernel(KvSelectProblem p,
                                                                                                  SelectShape sh) {
  constexpr int NW = HS == kOne ? kSelectWaves : kManyWaves;
  extern __shared__ __align__(16) uint8_t lds[];
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
  uint8_t* stage = reinterpret_cast<uint8_t*>(codes + (size_t)16 * sh.blocks * sh.groups * D);
  if (pages > 0) {
    select_scores<D, HS, NW>(p, s.table + (size_t)q.r * s.width, h, pages, sh, codes, tops, keys, stage,
                             [&]() { select_rows<D, HS>(p, q, h, tok0, sh, codes, tops); });
    __syncthreads();
  }
  // the lists lie where the pages' codes came in: a wave's own place, or all of them for one token
  uint16_t* list = reinterpret_cast<uint16_t*>(stage + wave * 16 * D);
  for (int t = wave; t < toks; t += NW) {
    const int pos = pos0 + t;
    int32_t* out = p.selected + ((size_t)(q.row0 + tok0 + t) * hkv + h) * p.top_k;
    if (pos < 0) {
      for (int i = tid & 63; i < p.top_k; i += 64) out[i] = -1;
    } else {
      select_take<REGS ? held_pages(HS) : 0>(p, keys + (size_t)t * sh.stride, pos / s.page_size, list, HS == kOne ? NW * 8 * D : 8 * D, out);
    }
  }
}

// LDS of a workgroup, and what fits: a compute unit holds 160 KB, three workgroups of several groups of tokens are wanted
// on it (chunks of 1024 and 748 rows on 44726 and 60000 positions, 32/8 heads of 128, top 32: 40.2 us; with LDS for two
// 48.1).
constexpr int kSelectLds = 150 << 10, kSelectThird = 52 << 10;

size_t select_lds(const SelectShape& s, int32_t D, int waves) {
  return (size_t)s.tokens * s.stride * 4 + (size_t)16 * s.blocks * s.groups * (4 + D) +
         (size_t)waves * 16 * D;
}

// One token per workgroup where the step may be of single tokens (T <= R); otherwise as many groups of tokens as leave
// 512 workgroups and fit, since all of them share what a workgroup reads of the index.  The chunks above take two groups,
// 40.2 us (one 51.3, a token per workgroup 218); 64 rows on 16000 positions one, 8.5 us (four 14.8, a token each 11.7).
// The host knows the table's width, not the lengths, and makes room for keys of all its columns: the same chunks take 40
// us up to 960 columns, 62 from 1025 on (the keys leave the registers, four tokens a workgroup), 144 at 4096 and 8192 (one
// workgroup per compute unit) and 470 at 16384 (a token per workgroup); 64 single tokens 12.7 us up to 2048, 16.7 at 16384.
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
      const bool fits = select_lds(*s, D, kManyWaves) <= (groups > 1 ? kSelectThird : kSelectLds);
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

// A wave per page and head where it has at most three units, which it sums in one go, else four.  Other side in brackets:
// the prompts of kv_index_kernel with pages of 32 21.5 [39.4] us, of 96 14.3 [20.6], of 128 18.4 [14.2], of 256 14.1 [14.2];
// the last pages of 64 requests, of 64 4.3 [4.6], of 128 4.7 [5.2], of 256 5.3 [7.1].
moe_status_t launch_kv_index_update(const moe_nvfp4_kv_cache_t& c, const moe_nvfp4_kv_index_t& index, const KvStep& s,
                                    hipStream_t stream) {
  const int64_t items = kv_index_items(s.T, s.R, s.page_size);
  with_head_dim(c.head_dim, [&](auto tag) {
    constexpr int D = decltype(tag)::value;
    if (c.page_size <= 3 * kKvUnit)
      hipLaunchKernelGGL((kv_index_kernel<D, 1>), dim3((unsigned)((items * c.kv_heads + 3) / 4)), dim3(256), 0, stream, c,
                         index.codes, index.scales, s, (int)items);
    else
      hipLaunchKernelGGL((kv_index_kernel<D, 4>), dim3((unsigned)(items * c.kv_heads)), dim3(256), 0, stream, c,
                         index.codes, index.scales, s, (int)items);
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
  const size_t bytes = select_lds(s, p.index.head_dim, HS == kOne ? kSelectWaves : kManyWaves);
  with_head_dim(p.index.head_dim, [&](auto tag) {
    constexpr int D = decltype(tag)::value;
    auto launch = [&](auto heads) {
      constexpr int H = decltype(heads)::value;
      const dim3 block(64 * (H == kOne ? kSelectWaves : kManyWaves));
      if (p.step.width <= held_pages(H)) hipLaunchKernelGGL((kv_select_kernel<D, H, true>), grid, block, bytes, stream, p, s);
      else hipLaunchKernelGGL((kv_select_kernel<D, H, false>), grid, block, bytes, stream, p, s);
    };
    if (HS == kOne) launch(DimC<kOne>{});
    else if (HS == 1) launch(DimC<1>{});
    else if (HS == 2) launch(DimC<2>{});
    else launch(DimC<4>{});
  });
  return launch_status();
}

}  // namespace moe
