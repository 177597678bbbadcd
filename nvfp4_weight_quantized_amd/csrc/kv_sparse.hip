// Attention of query rows over the pages chosen for them (kv_select), from the paged NVFP4 key/value cache.
//
// The mathematics, the operands and the softmax reference are those of kv_attention.hip: scores, maxima, sums and
// outputs in fp32, keys and values exact in fp16, p rounded to fp16 for the value product.  What differs is which
// units a row sees: those of the pages in its token's list for its kv head, up to its own position.
#include "kv_operands.h"
#include "kv_step.h"

namespace moe {
namespace {

// ------------------------------------------------------------------------------------ tiles
// A workgroup takes a tile: the rows of one kv head of up to `tokens` consecutive tokens of a request, 16 * MI rows at
// most (a token with more rows than that is cut into `parts`).  It goes through the union of its tokens' lists, a page
// once for all of them, with a bit per token that says whose list holds the page: a unit's codes are turned into
// operands once, which is most of the work, and the rows that do not see it are masked.  Where lists have nothing in
// common this costs what tiles of one token would, since the columns of the matrix products would lie idle there.
// Each of the NW waves takes every NW-th unit through an LDS ring of its own; their sums meet in LDS at the end.
// Few tiles with long lists are cut into splits of their units, whose partial sums a second launch joins.
struct SparseTiles {
  int tokens;      // per tile
  int parts;       // tiles per token (tokens == 1)
  int splits;      // of a tile's units
  uint32_t page_units;      // 2^32 / units of a page, rounded up (0: one unit)
  int bm;          // rows of a tile
  float* o;        // partial sums [tile][split][bm][D], unnormalised
  float* ml;       // [tile][split][2][bm]: reference maximum, sum
};

// Bound by memory where each page is read by one tile: 64 requests on up to 16000 positions, 64/8 heads of dimension 128, 48
// pages of 64 each (210 MB) 42.3 us, 5.0 TB/s, the rate of a copy, with loads that pass the caches by.  Where tokens have
// lists of their own no unit is full: chunks of 1024 and 748 rows on 26185 and 30000 positions, 32/8 heads, 24 pages each,
// 198 us, the vector unit 67% busy with about 360 instructions per unit (172 of them turn codes into operands) beside 32
// matrix instructions, the matrix unit 23%.

constexpr int kEntries = kKvMaxSelected;      // of a tile's lists

// The tile `index` (over requests, tokens and parts) of the step: its request, first token and part.
__device__ __forceinline__ bool sparse_find(const KvAttentionProblem& a, const SparseTiles& tiles, int index,
                                            StepRequest* rq, int* tok0, int* part) {
  const KvStep s{a.offsets, a.lens, a.table, a.R, a.T, a.width, a.cache.page_size};
  int item;
  if (!step_find(s, index, [&](const StepRequest& x) { return (x.n + tiles.tokens - 1) / tiles.tokens * tiles.parts; },
                 rq, &item))
    return false;
  *part = item % tiles.parts;
  *tok0 = item / tiles.parts * tiles.tokens;
  return true;
}

template <int D, int MI, int NW>
__global__ __launch_bounds__(64 * NW, (D == 256 && MI == 2 ? 1 : 2)) void kv_sparse_kernel(KvSparseProblem p,
                                                                                               SparseTiles tiles) {
  using U = KvUnit<D>;
  constexpr int NS = D / 32, BM = 16 * MI, NL = NS / 2;
  constexpr int kFull = U::kBytes / 1024, kTail = U::kBytes % 1024 / 256;   // 1024- and 256-byte loads of a unit
  constexpr int kOut = NW * BM * 36 * 4, kRings = NW * kRing * U::kBytes;
  // the lists; then the waves' rings; at the end one 32-element range of the sums (rows padded to 36 floats)
  __shared__ __align__(16) uint8_t lds[kOut > kRings ? kOut : kRings];
  static_assert(sizeof(lds) >= 4 * kEntries, "the lists lie where the rings will");
  __shared__ float m_lds[NW][BM], l_lds[NW][BM];
  // logical page and page of the cache (-1: bad) of each entry, then the tokens that list it
  extern __shared__ __align__(16) int entry[];
  __shared__ int chunk_count[kEntries / 64];
  const KvAttentionProblem& a = p.a;
  if (blockIdx.x >= a.work_groups) return kv_fill_rows<D>(a, blockIdx.x - a.work_groups, gridDim.x - a.work_groups);
  using lds_bytes = __attribute__((address_space(3))) uint8_t*;
  float(*o_lds)[BM][36] = reinterpret_cast<float(*)[BM][36]>(lds);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q4 = lane >> 4, n16 = lane & 15;
  const int hkv = a.cache.kv_heads, ps = a.cache.page_size, upp = ps / kKvUnit;
  const int h = blockIdx.x % hkv, split = blockIdx.x / hkv % tiles.splits, tile = blockIdx.x / hkv / tiles.splits;
  StepRequest rq;
  int tok0, part;
  if (!sparse_find(a, tiles, tile, &rq, &tok0, &part)) return;
  const int toks = min(tiles.tokens, rq.n - tok0), g0 = part * BM, most = tiles.tokens * p.top_k;
  int* const entry_page = entry;
  int* const entry_phys = entry + most;
  uint16_t* const entry_mask = reinterpret_cast<uint16_t*>(entry + 2 * most);
  const int rows = tiles.parts > 1 ? min(BM, a.G - g0) : toks * a.G;
  const int pos0 = rq.len - rq.n + tok0, pos_last = pos0 + toks - 1;      // positions of the first and last token

  // the query rows, asked for first: row n16 of block mi, elements [32s + 8*q4, +8)
  u32x4 raw[MI][NS];
  int pos[MI], bit[MI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    const int row = 16 * mi + n16;
    const bool valid = row < rows;
    const int t = valid && tiles.parts == 1 ? row / a.G : 0, g = valid ? g0 + row - t * a.G : 0;
    pos[mi] = valid ? pos0 + t : -1;
    bit[mi] = t;
    const uint16_t* src = a.q + (int64_t)(rq.row0 + tok0 + t) * a.q_stride + (size_t)(h * a.G + g) * D + 8 * q4;
#pragma unroll
    for (int k = 0; k < NS; ++k) raw[mi][k] = *reinterpret_cast<const u32x4*>(src + 32 * k);
  }

  // ---- the union of the lists
  int entries = 0;
  {
    uint32_t* lists = reinterpret_cast<uint32_t*>(lds);
    const int K = p.top_k, all = toks * K;
    const int32_t* src = p.selected + ((size_t)(rq.row0 + tok0) * hkv + h) * K;
    for (int i = tid; i < all; i += 64 * NW) {
      const int t = i / K;
      lists[i] = (uint32_t)src[(size_t)t * hkv * K + (i - t * K)];
    }
    __syncthreads();
    const int32_t* table = a.table + (size_t)rq.r * a.width;
    // a lane per entry of the lists: whether it opens one of the union, which no earlier token's list does, and the tokens
    // whose lists hold the page
    constexpr int kChunks = kEntries / 64 / NW;
    int page_of[kChunks], phys_of[kChunks];
    uint32_t mask_of[kChunks];
    uint64_t opens[kChunks];
#pragma unroll
    for (int x = 0; x < kChunks; ++x) {
      const int c = wave + NW * x, i = 64 * c + lane;
      opens[x] = 0;
      if (64 * c >= all) break;
      bool open = false;
      if (i < all) {
        const int t = i / K, k = i - t * K;
        const uint32_t b = lists[i];
        uint32_t mask = 1u << t;
        open = (int)b >= 0 && (long long)b * ps <= pos0 + t && (k == 0 || lists[i - 1] != b);
        const int page = open && (int)b < a.width ? table[b] : -1;
        for (int o = 0; o < toks; ++o) {
          if (o == t) continue;
          int lo = 0, hi = K;      // the first element of list o not below b
          while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (lists[o * K + mid] < b) lo = mid + 1;
            else hi = mid;
          }
          // a token that lists a page ahead of its own position does not see it
          if (lo < K && lists[o * K + lo] == b && (long long)b * ps <= pos0 + o) {
            mask |= 1u << o;
            open &= o > t;
          }
        }
        page_of[x] = (int)b;
        phys_of[x] = page >= 0 && page < a.cache.num_pages ? page : -1;
        mask_of[x] = mask;
      }
      opens[x] = __ballot(open);
      if (lane == 0) chunk_count[c] = __popcll(opens[x]);
    }
    __syncthreads();
    const int chunks = (all + 63) / 64;
    const int mine = lane < chunks ? chunk_count[lane] : 0, before = wave_inclusive_scan(mine) - mine;      // chunks <= 16
    entries = __builtin_amdgcn_readlane(before + mine, 63);
#pragma unroll
    for (int x = 0; x < kChunks; ++x) {
      const int c = wave + NW * x;
      if (64 * c >= all) break;
      if ((opens[x] >> lane) & 1) {
        const uint64_t below = lane == 0 ? 0 : ~0ull >> (64 - lane);
        const int at = __builtin_amdgcn_readlane(before, c) + __popcll(opens[x] & below);
        entry_page[at] = page_of[x];
        entry_phys[at] = phys_of[x];
        entry_mask[at] = (uint16_t)mask_of[x];
      }
    }
    __syncthreads();      // the lists have been read
  }
  // this split's units of the union, a whole number of rounds of the waves
  const int all_units = entries * upp, per = ((all_units + tiles.splits - 1) / tiles.splits + NW - 1) / NW * NW;
  const int u0 = min(split * per, all_units), units = min(all_units - u0, per);
  const int mine = units > wave ? (units - wave + NW - 1) / NW : 0;
  const lds_bytes ring = (lds_bytes)lds + wave * kRing * U::kBytes;

  // unit u of the union is in entry u / upp, exactly for u < 2^32 / upp
  auto entry_of = [&](int u) { return tiles.page_units ? (int)__umulhi((uint32_t)u, tiles.page_units) : u; };
  // the wave's unit i is unit u0 + wave + NW * i of the union
  auto issue = [&](int i, int slot) {
    const int u = u0 + wave + NW * i, e = entry_of(u), page = __builtin_amdgcn_readfirstlane(entry_phys[e]);
    const uint8_t* base = a.cache.pages;
    if (page >= 0) base += (((uint64_t)page * hkv + h) * upp + (u - e * upp)) * (uint64_t)U::kBytes;
    const uint32_t dst = (uint32_t)(uintptr_t)ring + slot * U::kBytes;
#pragma unroll
    for (int j = 0; j < kFull; ++j) {
      if (NW > 4) direct_load16_nt(base + 1024 * j, 16 * lane, dst + 1024 * j);
      else direct_load16(base + 1024 * j, 16 * lane, dst + 1024 * j);
    }
#pragma unroll
    for (int j = 0; j < kTail; ++j) {
      if (NW > 4) direct_load4_nt(base + 1024 * kFull + 256 * j, 4 * lane, dst + 1024 * kFull + 256 * j);
      else direct_load4(base + 1024 * kFull + 256 * j, 4 * lane, dst + 1024 * kFull + 256 * j);
    }
  };
  for (int i = 0; i < min(mine, kRing); ++i) issue(i, i);

  // query operands
  f16x8 qf[MI][NS];
  float c[MI];
  bool rare = false;      // a row of the wave has a far reference, or a query with an infinity or NaN
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    const auto& w = raw[mi];
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < NS; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, max(w[k][j] & 0x7FFFu, (w[k][j] >> 16) & 0x7FFFu));
    int e = (int)(top >> 7);    // the row's largest exponent field
    e = max(e, __shfl_xor(e, 16));
    e = max(e, __shfl_xor(e, 32));
    rare |= __any(e == 255);
    const int shift = row_shift(e, a.scale * kLog2e);
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      const f16x2 p0 = bf16x2_to_f16(w[k][0], shift), p1 = bf16x2_to_f16(w[k][1], shift);
      const f16x2 p2 = bf16x2_to_f16(w[k][2], shift), p3 = bf16x2_to_f16(w[k][3], shift);
      qf[mi][k] = f16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
    }
    c[mi] = fminf(ldexpf(a.scale * kLog2e, -shift), FLT_MAX);      // a score of 0 stays 0
  }

  f32x4 o[MI][NS][2];
  float m[MI], l[MI];
  bool far[MI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    far[mi] = false;
    m[mi] = kNone;
    l[mi] = 0.f;
#pragma unroll
    for (int r = 0; r < NS; ++r) o[mi][r][0] = o[mi][r][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  auto compute = [&](int i, int slot) {
    const int u = u0 + wave + NW * i, e = entry_of(u);
    const int key0 = __builtin_amdgcn_readfirstlane(entry_page[e]) * ps + (u - e * upp) * kKvUnit;
    if (key0 > pos_last) return;
    const int mask = __builtin_amdgcn_readfirstlane((int)entry_mask[e]);
    const bool bad = __builtin_amdgcn_readfirstlane(entry_phys[e]) < 0;
    const lds_bytes unit_lds = ring + slot * U::kBytes;
    u32x4 kc[NL];
    uint32_t ks[NS / 2];      // 2*NS scale bytes: word w = block*NS + step
#pragma unroll
    for (int j = 0; j < NL; ++j)
      kc[j] = *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(unit_lds + 1024 * j + 16 * lane);
#pragma unroll
    for (int j = 0; j < NS / 2; ++j)
      ks[j] = *reinterpret_cast<const __attribute__((address_space(3))) uint32_t*>(
          unit_lds + U::kKScales + (16 * (q4 >> 1) + n16) * 2 * NS + 4 * j);
    f32x4 sc[MI][2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) sc[mi][kb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < NS; ++k) {
        const int w = kb * NS + k;
        const f16x2 sp = scale_pair(ks[w >> 2], (w & 2) != 0);
        const f16x8 kf = k_operand(kc[w >> 2][w & 3], (w & 1) ? sp[1] : sp[0]);
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
          sc[mi][kb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[mi][k], sc[mi][kb], 0, 0, 0);
      }
    }
    // a unit that every listed token sees whole: the other tokens' rows are hidden by a reference of +inf, which leaves a
    // NaN score a NaN (rare); else by positions, and nothing from positions past the length
    const bool inside = key0 + kKvUnit - 1 <= pos0 && !bad;
    bool hidden[MI];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) hidden[mi] = ((mask >> bit[mi]) & 1) == 0;
    if (!inside) {
      const int quarter = 4 * (lane_now() >> 4);
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool seen = key0 + 16 * kb + quarter + k <= pos[mi] && !hidden[mi];
            sc[mi][kb][k] = !seen ? -INFINITY : bad ? NAN : sc[mi][kb][k];
          }
      }
      if (key0 + kKvUnit > rq.len || bad) {
        // value scales of positions past the length to zero, in the ring
        const u32x2 keep = {bad ? 0u : keep_bytes(key0 + quarter, rq.len),
                            bad ? 0u : keep_bytes(key0 + 16 + quarter, rq.len)};
        const int half = (lane_now() & 15) >> 3;
#pragma unroll
        for (int r = 0; r < NS; ++r) {
          auto* vs = reinterpret_cast<__attribute__((address_space(3))) u32x2*>(
              unit_lds + U::kVScales + ((quarter / 2 + half) * NS + r) * 8);
          *vs &= keep;      // the eight lanes that share the bytes write the same
        }
      }
    }
    f16x8 pf[MI];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      float t[8];
      auto exponents = [&]() {
        const float ref = hidden[mi] ? INFINITY : m[mi] - kPExp;
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = __fmaf_rn(sc[mi][k >> 2][k & 3], c[mi], -ref);
        if (__builtin_expect(rare, 0)) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            t[k] = hidden[mi] ? -INFINITY : far[mi] ? __fmaf_rn(sc[mi][k >> 2][k & 3] - m[mi], c[mi], kPExp) : t[k];
        }
      };
      exponents();
      const float most =
          fmaxf(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])), fmaxf(fmaxf(t[4], t[5]), fmaxf(t[6], t[7])));
      if (__any(most > kSlack + kPExp)) {
        float mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < 8; ++k) mx = fmaxf(mx, sc[mi][k >> 2][k & 3]);
        const float f = kv_move(hidden[mi] ? -INFINITY : quarter_max(mx), c[mi], m[mi], far[mi]);
        rare |= __any(far[mi]);
        l[mi] *= f;
#pragma unroll
        for (int r = 0; r < NS; ++r)
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[mi][r][x][k] *= f;
        exponents();
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k] = exp2_hw(t[k]);
      l[mi] += ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const f16x2 pr = __builtin_convertvector((f32x2){t[k], t[4 + k]}, f16x2);      // the order of v_octet
        pf[mi][2 * k] = pr[0];
        pf[mi][2 * k + 1] = pr[1];
      }
    }
#pragma unroll
    for (int r = 0; r < NS; ++r) {
      const u32x2 vc = *reinterpret_cast<const __attribute__((address_space(3))) u32x2*>(
          unit_lds + U::kVCodes + 1024 * (r >> 1) + 16 * lane + 8 * (r & 1));
      const u32x2 vs = *reinterpret_cast<const __attribute__((address_space(3))) u32x2*>(
          unit_lds + U::kVScales + ((2 * q4 + (n16 >> 3)) * NS + r) * 8);
      f16x8 ve, vo;
      v_octet(vc[0], vc[1], vs[0], vs[1], &ve, &vo);
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) {
        o[mi][r][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ve, pf[mi], o[mi][r][0], 0, 0, 0);
        o[mi][r][1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vo, pf[mi], o[mi][r][1], 0, 0, 0);
      }
    }
  };

  for (int i = 0, slot = 0; i < mine; ++i) {
    wait_units<kFull + kTail>(min(kRing, mine - i) - 1);
    compute(i, slot);
    if (i + kRing < mine) {
      asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");   // the slot has been read
      issue(i + kRing, slot);
    }
    slot = slot + 1 == kRing ? 0 : slot + 1;
  }

  // the waves' sums: common reference maximum per row, then range by range through LDS
  __syncthreads();      // every wave has read its ring
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    const float ls = quarter_sum(l[mi]);
    m[mi] = kv_reference(m[mi], c[mi], far[mi]);
    if (q4 == 0) {
      m_lds[wave][16 * mi + n16] = m[mi];
      l_lds[wave][16 * mi + n16] = ls;
    }
  }
  __syncthreads();
  float f[MI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    const int rr = 16 * mi + n16;
    float top = m_lds[0][rr];
#pragma unroll
    for (int w = 1; w < NW; ++w) top = fmaxf(top, m_lds[w][rr]);
    f[mi] = exp2_hw(m[mi] - top);
  }
  // of the first 256 threads: thread -> row tid / (256 / BM), consecutive elements of the range
  constexpr int TPR = 256 / BM, EPT = 32 / TPR;
  const int orow = (tid & 255) / TPR, oc = (tid % TPR) * EPT;
  float top = kNone, sum = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) top = fmaxf(top, m_lds[w][orow]);
#pragma unroll
  for (int w = 0; w < NW; ++w) sum += l_lds[w][orow] * exp2_hw(m_lds[w][orow] - top);
  const bool valid = orow < rows && tid < 256, any = sum > 0.f || sum != sum;
  const int t = tiles.parts == 1 ? orow / a.G : 0, g = g0 + orow - t * a.G;
  const size_t dst_row = (size_t)(rq.row0 + tok0 + t) * a.Hq + h * a.G + g;
  const float norm = any ? a.cache.v_gscale / sum : 0.f;
  const size_t slot = ((size_t)tile * hkv + h) * tiles.splits + split;
  const bool whole = tiles.splits == 1;
  if (tid % TPR == 0 && valid) {
    if (!whole) {
      tiles.ml[slot * 2 * BM + orow] = top;
      tiles.ml[slot * 2 * BM + BM + orow] = sum;
    } else if (a.lse) {
      a.lse[dst_row] = any ? kLn2 * (top + (__builtin_amdgcn_logf(sum) - kPExp)) : -INFINITY;
    }
  }
  if (!whole && units == 0) return;      // the join does not read the outputs of an empty split
#pragma unroll
  for (int r = 0; r < NS; ++r) {
    if (r > 0) __syncthreads();
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      float* dst = &o_lds[wave][16 * mi + n16][8 * q4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        dst[2 * k] = o[mi][r][0][k] * f[mi];
        dst[2 * k + 1] = o[mi][r][1][k] * f[mi];
      }
    }
    __syncthreads();
    float v[EPT];
#pragma unroll
    for (int x = 0; x < EPT; ++x) v[x] = 0.f;
#pragma unroll
    for (int w = 0; w < NW; w += 2)
#pragma unroll
      for (int x = 0; x < EPT; ++x) v[x] += o_lds[w][orow][oc + x] + o_lds[w + 1][orow][oc + x];
    if (valid && whole) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + dst_row * D + 32 * r + oc);
#pragma unroll
      for (int x = 0; x < EPT / 2; ++x) dst[x] = f32x2_to_bf16x2(v[2 * x] * norm, v[2 * x + 1] * norm);
    } else if (valid) {
      float* dst = tiles.o + (slot * BM + orow) * D + 32 * r + oc;
#pragma unroll
      for (int x = 0; x < EPT; ++x) dst[x] = v[x];
    }
  }
}

// The splits of a tile joined, a wave per row: the splits' weights from their references and sums, one lane per split,
// then the outputs, four elements per lane and 256 / D splits at once.
template <int D>
__global__ __launch_bounds__(256) void kv_sparse_join_kernel(KvSparseProblem p, SparseTiles tiles) {
  constexpr int LPR = D / 4, PER = 64 / LPR, kAhead = 4;
  const KvAttentionProblem& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, hkv = a.cache.kv_heads;
  const int h = blockIdx.x % hkv, tile = blockIdx.x / hkv, row = 4 * blockIdx.y + wave, S = tiles.splits;
  StepRequest rq;
  int tok0, part;
  if (!sparse_find(a, tiles, tile, &rq, &tok0, &part)) return;
  const int toks = min(tiles.tokens, rq.n - tok0), g0 = part * tiles.bm;
  if (row >= (tiles.parts > 1 ? min(tiles.bm, a.G - g0) : toks * a.G)) return;
  const size_t slot0 = ((size_t)tile * hkv + h) * S;
  const int sub = lane / LPR, d0 = 4 * (lane % LPR);
  float top = kNone, sum = 0.f;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int i0 = 0; i0 < S; i0 += 64) {
    float mi = kNone, li = 0.f;
    if (i0 + lane < S) {
      const float* ml = tiles.ml + (slot0 + i0 + lane) * 2 * tiles.bm + row;
      mi = ml[0];
      li = ml[tiles.bm];
    }
    float most = fmaxf(mi, top);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) most = fmaxf(most, __shfl_xor(most, off));
    const float f = exp2_hw(top - most), w = li != 0.f ? exp2_hw(mi - most) : 0.f;
    top = most;
    sum = sum * f + w * li;
    v *= f;
    const int n = min(64, S - i0);
    for (int j = 0; j < n; j += kAhead * PER) {
      f32x4 x[kAhead];
      float wk[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = j + k * PER + sub;
        wk[k] = __shfl(w, min(i, 63));
        x[k] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (i >= n) wk[k] = 0.f;
        if (wk[k] != 0.f) x[k] = *reinterpret_cast<const f32x4*>(tiles.o + ((slot0 + i0 + i) * tiles.bm + row) * D + d0);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) v += wk[k] * x[k];
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off);
#pragma unroll
  for (int off = LPR; off < 64; off <<= 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += __shfl_xor(v[e], off);
  const bool any = sum > 0.f || sum != sum;
  const float norm = any ? a.cache.v_gscale / sum : 0.f;
  const int t = tiles.parts == 1 ? row / a.G : 0, g = g0 + row - t * a.G;
  const size_t dst = (size_t)(rq.row0 + tok0 + t) * a.Hq + h * a.G + g;
  if (sub == 0)
    *reinterpret_cast<u32x2*>(a.out + dst * D + d0) =
        u32x2{f32x2_to_bf16x2(v[0] * norm, v[1] * norm), f32x2_to_bf16x2(v[2] * norm, v[3] * norm)};
  if (a.lse && lane == 0) a.lse[dst] = any ? kLn2 * (top + (__builtin_amdgcn_logf(sum) - kPExp)) : -INFINITY;
}

// The launch of a call, from its sizes.  Measured on random lists of which neighbouring tokens share about half, 32/8 heads
// of dimension 128, pages of 64, top 24, contexts of 30000 unless said; other side in brackets.
//   Tokens per tile: one while that makes at most kPlaces tiles, which then end sooner (64 tokens 24.1 [28.8] us; 17 requests
//   of 5 tokens on 9000, 18/3 heads of 64, pages of 32, top 25, 10.0 [12.0]), else as many as the rows hold (256 tokens 46.8
//   [64.3]; 2048 226 [460]).
//   Rows per tile: 32 with kWideRows rows over all heads (2048 tokens 226 [241] us; the chunks of 1024 and 748 199 [210];
//   512 tokens 70.9 [76.6], 512 of 64/4 heads 66.0 [71.9] with 16).  Either side may be the better one by a round of
//   workgroups between 32768 and 45056 rows: 32 against 16 rows, 1024 tokens 127.8 / 128.7, 1152 147.9 / 142.8, 1280 151.1 /
//   156.8, 1408 171.6 / 170.8, and of 64/8 heads 640 115.0 / 114.5, 704 130.5 / 125.6; from 49152 on 32 is no slower: 1536
//   175.1 / 184.8, of 64/8 heads 768 133.6 / 135.4.  For groups of 4 heads or more: with fewer a token looks into many other
//   lists (512 tokens of 16/8 heads of 64 46.9 [66.9]; 4096 of 16/8 heads 320 [318]), and a mask holds 16 tokens.
//   Splits: few tiles with 48 units of dimension 128 or more (one token on 131072, 32/4 heads, top 32, 11.5 [17.4] us; top 64
//   13.4 [28.6]; 8 tokens, top 32, 13.2 [18.5]; dimension 256, 16/2 heads, top 32, 15.3 [29.0]); top 16 stays whole, 12.0
//   [10.7], and saves a launch.
//   Waves: eight where the tiles alone leave places free and are not short (64 requests on up to 16000 of 64/8 heads, top 48,
//   42.8 [47.3] us, 48 of them 38.8 [41.7]; 17 requests of 2 to 5 tokens, 18/3 heads of 64, 10.1 [10.9]; but 64 requests, top
//   16, 21.1 with four [23.4]).
constexpr int kPlaces = 512;      // workgroups of four waves
constexpr int64_t kWideRows = 40000;

struct SparsePlan {
  SparseTiles t;
  int64_t tiles;      // bound on their number, over requests, tokens and parts
  int waves;          // of a workgroup
  size_t o_bytes, bytes;
};

SparsePlan sparse_plan(int32_t T, int32_t R, int32_t G, int32_t hkv, int32_t D, int32_t page_size, int32_t top_k) {
  SparsePlan p{};
  const bool many = (int64_t)T * hkv * ((G + 31) / 32) > kPlaces;
  p.t.bm = G > 16 || (many && D != 256 && G >= 4 && (int64_t)T * hkv * G >= kWideRows) ? 32 : 16;
  p.t.parts = (G + p.t.bm - 1) / p.t.bm;
  p.t.tokens = many ? std::max(1, std::min(p.t.bm / G, kEntries / top_k)) : 1;
  p.t.page_units = (uint32_t)((((uint64_t)1 << 32) + page_size / kKvUnit - 1) / (page_size / kKvUnit));
  p.tiles = std::min((int64_t)T, (int64_t)T / p.t.tokens + std::min(T, R)) * p.t.parts;
  const int64_t most = (int64_t)p.t.tokens * top_k * (page_size / kKvUnit), grid = std::max(p.tiles * hkv, (int64_t)1);
  p.t.splits = 1;
  if (most * D >= 48 * 128 && 4 * grid <= kPlaces) p.t.splits = (int)std::min(kPlaces / grid, (most + 3) / 4);
  const bool eight = p.t.splits == 1 && p.t.bm == 16 && D != 256;
  p.waves = eight && (2 * grid <= kPlaces || (grid <= kPlaces && most >= 64)) ? 8 : 4;
  if (p.t.splits > 1) {
    p.o_bytes = (size_t)grid * p.t.splits * p.t.bm * D * 4;
    p.bytes = p.o_bytes + (size_t)grid * p.t.splits * 2 * p.t.bm * 4;
  }
  return p;
}

}  // namespace

bool kv_sparse_launchable(int32_t T, int32_t R, int32_t G, int32_t hkv, int32_t D, int32_t page_size, int32_t top_k) {
  const SparsePlan p = sparse_plan(T, R, G, hkv, D, page_size, top_k);
  return (p.tiles * hkv * p.t.splits + 256) * 64 * p.waves < (int64_t)1 << 32;
}

size_t kv_sparse_workspace(int32_t T, int32_t R, int32_t G, int32_t hkv, int32_t D, int32_t page_size, int32_t top_k) {
  return T == 0 || R == 0 ? 0 : sparse_plan(T, R, G, hkv, D, page_size, top_k).bytes;
}

moe_status_t launch_kv_sparse_attention(const KvSparseProblem& problem, void* workspace, hipStream_t stream) {
  KvSparseProblem p = problem;
  KvAttentionProblem& a = p.a;
  const int hkv = a.cache.kv_heads;
  const int64_t fill = a.fill ? std::min(((int64_t)a.T + 3) / 4, (int64_t)256) : 0;
  SparsePlan plan = sparse_plan(a.T, a.R, a.G, hkv, a.cache.head_dim, a.cache.page_size, p.top_k);
  SparseTiles& t = plan.t;
  t.o = static_cast<float*>(workspace);
  t.ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.o_bytes);
  const int64_t grid = a.R == 0 ? 0 : plan.tiles * hkv * t.splits;
  a.work_groups = (uint32_t)grid;
  const size_t lds = (size_t)t.tokens * p.top_k * 10;
  with_head_dim(a.cache.head_dim, [&](auto tag) {
    constexpr int D = decltype(tag)::value;
    const dim3 blocks((unsigned)(grid + fill));
    if (plan.waves == 8)
      hipLaunchKernelGGL((kv_sparse_kernel<D, 1, D == 256 ? 4 : 8>), blocks, dim3(512), lds, stream, p, t);
    else if (t.bm == 16)
      hipLaunchKernelGGL((kv_sparse_kernel<D, 1, 4>), blocks, dim3(256), lds, stream, p, t);
    else
      hipLaunchKernelGGL((kv_sparse_kernel<D, 2, 4>), blocks, dim3(256), lds, stream, p, t);
    if (t.splits > 1 && grid > 0)
      hipLaunchKernelGGL(kv_sparse_join_kernel<D>, dim3((unsigned)(plan.tiles * hkv), t.bm / 4), dim3(256), 0, stream,
                         p, t);
  });
  return launch_status();
}

}  // namespace moe
