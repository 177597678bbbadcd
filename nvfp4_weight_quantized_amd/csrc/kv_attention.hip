// Attention over the paged NVFP4 key/value cache.
//
// For a query row q at position i and the keys and values of its request:
//   s_j = scale * d_k * (q . K_j),  p_j = exp(s_j - m),  out = d_v * sum_j p_j V_j / sum_j p_j,
//   lse = m + ln sum_j p_j, over the positions j <= i (and j > i - window).
// K_j and V_j are e2m1 * e4m3, built in registers as fp16 matrix operands (exact); a query row enters as
// fp16 after scaling by a power of two that puts its largest element in [2^14, 2^15) (exact for every
// element within 2^-31 of it), undone in the fp32 scores.  Scores, maxima, sums and outputs are fp32;
// p_j is rounded to fp16 (11 bits, 8 times finer than the bf16 output) for the value product.
//
// Both products keep the cache operand first: S^T = K Q^T leaves, in each lane, the scores of one query
// row, and the eight (sixteen) keys a lane then holds are the contraction elements of its operand in
// O^T = V^T P^T when the keys are taken in that order, which is the order the value codes are stored
// in: p goes from one product into the next without leaving its lane.
//
// The running maximum is a reference that only moves when a score exceeds it by more than 2^8 (in
// powers of two): p_j <= 2^8 relative to it, so the sums stay in range and exact in the same way, and
// the usual unit needs no exchange between lanes and no rescale.  p carries another factor 2^7, which
// cancels in out, so that fp16 p reaches down to 2^-31 of the largest.
#include <cfloat>

#include "kv_layout.h"
#include "kv_schedule.h"

namespace moe {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kSlack = 8.f;     // how far a score may exceed the reference maximum
constexpr float kPExp = 7.f;      // power of two carried by p
constexpr float kNone = -FLT_MAX; // reference maximum of a row that has seen nothing

// Eight codes (one dword) of one position times their scale.
__device__ __forceinline__ f16x8 k_operand(uint32_t codes, _Float16 s) {
  const f16x2 ss = {s, s};
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 0) * ss;
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 1) * ss;
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 2) * ss;
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 3) * ss;
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ f16x2 scale_pair(uint32_t bytes, bool high) {
  return high ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(bytes, 1.0f, true)
              : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(bytes, 1.0f, false);
}

// Four positions' bytes (two elements each) with their four scale bytes -> the four values of the even
// element and the four of the odd one.
__device__ __forceinline__ void v_quad(uint32_t codes, uint32_t scales, f16x4* even, f16x4* odd) {
  const f16x2 s01 = scale_pair(scales, false), s23 = scale_pair(scales, true);
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 0);
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 1);
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 2);
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 3);
  const f16x2 e0 = f16x2{a[0], b[0]} * s01, e1 = f16x2{c[0], d[0]} * s23;
  const f16x2 o0 = f16x2{a[1], b[1]} * s01, o1 = f16x2{c[1], d[1]} * s23;
  *even = f16x4{e0[0], e0[1], e1[0], e1[1]};
  *odd = f16x4{o0[0], o0[1], o1[0], o1[1]};
}

// max / sum over the lanes 16 and 32 apart (the lanes that share a query row of a 16-row block)
__device__ __forceinline__ float quarter_max(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float quarter_sum(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// bf16 pair times 2^sh as fp16
__device__ __forceinline__ f16x2 bf16x2_to_f16(uint32_t w, int sh) {
  const f32x2 v = {ldexpf(__uint_as_float(w << 16), sh), ldexpf(__uint_as_float(w & 0xFFFF0000u), sh)};
  return __builtin_convertvector(v, f16x2);
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Keys of dword `first`.. of a unit that lie before position len: byte mask of four scale bytes.
__device__ __forceinline__ uint32_t keep_bytes(int first, int len) {
  const int v = len - first;
  return v >= 4 ? 0xFFFFFFFFu : v <= 0 ? 0u : (1u << (8 * v)) - 1u;
}

struct KvPartials {
  float* o;    // [slot * Hkv + h][BM][D], unnormalised
  float* ml;   // [slot * Hkv + h][2][BM]: reference maximum, sum
};

// ------------------------------------------------------------------------- few rows per request
// One workgroup (four waves) per (kv head, row tile of 16*MI rows, split of the units); each wave takes
// every fourth unit of the split, from 36*D contiguous bytes straight into registers, the next unit's
// loads in flight while this one is multiplied.  The four waves' sums meet in LDS at the end.
template <int D, int MI>
__global__ __launch_bounds__(256) void kv_attention_rows_kernel(KvAttentionProblem a, KvSchedule s, KvPartials part) {
  using U = KvUnit<D>;
  constexpr int NS = D / 32, BM = 16 * MI, NL = NS / 2;
  __shared__ float o_lds[4][BM][36];    // one 32-element range at a time; rows padded to 36 floats
  __shared__ float m_lds[4][BM], l_lds[4][BM];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q4 = lane >> 4, n16 = lane & 15;
  const int hkv = a.cache.kv_heads;
  const int h = blockIdx.x % hkv;
  KvItem it;
  if (!kv_find<false>(a, s, blockIdx.x / hkv, &it)) return;
  const int rows = it.q.n * a.G, row_base = it.tile * BM;
  const int pos0 = it.q.len - it.q.n;          // position of the request's first row

  // query operands: row n16 of block mi, elements [32s + 8*q4, +8)
  f16x8 qf[MI][NS];
  float c[MI];
  int pos[MI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    const int row = row_base + 16 * mi + n16;
    const bool valid = row < rows;
    const int tok = valid ? row / a.G : 0, g = valid ? row - tok * a.G : 0;
    pos[mi] = valid ? pos0 + tok : -1;
    const uint16_t* src = a.q + (int64_t)(it.q.row0 + tok) * a.q_stride + (size_t)(h * a.G + g) * D + 8 * q4;
    u32x4 w[NS];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      w[i] = *reinterpret_cast<const u32x4*>(src + 32 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, max(w[i][j] & 0x7FFFu, (w[i][j] >> 16) & 0x7FFFu));
    }
    int e = (int)(top >> 7);    // the row's largest exponent field
    e = max(e, __shfl_xor(e, 16));
    e = max(e, __shfl_xor(e, 32));
    const int sh = 141 - e;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const f16x2 p0 = bf16x2_to_f16(w[i][0], sh), p1 = bf16x2_to_f16(w[i][1], sh);
      const f16x2 p2 = bf16x2_to_f16(w[i][2], sh), p3 = bf16x2_to_f16(w[i][3], sh);
      qf[mi][i] = f16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
    }
    c[mi] = ldexpf(a.scale * kLog2e, -sh);
  }
  // positions seen by the tile's rows
  const int tok_first = row_base / a.G, tok_last = (min(row_base + BM, rows) - 1) / a.G;
  const int pos_min = pos0 + tok_first, pos_max = pos0 + tok_last;
  int u0 = it.q.lo + it.split * it.chunk, u1 = min(u0 + it.chunk, it.q.hi);
  // every row sees [see_all, pos_min], none anything before see_any
  const int see_all = a.window > 0 ? (int)max(0ll, (long long)pos_max - a.window + 1) : 0;
  const int see_any = a.window > 0 ? (int)max(0ll, (long long)pos_min - a.window + 1) : 0;
  u0 = max(u0, see_any / kKvUnit);
  u1 = pos_max < 0 ? u0 : min(u1, pos_max / kKvUnit + 1);

  f32x4 o[MI][NS][2];
  float m[MI], l[MI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    m[mi] = kNone;
    l[mi] = 0.f;
#pragma unroll
    for (int r = 0; r < NS; ++r) o[mi][r][0] = o[mi][r][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const int upp = a.cache.page_size / kKvUnit;
  const int32_t* table = a.table + (size_t)it.r * a.width;
  // page of unit u, -1 for a bad entry
  auto page_of = [&](int u) {
    const int b = u / upp;
    const int p = b < a.width ? table[b] : -1;
    return p >= 0 && p < a.cache.num_pages ? p : -1;
  };
  struct Regs {
    u32x4 k[NL], v[NL];
    uint32_t ks[NS / 2];      // 2*NS scale bytes
    u32x2 vs[NS];
    int bad;
  };
  int pages = -1;   // lane i: page of the wave's unit u0 + wave + 4*(64*batch + i)
  auto load = [&](int u, int i, Regs& x) {
    if ((i & 63) == 0) {
      const int uu = u + 4 * lane;
      pages = uu < u1 ? page_of(uu) : 0;
    }
    const int p = __builtin_amdgcn_readlane(pages, i & 63);
    x.bad = p < 0;
    const uint8_t* base = a.cache.pages + (((size_t)max(p, 0) * hkv + h) * upp + u % upp) * (size_t)U::kBytes;
#pragma unroll
    for (int j = 0; j < NL; ++j) {
      x.k[j] = *reinterpret_cast<const u32x4*>(base + 1024 * j + 16 * lane);
      x.v[j] = *reinterpret_cast<const u32x4*>(base + U::kVCodes + 1024 * j + 16 * lane);
    }
    const uint32_t* ks = reinterpret_cast<const uint32_t*>(base + U::kKScales + (16 * (q4 >> 1) + n16) * 2 * NS);
#pragma unroll
    for (int j = 0; j < NS / 2; ++j) x.ks[j] = ks[j];
    const u32x2* vs = reinterpret_cast<const u32x2*>(base + U::kVScales + (2 * q4 + (n16 >> 3)) * NS * 8);
#pragma unroll
    for (int j = 0; j < NS; ++j) x.vs[j] = vs[j];
  };

  auto compute = [&](int u, Regs& x) {
    const int key0 = kKvUnit * u;
    f32x4 sc[MI][2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) sc[mi][kb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int w = kb * NS + i;
        const f16x2 sp = scale_pair(x.ks[w >> 2], (w & 2) != 0);
        const f16x8 kf = k_operand(x.k[w >> 2][w & 3], (w & 1) ? sp[1] : sp[0]);
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
          sc[mi][kb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[mi][i], sc[mi][kb], 0, 0, 0);
      }
    }
    // units that some row does not see whole: masks, and nothing from positions past the length
    const bool whole = key0 + kKvUnit - 1 <= pos_min && key0 >= see_all;
    if (!whole || x.bad) {
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = key0 + 16 * kb + 4 * q4 + i;
            const bool seen = key <= pos[mi] && (a.window == 0 || pos[mi] - key < a.window);
            sc[mi][kb][i] = !seen ? -INFINITY : x.bad ? NAN : sc[mi][kb][i];
          }
      const uint32_t k0 = x.bad ? 0u : keep_bytes(key0 + 4 * q4, it.q.len);
      const uint32_t k1 = x.bad ? 0u : keep_bytes(key0 + 16 + 4 * q4, it.q.len);
#pragma unroll
      for (int r = 0; r < NS; ++r) {
        x.vs[r][0] &= k0;
        x.vs[r][1] &= k1;
      }
    }
    f16x8 pf[MI];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = sc[mi][i >> 2][i & 3] * c[mi];
      float mx = fmaxf(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])), fmaxf(fmaxf(t[4], t[5]), fmaxf(t[6], t[7])));
      if (__any(mx > m[mi] + kSlack)) {
        mx = fmaxf(quarter_max(mx), m[mi]);
        const float f = exp2_hw(m[mi] - mx);
        m[mi] = mx;
        l[mi] *= f;
#pragma unroll
        for (int r = 0; r < NS; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[mi][r][e][i] *= f;
      }
      const float ref = m[mi] - kPExp;
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = exp2_hw(t[i] - ref);
      l[mi] += ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f16x2 pr = __builtin_convertvector((f32x2){t[2 * i], t[2 * i + 1]}, f16x2);
        pf[mi][2 * i] = pr[0];
        pf[mi][2 * i + 1] = pr[1];
      }
    }
#pragma unroll
    for (int r = 0; r < NS; ++r) {
      f16x4 e0, o0, e1, o1;
      v_quad(x.v[r >> 1][2 * (r & 1)], x.vs[r][0], &e0, &o0);
      v_quad(x.v[r >> 1][2 * (r & 1) + 1], x.vs[r][1], &e1, &o1);
      const f16x8 ve = __builtin_shufflevector(e0, e1, 0, 1, 2, 3, 4, 5, 6, 7);
      const f16x8 vo = __builtin_shufflevector(o0, o1, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) {
        o[mi][r][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ve, pf[mi], o[mi][r][0], 0, 0, 0);
        o[mi][r][1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vo, pf[mi], o[mi][r][1], 0, 0, 0);
      }
    }
  };

  {
    int u = u0 + wave, i = 0;
    Regs cur, nxt;
    if (u < u1) load(u, 0, cur);
    for (; u < u1; u += 4, ++i) {
      if (u + 4 < u1) load(u + 4, i + 1, nxt);
      compute(u, cur);
      cur = nxt;
    }
  }

  // the four waves' sums: common reference maximum per row, then range by range through LDS
  float f[MI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    const float ls = quarter_sum(l[mi]);
    if (q4 == 0) {
      m_lds[wave][16 * mi + n16] = m[mi];
      l_lds[wave][16 * mi + n16] = ls;
    }
  }
  __syncthreads();
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    const int rr = 16 * mi + n16;
    const float top = fmaxf(fmaxf(m_lds[0][rr], m_lds[1][rr]), fmaxf(m_lds[2][rr], m_lds[3][rr]));
    f[mi] = exp2_hw(m[mi] - top);
  }
  const bool direct = it.splits == 1;
  // thread -> row tid / (256 / BM), consecutive elements of the range
  constexpr int TPR = 256 / BM, EPT = 32 / TPR;
  const int orow = tid / TPR, oc = (tid % TPR) * EPT;
  float top = kNone, sum = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) top = fmaxf(top, m_lds[w][orow]);
#pragma unroll
  for (int w = 0; w < 4; ++w) sum += l_lds[w][orow] * exp2_hw(m_lds[w][orow] - top);
  const int grow = row_base + orow;
  const bool valid = grow < rows;
  const int tok = grow / a.G, g = grow - tok * a.G;
  const size_t at = (size_t)(it.q.row0 + tok) * a.Hq + h * a.G + g;
  const size_t slot = (size_t)(it.slot + it.split) * hkv + h;
  const float norm = sum > 0.f || sum != sum ? a.cache.v_gscale / sum : 0.f;
  if (tid % TPR == 0 && valid) {
    if (direct) {
      if (a.lse) a.lse[at] = sum > 0.f || sum != sum ? kLn2 * (top + (__builtin_amdgcn_logf(sum) - kPExp)) : -INFINITY;
    } else {
      part.ml[slot * 2 * BM + orow] = top;
      part.ml[slot * 2 * BM + BM + orow] = sum;
    }
  }
#pragma unroll
  for (int r = 0; r < NS; ++r) {
    __syncthreads();
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      float* dst = &o_lds[wave][16 * mi + n16][8 * q4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dst[2 * i] = o[mi][r][0][i] * f[mi];
        dst[2 * i + 1] = o[mi][r][1][i] * f[mi];
      }
    }
    __syncthreads();
    float v[EPT];
#pragma unroll
    for (int e = 0; e < EPT; ++e)
      v[e] = (o_lds[0][orow][oc + e] + o_lds[1][orow][oc + e]) + (o_lds[2][orow][oc + e] + o_lds[3][orow][oc + e]);
    if (valid) {
      if (direct) {
        uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + at * D + 32 * r + oc);
#pragma unroll
        for (int e = 0; e < EPT / 2; ++e) dst[e] = f32x2_to_bf16x2(v[2 * e] * norm, v[2 * e + 1] * norm);
      } else {
        float* dst = part.o + (slot * BM + orow) * D + 32 * r + oc;
#pragma unroll
        for (int e = 0; e < EPT; ++e) dst[e] = v[e];
      }
    }
  }
}

// ------------------------------------------------------------------------ many rows per request
// One workgroup (NW waves of 32 rows) per (kv head, row tile, split).  Two units (64 positions) at a
// time are dequantized once into LDS, as fp16 operands of the 32x32x16 instruction in fragment order
// (lane l's 16 bytes at 16*l), and multiplied by every wave; the next pair's codes are in registers and
// its operands written to the other LDS buffer meanwhile.
//   key operand, unit b, step t (16 elements): lane 32z + p holds position p, elements [16t + 8z, +8)
//   value operand, unit b, step t (16 positions), range r: lane 32z + d holds element 32r + d, positions
//     16t + 4z + {0..3} and 16t + 8 + 4z + {0..3}: the ones whose scores lane 32z + n holds after S^T.
template <int D, int NW>
__global__ __launch_bounds__(64 * NW, NW == 8 ? 2 : 1) void kv_attention_tiles_kernel(KvAttentionProblem a,
                                                                                      KvSchedule s, KvPartials part) {
  using U = KvUnit<D>;
  constexpr int NS = D / 32, NT = D / 16, BM = 32 * NW, THREADS = 64 * NW;
  constexpr int kPieces = 8 * D / THREADS;          // 8-byte code pieces per thread and pair of units
  __shared__ __align__(16) uint8_t lds[2][256 * D];   // 64 positions: keys 128*D bytes, then values
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int z = lane >> 5, n32 = lane & 31;
  const int hkv = a.cache.kv_heads;
  const int h = blockIdx.x % hkv;
  KvItem it;
  if (!kv_find<false>(a, s, blockIdx.x / hkv, &it)) return;
  {
    // late rows see the most: their tiles first
    const int t = it.q.tiles - 1 - it.tile;
    it.slot += (t - it.tile) * it.splits;
    it.tile = t;
  }
  const int rows = it.q.n * a.G, row_base = it.tile * BM;
  const int pos0 = it.q.len - it.q.n;

  // query operand: row n32 of the wave, elements [16t + 8z, +8)
  const int row = row_base + 32 * wave + n32;
  const bool valid = row < rows;
  const int tok = valid ? row / a.G : 0, g = valid ? row - tok * a.G : 0;
  int pos = valid ? pos0 + tok : -1;
  f16x8 qf[NT];
  float c;
  {
    const uint16_t* src = a.q + (int64_t)(it.q.row0 + tok) * a.q_stride + (size_t)(h * a.G + g) * D + 8 * z;
    u32x4 w[NT];
    uint32_t top = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      w[t] = *reinterpret_cast<const u32x4*>(src + 16 * t);
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, max(w[t][j] & 0x7FFFu, (w[t][j] >> 16) & 0x7FFFu));
    }
    int e = (int)(top >> 7);
    e = max(e, __shfl_xor(e, 32));
    const int sh = 141 - e;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const f16x2 p0 = bf16x2_to_f16(w[t][0], sh), p1 = bf16x2_to_f16(w[t][1], sh);
      const f16x2 p2 = bf16x2_to_f16(w[t][2], sh), p3 = bf16x2_to_f16(w[t][3], sh);
      qf[t] = f16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
    }
    c = ldexpf(a.scale * kLog2e, -sh);
  }
  // positions that the rows of [first, last) see: all of [*see_all, *pos_min], none outside
  // [*see_any, *pos_max]
  auto reach = [&](int first, int last, int* pos_min, int* pos_max, int* see_all, int* see_any) {
    *pos_min = pos0 + first / a.G;
    *pos_max = pos0 + (min(last, rows) - 1) / a.G;
    *see_all = a.window > 0 ? (int)max(0ll, (long long)*pos_max - a.window + 1) : 0;
    *see_any = a.window > 0 ? (int)max(0ll, (long long)*pos_min - a.window + 1) : 0;
  };
  int pos_min, pos_max, see_all, see_any, u0, u1;
  {
    int t0, t1, t2, t3;
    reach(row_base, row_base + BM, &t0, &t1, &t2, &t3);
    u0 = max(it.q.lo + it.split * it.chunk, t3 / kKvUnit);
    u1 = t1 < 0 ? u0 : min(min(it.q.lo + it.split * it.chunk + it.chunk, it.q.hi), t1 / kKvUnit + 1);
  }
  const int wrow = row_base + 32 * wave;
  const bool live = wrow < rows;                    // the wave has rows
  reach(min(wrow, rows - 1), wrow + 32, &pos_min, &pos_max, &see_all, &see_any);
  // the last pair may reach into the unit behind this split: nothing from `end` on counts
  const int end = min(it.q.len, (int)min((long long)u1 * kKvUnit, 0x7FFFFFFFll));
  const int low = a.window > 0 ? (int)max(0ll, (long long)pos - a.window + 1) : 0;
  pos = min(pos, end - 1);
  pos_min = min(pos_min, end - 1);

  f32x16 o[NS];
  float m = kNone, l = 0.f;
#pragma unroll
  for (int r = 0; r < NS; ++r)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[r][i] = 0.f;

  const int upp = a.cache.page_size / kKvUnit;
  const int32_t* table = a.table + (size_t)it.r * a.width;
  auto page_of = [&](int u) {
    const int b = u / upp;
    const int p = b < a.width ? table[b] : -1;
    return p >= 0 && p < a.cache.num_pages ? p : -1;
  };
  int pages = -1;        // lane i: page of unit u0 + 64*batch + i, -1 bad
  // code pieces of the pair of units at u: piece p < 4D key words, then value words
  u32x2 code[kPieces];
  u32x2 sc[kPieces];
  uint32_t bad_now = 0, bad_next = 0;               // bit b: unit b of the pair has a bad page
  auto load = [&](int u) {
    const int i = u - u0;
    if ((i & 63) == 0) {
      const int uu = u + lane;
      pages = uu < u1 ? page_of(uu) : 0;
    }
    const uint8_t* base[2];
    bad_next = 0;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int p = __builtin_amdgcn_readlane(pages, (i & 63) + b);
      bad_next |= p < 0 ? 1u << b : 0u;
      base[b] = a.cache.pages + (((size_t)max(p, 0) * hkv + h) * upp + (u + b) % upp) * (size_t)U::kBytes;
    }
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int p = tid + THREADS * j;
      const bool is_v = p >= 4 * D;
      const int pp = p & (4 * D - 1), b = pp / (2 * D), x = pp & (2 * D - 1);   // 8-byte piece x of unit b
      const uint8_t* ub = b ? base[1] : base[0];
      code[j] = *reinterpret_cast<const u32x2*>(ub + (is_v ? U::kVCodes : 0) + 8 * x);
      const int ln = (x >> 1) & 63, w = 4 * (x >> 7) + 2 * (x & 1);      // lane of the 16-row operand, word / 2*range
      if (is_v)
        sc[j] = *reinterpret_cast<const u32x2*>(ub + U::kVScales +
                                                ((2 * (ln >> 4) + ((ln & 15) >> 3)) * NS + (w >> 1)) * 8);
      else
        sc[j][0] = *reinterpret_cast<const uint16_t*>(ub + U::kKScales + (16 * (ln >> 5) + (ln & 15)) * 2 * NS + w);
    }
  };
  // the pair at u from registers to LDS buffer `buf`
  auto store = [&](int u, int buf) {
    uint8_t* kl = lds[buf];
    uint8_t* vl = lds[buf] + 128 * D;
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int p = tid + THREADS * j;
      const bool is_v = p >= 4 * D;
      const int pp = p & (4 * D - 1), b = pp / (2 * D), x = pp & (2 * D - 1);
      const int ln = (x >> 1) & 63, w = 4 * (x >> 7) + 2 * (x & 1), q4 = ln >> 4, n16 = ln & 15;
      if (is_v) {
        const int r = w >> 1, key0 = kKvUnit * (u + b);
        u32x2 sv = sc[j];
        if (bad_now & (1u << b)) sv[0] = sv[1] = 0;
        sv[0] &= keep_bytes(key0 + 4 * q4, end);
        sv[1] &= keep_bytes(key0 + 16 + 4 * q4, end);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          f16x4 even, odd;
          v_quad(code[j][t], sv[t], &even, &odd);
          // positions 4*q4..: lane half z = q4 & 1, bytes 8*(q4 >> 1) of its 16
          uint8_t* dst = vl + ((b * 2 + t) * NS + r) * 1024 + 16 * (32 * (q4 & 1) + 2 * n16) + 8 * (q4 >> 1);
          *reinterpret_cast<f16x4*>(dst) = even;
          *reinterpret_cast<f16x4*>(dst + 16) = odd;
        }
      } else {
        const f16x2 sp = scale_pair(sc[j][0], false);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int ww = w + e, kb = ww / NS, i = ww % NS;
          const f16x8 kf = k_operand(code[j][e], sp[e]);
          uint8_t* dst = kl + (b * NT + 2 * i + (q4 >> 1)) * 1024 + 16 * (32 * (q4 & 1) + 16 * kb + n16);
          *reinterpret_cast<f16x8*>(dst) = kf;
        }
      }
    }
  };

  auto compute = [&](int u, int buf, uint32_t bad) {
    const int key0 = kKvUnit * u;
    const uint8_t* kl = lds[buf] + 16 * lane;
    const uint8_t* vl = kl + 128 * D;
    f32x16 sacc[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
      for (int i = 0; i < 16; ++i) sacc[b][i] = 0.f;
#pragma unroll
      for (int t = 0; t < NT; ++t)
        sacc[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(*reinterpret_cast<const f16x8*>(kl + (b * NT + t) * 1024),
                                                         qf[t], sacc[b], 0, 0, 0);
    }
    if (key0 + 63 > pos_min || key0 < see_all || bad) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int key = key0 + 32 * b + 8 * (i >> 2) + 4 * z + (i & 3);
          const bool seen = key <= pos && key >= low;
          sacc[b][i] = !seen ? -INFINITY : (bad >> b) & 1u ? NAN : sacc[b][i];
        }
    }
    float mx = -INFINITY;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        sacc[b][i] *= c;
        mx = fmaxf(mx, sacc[b][i]);
      }
    if (__any(mx > m + kSlack)) {
      const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(mx), __float_as_uint(mx), false, false);
      mx = fmaxf(fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1])), m);
      const float f = exp2_hw(m - mx);
      m = mx;
      l *= f;
#pragma unroll
      for (int r = 0; r < NS; ++r)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[r][i] *= f;
    }
    const float ref = m - kPExp;
    f16x8 pf[2][2];
    float part_sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float p0 = exp2_hw(sacc[b][i] - ref), p1 = exp2_hw(sacc[b][i + 1] - ref);
        part_sum[(i >> 1) & 3] += p0 + p1;
        const f16x2 pr = __builtin_convertvector((f32x2){p0, p1}, f16x2);
        pf[b][i >> 3][i & 7] = pr[0];
        pf[b][i >> 3][(i & 7) + 1] = pr[1];
      }
    l += (part_sum[0] + part_sum[1]) + (part_sum[2] + part_sum[3]);
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < NS; ++r)
          o[r] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
              *reinterpret_cast<const f16x8*>(vl + ((b * 2 + t) * NS + r) * 1024), pf[b][t], o[r], 0, 0, 0);
  };

  if (u0 < u1) {
    load(u0);
    bad_now = bad_next;
    store(u0, 0);
    uint32_t bad = bad_now;
    if (u0 + 2 < u1) load(u0 + 2);
    __syncthreads();
    int buf = 0;
    for (int u = u0; u < u1; u += 2) {
      if (live && kKvUnit * u <= pos_max && kKvUnit * u + 63 >= see_any) compute(u, buf, bad);
      if (u + 2 < u1) {
        bad_now = bad_next;
        bad = bad_now;
        store(u + 2, buf ^ 1);
        if (u + 4 < u1) load(u + 4);
      }
      __syncthreads();
      buf ^= 1;
    }
  }

  {
    const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
    l = __uint_as_float(y[0]) + __uint_as_float(y[1]);
  }
  if (!valid) return;
  const size_t at = (size_t)(it.q.row0 + tok) * a.Hq + h * a.G + g;
  if (it.splits == 1) {
    const bool any = l > 0.f || l != l;
    const float norm = any ? a.cache.v_gscale / l : 0.f;
    if (a.lse && z == 0) a.lse[at] = any ? kLn2 * (m + (__builtin_amdgcn_logf(l) - kPExp)) : -INFINITY;
#pragma unroll
    for (int r = 0; r < NS; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<u32x2*>(a.out + at * D + 32 * r + 8 * i + 4 * z) =
            u32x2{f32x2_to_bf16x2(o[r][4 * i] * norm, o[r][4 * i + 1] * norm),
                  f32x2_to_bf16x2(o[r][4 * i + 2] * norm, o[r][4 * i + 3] * norm)};
  } else {
    const size_t slot = (size_t)(it.slot + it.split) * hkv + h;
    const int lrow = 32 * wave + n32;
    if (z == 0) {
      part.ml[slot * 2 * BM + lrow] = m;
      part.ml[slot * 2 * BM + BM + lrow] = l;
    }
    float* dst = part.o + (slot * BM + lrow) * D + 4 * z;
#pragma unroll
    for (int r = 0; r < NS; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(dst + 32 * r + 8 * i) =
            float4{o[r][4 * i], o[r][4 * i + 1], o[r][4 * i + 2], o[r][4 * i + 3]};
  }
}

// ------------------------------------------------------------------------- combine
// Sixteen rows of one tile per workgroup: the partial sums of its splits added in split order.
template <int D>
__global__ __launch_bounds__(256) void kv_combine_kernel(KvAttentionProblem a, KvSchedule s, KvPartials part) {
  const int hkv = a.cache.kv_heads, tid = threadIdx.x;
  const int h = blockIdx.x % hkv;
  KvItem it;
  if (!kv_find<true>(a, s, blockIdx.x / hkv, &it)) return;
  if (it.splits == 1) return;
  const int row = 16 * blockIdx.y + tid / 16, grow = it.tile * s.bm + row;
  if (grow >= it.q.n * a.G) return;
  constexpr int EPT = D / 16;
  const int d0 = (tid % 16) * EPT;
  const size_t stride = (size_t)hkv * 2 * s.bm, first = ((size_t)it.slot * hkv + h) * 2 * s.bm + row;
  float top = kNone;
  for (int i = 0; i < it.splits; ++i) top = fmaxf(top, part.ml[first + i * stride]);
  float sum = 0.f, v[EPT];
#pragma unroll
  for (int e = 0; e < EPT; ++e) v[e] = 0.f;
  for (int i = 0; i < it.splits; ++i) {
    const float w = exp2_hw(part.ml[first + i * stride] - top);
    sum += w * part.ml[first + i * stride + s.bm];
    const float4* src = reinterpret_cast<const float4*>(
        part.o + (((size_t)(it.slot + i) * hkv + h) * s.bm + row) * D + d0);
#pragma unroll
    for (int e = 0; e < EPT / 4; ++e) {
      const float4 x = src[e];
      v[4 * e] += w * x.x;
      v[4 * e + 1] += w * x.y;
      v[4 * e + 2] += w * x.z;
      v[4 * e + 3] += w * x.w;
    }
  }
  const bool any = sum > 0.f || sum != sum;
  const float norm = any ? a.cache.v_gscale / sum : 0.f;
  const int tok = grow / a.G, g = grow - tok * a.G;
  const size_t at = (size_t)(it.q.row0 + tok) * a.Hq + h * a.G + g;
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + at * D + d0);
#pragma unroll
  for (int e = 0; e < EPT / 2; ++e) dst[e] = f32x2_to_bf16x2(v[2 * e] * norm, v[2 * e + 1] * norm);
  if (a.lse && tid % 16 == 0)
    a.lse[at] = any ? kLn2 * (top + (__builtin_amdgcn_logf(sum) - kPExp)) : -INFINITY;
}

// Host side of one launch: schedule, grid and workspace.
struct Launch {
  KvSchedule s;
  int64_t tiles;    // bound on the row tiles of a kv head
  int64_t items;    // bound on the items of a kv head
  size_t o_bytes, bytes;
};

// bm rows per tile, about `target` items over all heads.  With chunk >= sum(tiles*units)/target the
// items are sum tiles*ceil(units/chunk) <= tiles + target; those of requests with two splits or more
// number at most twice target.
Launch plan_launch(const KvSchedule& s, int32_t T, int32_t R, int32_t G, int32_t hkv, int32_t D) {
  Launch p{};
  p.s = s;
  p.s.target = std::max(1, s.target / hkv);
  p.tiles = std::min((int64_t)R, (int64_t)T) + (int64_t)T * G / s.bm;
  p.items = p.tiles + p.s.target;
  const size_t slots = 2 * (size_t)p.s.target * hkv;
  p.o_bytes = slots * s.bm * D * 4;
  p.bytes = p.o_bytes + slots * 2 * s.bm * 4;
  return p;
}

constexpr int kRowsTarget = 1024;      // items of the few-row kernel over all heads
constexpr int kRowsMinChunk = 4;       // units: one per wave
constexpr int kTilesTarget = 512;
constexpr int kTilesMinChunk = 16;
constexpr int kRowsSplit = 64;         // requests of more rows go to the tile kernel where both run

// The launches of a call: the few-row kernel, the tile kernel, or both, each on its requests.
struct Launches {
  int n;
  bool tiles[2];
  Launch l[2];
};

Launches plan_launches(int32_t T, int32_t R, int32_t G, int32_t hkv, int32_t D) {
  Launches x{};
  const int64_t rows = (int64_t)T * G;
  const bool tiles = rows > (int64_t)kRowsSplit * R || (T >= 1024 && T > R);
  const bool few = !tiles || R > 1;
  if (tiles) {
    const int bm = D == 256 ? 128 : 256;
    x.tiles[x.n] = true;
    x.l[x.n++] = plan_launch(KvSchedule{bm, kTilesTarget, kTilesMinChunk, few ? kRowsSplit : 0, 0x7FFFFFFF}, T, R, G,
                             hkv, D);
  }
  if (few) {
    const int bm = tiles || rows > 16 * (int64_t)R ? 32 : 16;
    x.l[x.n++] = plan_launch(KvSchedule{bm, kRowsTarget, kRowsMinChunk, 0, tiles ? kRowsSplit : 0x7FFFFFFF}, T, R, G,
                             hkv, D);
  }
  return x;
}

}  // namespace

size_t kv_attention_workspace(int32_t T, int32_t R, int32_t Hq, int32_t hkv, int32_t D) {
  if (T == 0 || R == 0) return 0;
  const Launches x = plan_launches(T, R, Hq / hkv, hkv, D);
  size_t bytes = 0;
  for (int i = 0; i < x.n; ++i) bytes = std::max(bytes, x.l[i].bytes);
  return bytes;
}

moe_status_t launch_kv_attention(const KvAttentionProblem& a, void* workspace, hipStream_t stream) {
  const int hkv = a.cache.kv_heads, D = a.cache.head_dim;
  const Launches x = plan_launches(a.T, a.R, a.G, hkv, D);
  for (int i = 0; i < x.n; ++i)
    if (x.l[i].items * hkv > 0x7FFFFFFFLL) return MOE_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < x.n; ++i) {
    const Launch& p = x.l[i];
    KvPartials part{static_cast<float*>(workspace), nullptr};
    part.ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.o_bytes);
    with_head_dim(D, [&](auto tag) {
      constexpr int DD = decltype(tag)::value;
      constexpr int NW = DD == 256 ? 4 : 8;
      const dim3 grid((unsigned)(p.items * hkv));
      if (x.tiles[i])
        hipLaunchKernelGGL((kv_attention_tiles_kernel<DD, NW>), grid, dim3(64 * NW), 0, stream, a, p.s, part);
      else if (p.s.bm == 16)
        hipLaunchKernelGGL((kv_attention_rows_kernel<DD, 1>), grid, dim3(256), 0, stream, a, p.s, part);
      else
        hipLaunchKernelGGL((kv_attention_rows_kernel<DD, 2>), grid, dim3(256), 0, stream, a, p.s, part);
      hipLaunchKernelGGL(kv_combine_kernel<DD>, dim3((unsigned)(p.tiles * hkv), p.s.bm / 16), dim3(256), 0, stream, a,
                         p.s, part);
    });
    if (moe_status_t st = launch_status()) return st;
  }
  return MOE_OK;
}

}  // namespace moe
