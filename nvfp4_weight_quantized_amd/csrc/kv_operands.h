// Operands, softmax references and row filling that the attention kernels over the paged cache share (device code).
#pragma once

#include <cfloat>

#include "kv_layout.h"

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
constexpr float kFar = 0x1p16f;   // reference maximum from which it is held as a raw score

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

// Eight positions' bytes (two elements each): x of the positions 4q + i, y of 16 + 4q + i, with their scale
// bytes -> the operands of the even and of the odd element, positions in the order (i of x, i of y), i =
// 0..3.  The nibbles are paired before they are converted: two shifts and two bit selects for eight pairs.
__device__ __forceinline__ void v_octet(uint32_t x, uint32_t y, uint32_t sx, uint32_t sy, f16x8* even, f16x8* odd) {
  const uint32_t e = ((y << 4) & 0xF0F0F0F0u) | (x & 0x0F0F0F0Fu), o = (y & 0xF0F0F0F0u) | ((x >> 4) & 0x0F0F0F0Fu);
  const uint32_t s01 = __builtin_amdgcn_perm(sy, sx, 0x05010400u), s23 = __builtin_amdgcn_perm(sy, sx, 0x07030602u);
  const f16x2 s0 = scale_pair(s01, false), s1 = scale_pair(s01, true), s2 = scale_pair(s23, false), s3 = scale_pair(s23, true);
  const f16x2 e0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(e, 1.0f, 0) * s0, e1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(e, 1.0f, 1) * s1;
  const f16x2 e2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(e, 1.0f, 2) * s2, e3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(e, 1.0f, 3) * s3;
  const f16x2 o0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(o, 1.0f, 0) * s0, o1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(o, 1.0f, 1) * s1;
  const f16x2 o2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(o, 1.0f, 2) * s2, o3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(o, 1.0f, 3) * s3;
  *even = f16x8{e0[0], e0[1], e1[0], e1[1], e2[0], e2[1], e3[0], e3[1]};
  *odd = f16x8{o0[0], o0[1], o1[0], o1[1], o2[0], o2[1], o3[0], o3[1]};
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

// the same over the two lanes 32 apart (a row of a 32-row block)
__device__ __forceinline__ float half_max(float v) {
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// bf16 pair times 2^sh as fp16
__device__ __forceinline__ f16x2 bf16x2_to_f16(uint32_t w, int sh) {
  const f32x2 v = {ldexpf(__uint_as_float(w << 16), sh), ldexpf(__uint_as_float(w & 0xFFFF0000u), sh)};
  return __builtin_convertvector(v, f16x2);
}

// Power of two that brings a row with largest bf16 exponent field e to [2^14, 2^15), held below the one
// that would take the scores' factor c0 * 2^-shift out of the normal range (a row that small, zeros
// included, has scores of 0 for every purpose).
__device__ __forceinline__ int row_shift(int e, float c0) { return min(141 - e, ilogbf(c0) + 120); }

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// The reference maximum m of a row moved to the largest of it and of the raw score mx (-inf: none seen); the
// factor for its sums.  c: the scores' factor.  A row that was far stays so.  Branches of its own per lane: with one
// branch of the wave and selects behind it one request of 1024 takes 0.1 us less, but the tile kernel of dimension 256
// spills 36 registers (175 -> 242 us for the chunks).
__device__ __forceinline__ float kv_move(float mx, float c, float& m, bool& far) {
  float f = 1.f;
  if (!far) {
    const float top = fmaxf(mx * c, m);
    if (fabsf(top) < kFar || mx == -INFINITY) {
      f = exp2_hw(m - top);
      m = top;
      return f;
    }
    far = true;
    if (m != kNone) {      // from log2 units to the nearest raw score, the sums corrected by what that rounds
      const float raw = m / c;
      f = exp2_hw(__fmaf_rn(-raw, c, m));
      m = raw;
    }
  }
  const float top = fmaxf(mx, m);
  f *= exp2_hw((m - top) * c);
  m = top;
  return f;
}

// A far row's reference maximum in log2 units, where those of a row's partial sums are compared.
__device__ __forceinline__ float kv_reference(float m, float c, bool far) {
  return far ? fmaxf(fminf(m * c, FLT_MAX), -FLT_MAX) : m;
}

// Keys of dword `first`.. of a unit that lie before position len: byte mask of four scale bytes.
__device__ __forceinline__ uint32_t keep_bytes(int first, int len) {
  const int v = len - first;
  return v >= 4 ? 0xFFFFFFFFu : v <= 0 ? 0u : (1u << (8 * v)) - 1u;
}

// Zeros (lse: -inf) for the rows of no request, [0, offsets[0]) and [offsets[R], T): workgroup `index` of `count`.
// Workgroups of their own behind those of the launch, so the others neither wait for the offsets nor carry the stores.
// One per four rows, up to the card's compute units (1100 padded rows of 32 heads of 128, 9 MB: 32 workgroups take 7 us
// longer).  Inlined: a call gives the tile kernel a stack and spills (prompt of 8192 564 -> 632 us).
template <int D>
__device__ __forceinline__ void kv_fill_rows(const KvAttentionProblem& a, int index, int count) {
  const int before = a.R > 0 ? min(max(a.offsets[0], 0), a.T) : a.T;
  const int after = a.R > 0 ? min(max(a.offsets[a.R], before), a.T) : a.T;
  for (int i = index; i < before + a.T - after; i += count) {
    const size_t row = (size_t)(i < before ? i : i - before + after) * a.Hq;
    u32x4* out = reinterpret_cast<u32x4*>(a.out + row * D);
    for (int j = threadIdx.x; j < a.Hq * (D / 8); j += blockDim.x) out[j] = u32x4{0, 0, 0, 0};
    if (a.lse)
      for (int j = threadIdx.x; j < a.Hq; j += blockDim.x) a.lse[row + j] = -INFINITY;
  }
}

// For a step without requests.
template <int D>
__global__ __launch_bounds__(256) void kv_fill_kernel(KvAttentionProblem a) {
  kv_fill_rows<D>(a, blockIdx.x, gridDim.x);
}

// Units of a wave's ring in LDS: 147 of a compute unit's 160 KB for four workgroups of four waves, dimension 128.
constexpr int kRing = 2;

// Waits until at most n units' loads (PER instructions each) of this wave are in flight, n < kRing.
template <int PER>
__device__ __forceinline__ void wait_units(int n) {
  static_assert(kRing == 2 && PER <= 63, "the counter of loads in flight");
  if (n == 0) asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
  else asm volatile("s_waitcnt vmcnt(%0)" : : "n"(PER) : "memory");
}

}  // namespace
}  // namespace moe
