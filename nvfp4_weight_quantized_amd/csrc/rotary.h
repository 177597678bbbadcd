// Rotary positions on the device: the cosines and sines of a block's tokens, and the rotation of a row's elements.
//
// Pair i of a row turns by a = positions[axis_i][t] * inv_freq_i:
//   y1 = x1 cos a - x2 sin a,  y2 = x2 cos a + x1 sin a.
// The angle is formed and reduced in 64 bits, since in 32 an angle of 10^5 is already off by 2^-8; there is no table of
// positions to read.  Cosine and sine are rounded to fp32 once.  Products and their sum are rounded one by one (no
// fused multiply-add), so that rotated rows do not depend on how the compiler contracts them.
#pragma once

#include "common.h"
#include "rotary_launch.h"

namespace moe {
namespace {

// Entries are read four to a load by lanes that are 8 (or 4) entries apart; 16-byte pieces 256 bytes apart lie in the same
// banks, so those of each next 256 bytes are exchanged among four.
struct RotaryTable {
  float4 pieces[kRotaryEntries / 2];
  __device__ static int place(int piece) { return piece ^ ((piece >> 4) & 3); }
  __device__ float4 pair(int entry) const { return pieces[place(entry >> 1)]; }      // entry even: two entries
  __device__ float2& at(int entry) { return reinterpret_cast<float2*>(&pieces[place(entry >> 1)])[entry & 1]; }
};

// Division by a number that the host knows: of i with i * divisor < 2^32.
struct Divider {
  uint32_t divisor, magic;      // 2^32 / divisor, rounded up; 0: 1
  static Divider of(uint32_t d) { return Divider{d, (uint32_t)((((uint64_t)1 << 32) + d - 1) / d)}; }
  __device__ uint32_t operator()(uint32_t i) const { return magic ? __umulhi(i, magic) : i; }
};

// (cos a, sin a) * scale.  a = k pi/2 + r with |r| <= pi/4, pi/2 in two parts (|a| < 2^40: the parts reach 2^-106, so
// r is off by less than 2^-52), then the Taylor series: the first terms left out are r^17 / 17! < 2^-54 and
// r^18 / 18! < 2^-58.
__device__ __forceinline__ float2 rotary_turn(double a, float scale) {
  const double k = rint(a * 0.63661977236758134);
  double r = fma(-k, 1.5707963267948966, a);
  r = fma(-k, 6.123233995736766e-17, r);
  const double z = r * r;
  double s = fma(z, -1.0 / 1307674368000.0, 1.0 / 6227020800.0);
  s = fma(z, s, -1.0 / 39916800.0);
  s = fma(z, s, 1.0 / 362880.0);
  s = fma(z, s, -1.0 / 5040.0);
  s = fma(z, s, 1.0 / 120.0);
  s = fma(z, s, -1.0 / 6.0);
  s = fma(z * r, s, r);
  double c = fma(z, 1.0 / 20922789888000.0, -1.0 / 87178291200.0);
  c = fma(z, c, 1.0 / 479001600.0);
  c = fma(z, c, -1.0 / 3628800.0);
  c = fma(z, c, 1.0 / 40320.0);
  c = fma(z, c, -1.0 / 720.0);
  c = fma(z, c, 1.0 / 24.0);
  c = fma(z, c, -0.5);
  c = fma(z, c, 1.0);
  const int quadrant = (int)(k - 4.0 * floor(k * 0.25));
  const double x = quadrant & 1 ? s : c, y = quadrant & 1 ? c : s;
  const double cs = quadrant == 1 || quadrant == 2 ? -x : x, sn = quadrant >= 2 ? -y : y;
  return float2{(float)(cs * scale), (float)(sn * scale)};
}

// The entries of the tokens [t0, t0 + count): pairs * i + pair.
__device__ __forceinline__ void rotary_table(const moe_rotary_t& r, const int32_t* __restrict__ positions,
                                             int64_t position_stride, int t0, int count, RotaryTable& table) {
  for (int i = threadIdx.x; i < count * r.pairs; i += blockDim.x) {
    const int t = i / r.pairs, pair = i - t * r.pairs;
    const int axis = r.axis ? min(max(r.axis[pair], 0), r.axes - 1) : 0;
    const double angle = (double)positions[axis * position_stride + t0 + t] * r.inv_freq[pair];
    table.at(i) = rotary_turn(angle, r.scale);
  }
}

struct Chunk {      // eight elements
  float v[8];
};

__device__ __forceinline__ Chunk chunk_of(const uint4& w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  Chunk x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x.v[2 * i] = __uint_as_float(u[i] << 16);
    x.v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
  return x;
}

__device__ __forceinline__ uint4 bits_of(const Chunk& x) {
  return uint4{f32x2_to_bf16x2(x.v[0], x.v[1]), f32x2_to_bf16x2(x.v[2], x.v[3]), f32x2_to_bf16x2(x.v[4], x.v[5]),
               f32x2_to_bf16x2(x.v[6], x.v[7])};
}

__device__ __forceinline__ void rotate_pair(float c, float s, float& x, float& y) {
#pragma clang fp contract(off)
  const float xc = x * c, ys = y * s, yc = y * c, xs = x * s;
  x = xc - ys;
  y = yc + xs;
}

// a, b: the first and the second elements of eight pairs, whose entries begin at `entry`.
__device__ __forceinline__ void rotate_halves(const RotaryTable& table, int entry, Chunk& a, Chunk& b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 t = table.pair(entry + 2 * i);
    rotate_pair(t.x, t.y, a.v[2 * i], b.v[2 * i]);
    rotate_pair(t.z, t.w, a.v[2 * i + 1], b.v[2 * i + 1]);
  }
}

// Four pairs of neighbours.
__device__ __forceinline__ void rotate_neighbours(const RotaryTable& table, int entry, Chunk& a) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 t = table.pair(entry + 2 * i);
    rotate_pair(t.x, t.y, a.v[4 * i], a.v[4 * i + 1]);
    rotate_pair(t.z, t.w, a.v[4 * i + 2], a.v[4 * i + 3]);
  }
}

}  // namespace
}  // namespace moe
