// Quantization of key and value rows into the pages of the cache: what the appends share (device code).
#pragma once

#include "codec.h"
#include "kv_layout.h"

namespace moe {
namespace {

__device__ __forceinline__ void load_group16(const uint16_t* __restrict__ row, float (&x)[16]) {
  const uint4* src = reinterpret_cast<const uint4*>(row);
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    const uint4 w = src[a];
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      x[8 * a + 2 * b] = __uint_as_float(u[b] << 16);
      x[8 * a + 2 * b + 1] = __uint_as_float(u[b] & 0xFFFF0000u);
    }
  }
}

// Group g of head h, of the keys or the values, of the rows [t0, t0 + W) of a step into the cache; load(t, x) gives
// row t's 16 elements.  W = 4 takes every quad of positions that begins among the rows (kv_cache.hip).
template <int D, int W, typename Load>
__device__ __forceinline__ void append_window(const moe_nvfp4_kv_cache_t& c, Load&& load, float d, bool is_v, int h,
                                              int g, int t0, const int32_t* __restrict__ slots, int T) {
  using U = KvUnit<D>;
  const int cap = c.num_pages * c.page_size;
  for (int t = t0; t < min(t0 + W, T);) {
    const int s = slots[t];
    int n = 1;
    if (s < 0 || s >= cap) {
      ++t;
      continue;
    }
    if (W > 1) {
      if ((s & 3) != 0 && t > 0 && slots[t - 1] == s - 1) {      // the quad's first row takes this one
        ++t;
        continue;
      }
      while (n < 4 && ((s + n) & 3) != 0 && t + n < T && slots[t + n] == s + n) ++n;
    }
    uint8_t* unit = c.pages + kv_unit_offset<D>(c, s, h);
    const int p = s % kKvUnit;
    uint32_t lo[W], hi[W], sc[W];
#pragma unroll
    for (int r = 0; r < W; ++r) {
      if (r < n) {
        float x[16];
        load(t + r, x);
        quantize_group16_fast(x, d, &lo[r], &hi[r], &sc[r]);
      }
    }
    if (!is_v) {
#pragma unroll
      for (int r = 0; r < W; ++r) {
        if (r < n) {
          *reinterpret_cast<uint32_t*>(unit + U::k_word(p + r, 2 * g)) = lo[r];
          *reinterpret_cast<uint32_t*>(unit + U::k_word(p + r, 2 * g + 1)) = hi[r];
          unit[U::k_scale(p + r, g)] = (uint8_t)sc[r];
        }
      }
    } else if (W == 4 && n == 4) {
      // byte b of the four rows' words -> one dword
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        const uint32_t(&w)[W] = b < 4 ? lo : hi;
        const uint32_t sel = 0x0C0C0400u + 0x0101u * (b & 3);      // byte b & 3 of the second and of the first operand
        const uint32_t a01 = __builtin_amdgcn_perm(w[1 % W], w[0], sel), a23 = __builtin_amdgcn_perm(w[3 % W], w[2 % W], sel);
        *reinterpret_cast<uint32_t*>(unit + U::v_byte(p, 8 * g + b)) = a01 | (a23 << 16);
      }
      *reinterpret_cast<uint32_t*>(unit + U::v_scale(p, g)) = sc[0] | (sc[1 % W] << 8) | (sc[2 % W] << 16) | (sc[3 % W] << 24);
    } else {
#pragma unroll
      for (int r = 0; r < W; ++r) {
        if (r < n) {
#pragma unroll
          for (int b = 0; b < 8; ++b)
            unit[U::v_byte(p + r, 8 * g + b)] = (uint8_t)((b < 4 ? lo[r] >> (8 * b) : hi[r] >> (8 * b - 32)) & 255u);
          unit[U::v_scale(p + r, g)] = (uint8_t)sc[r];
        }
      }
    }
    t += n;
  }
}

}  // namespace
}  // namespace moe
