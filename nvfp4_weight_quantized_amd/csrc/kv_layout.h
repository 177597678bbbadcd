// Device-side addressing of the paged NVFP4 key/value cache (layout: include/moe_nvfp4.h).
#pragma once

#include "common.h"

namespace moe {
namespace {

// Byte offsets inside one 36*D-byte unit of 32 positions, p the position in the unit, d an element.
template <int D>
struct KvUnit {
  static constexpr int NS = D / 32;            // 32-element ranges of the head dimension
  static constexpr int kBytes = 36 * D;
  static constexpr int kVCodes = 16 * D;
  static constexpr int kKScales = 32 * D;
  static constexpr int kVScales = 34 * D;
  // four bytes (8 codes) of the key elements [8*g8, 8*g8 + 8)
  __device__ static int k_word(int p, int g8) {
    const int w = (p >> 4) * NS + (g8 >> 2);
    return 1024 * (w >> 2) + 16 * (16 * (g8 & 3) + (p & 15)) + 4 * (w & 3);
  }
  // the byte of the value elements 2*m2, 2*m2 + 1
  __device__ static int v_byte(int p, int m2) {
    const int r = m2 >> 4, q = (p & 15) >> 2;
    return kVCodes + 1024 * (r >> 1) + 16 * (16 * q + (m2 & 15)) + 8 * (r & 1) + 4 * (p >> 4) + (p & 3);
  }
  // scale byte of 16-element group g
  __device__ static int k_scale(int p, int g) {
    return kKScales + (16 * (g & 1) + (p & 15)) * 2 * NS + (p >> 4) * NS + (g >> 1);
  }
  __device__ static int v_scale(int p, int g) {
    const int q = (p & 15) >> 2;
    return kVScales + ((2 * q + (g & 1)) * NS + (g >> 1)) * 8 + 4 * (p >> 4) + (p & 3);
  }
};

// First byte of the unit holding position `slot` (page * page_size + offset) of head h.
template <int D>
__device__ __forceinline__ size_t kv_unit_offset(const moe_nvfp4_kv_cache_t& c, int slot, int h) {
  const int page = slot / c.page_size, off = slot % c.page_size;
  const int upp = c.page_size / kKvUnit;
  return (((size_t)page * c.kv_heads + h) * upp + off / kKvUnit) * (size_t)KvUnit<D>::kBytes;
}

// Calls f(tag) with the head dimension as a compile-time constant.
template <int N>
struct DimC {
  static constexpr int value = N;
};
template <typename F>
void with_head_dim(int d, F&& f) {
  if (d == 64) f(DimC<64>{});
  else if (d == 128) f(DimC<128>{});
  else f(DimC<256>{});
}

}  // namespace
}  // namespace moe
