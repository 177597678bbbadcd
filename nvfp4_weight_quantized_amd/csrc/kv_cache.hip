// Paged NVFP4 key/value cache: the step plan (block table entries, slots, offsets), the append that
// quantizes new rows into the pages, and the gather that dequantizes rows by slot.
#include "codec.h"
#include "kv_layout.h"

namespace moe {
namespace {

// ------------------------------------------------------------------------------------ plan
constexpr int kPlanThreads = 1024;
constexpr int kPlanPerThread = kKvMaxRequests / kPlanThreads;   // 4 consecutive requests per thread

__device__ __forceinline__ int sat31(long long v) { return (int)min(v, 0x7FFFFFFFll); }

// Every workgroup forms the two prefix sums over the requests (tokens, pages opened) in LDS and then
// places its own 1024 tokens; workgroup 0 also writes the per-request outputs.  A page is opened by
// exactly one token, the one at its first position, so no two workgroups write the same entry, and
// the entries read (pages held) are never written.
__global__ __launch_bounds__(kPlanThreads) void kv_plan_kernel(
    const int32_t* __restrict__ kv_lens, const int32_t* __restrict__ new_lens, int R, int ps, int num_pages,
    const int32_t* __restrict__ free_pages, int num_free, int32_t* block_table, int width, int T,
    int32_t* __restrict__ query_offsets, int32_t* __restrict__ seq_lens, int32_t* __restrict__ positions,
    int32_t* __restrict__ slots, int32_t* __restrict__ pages_used) {
  __shared__ int qo[kKvMaxRequests + 1];
  __shared__ int fo[kKvMaxRequests];
  __shared__ long long wave_tok[kPlanThreads / 64], wave_pg[kPlanThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  long long tok[kPlanPerThread], pg[kPlanPerThread], st = 0, sp = 0;
#pragma unroll
  for (int i = 0; i < kPlanPerThread; ++i) {
    const int r = tid * kPlanPerThread + i;
    long long o = 0, n = 0;
    if (r < R) {
      o = max(kv_lens[r], 0);
      n = max(new_lens[r], 0);
      if (blockIdx.x == 0) seq_lens[r] = sat31(o + n);
    }
    tok[i] = st;
    pg[i] = sp;
    st += n;
    sp += (o + n + ps - 1) / ps - (o + ps - 1) / ps;
  }
  long long it = st, ip = sp;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const long long a = __shfl_up(it, off), b = __shfl_up(ip, off);
    if (lane >= off) {
      it += a;
      ip += b;
    }
  }
  if (lane == 63) {
    wave_tok[wave] = it;
    wave_pg[wave] = ip;
  }
  __syncthreads();
  long long bt = it - st, bp = ip - sp, total_t = 0, total_p = 0;
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    if (w < wave) {
      bt += wave_tok[w];
      bp += wave_pg[w];
    }
    total_t += wave_tok[w];
    total_p += wave_pg[w];
  }
#pragma unroll
  for (int i = 0; i < kPlanPerThread; ++i) {
    const int r = tid * kPlanPerThread + i;
    if (r < R) {
      qo[r] = sat31(bt + tok[i]);
      fo[r] = sat31(bp + pg[i]);
      if (blockIdx.x == 0) query_offsets[r] = qo[r];
    }
  }
  if (tid == 0) {
    qo[R] = sat31(total_t);
    if (blockIdx.x == 0) {
      query_offsets[R] = sat31(total_t);
      pages_used[0] = sat31(total_p);
    }
  }
  __syncthreads();
  const long long tl = (long long)blockIdx.x * kPlanThreads + tid;
  if (tl >= T) return;
  const int t = (int)tl;
  if (t >= qo[R]) {
    positions[t] = 0;
    slots[t] = -1;
    return;
  }
  int lo = 0, hi = R;   // the last r with qo[r] <= t (an idle request never holds t: qo[r+1] == qo[r])
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (qo[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int r = lo;
  const int o = max(kv_lens[r], 0);
  const long long pos = (long long)o + (t - qo[r]);
  const long long b = pos / ps, have = ((long long)o + ps - 1) / ps;
  int page = -1;
  if (b < width) {
    int32_t* entry = block_table + (size_t)r * width + b;
    if (b < have) {
      page = *entry;
    } else {
      const long long fi = (long long)fo[r] + (b - have);
      if (fi < num_free) page = free_pages[fi];
    }
    if (page >= num_pages || page < 0) page = -1;
    if (b >= have && pos % ps == 0) *entry = page;
  }
  positions[t] = sat31(pos);
  slots[t] = page < 0 ? -1 : page * ps + (int)(pos % ps);
}

// ------------------------------------------------------------------------------------ append
// One thread per (token, head, K or V, 16-element group).
template <int D>
__global__ __launch_bounds__(256) void kv_append_kernel(moe_nvfp4_kv_cache_t c, const uint16_t* __restrict__ k,
                                                        const uint16_t* __restrict__ v, int64_t k_stride,
                                                        int64_t v_stride, const int32_t* __restrict__ slots, int T) {
  using U = KvUnit<D>;
  constexpr int NG = D / 16;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int per_token = 2 * c.kv_heads * NG;
  const long long tl = i / per_token;
  if (tl >= T) return;
  const int t = (int)tl, rest = (int)(i % per_token);
  const int g = rest % NG, h = (rest / NG) % c.kv_heads;
  const bool is_v = rest / NG >= c.kv_heads;
  const int slot = slots[t];
  if (slot < 0 || slot >= c.num_pages * c.page_size) return;
  const uint16_t* row = is_v ? v + t * v_stride : k + t * k_stride;
  const uint4* src = reinterpret_cast<const uint4*>(row + h * D + g * 16);
  float x[16];
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
  uint32_t lo, hi, sc;
  quantize_group16(x, is_v ? c.v_gscale : c.k_gscale, &lo, &hi, &sc);
  uint8_t* unit = c.pages + kv_unit_offset<D>(c, slot, h);
  const int p = slot % kKvUnit;
  if (is_v) {
#pragma unroll
    for (int b = 0; b < 8; ++b) unit[U::v_byte(p, 8 * g + b)] = (uint8_t)((b < 4 ? lo >> (8 * b) : hi >> (8 * b - 32)) & 255u);
    unit[U::v_scale(p, g)] = (uint8_t)sc;
  } else {
    *reinterpret_cast<uint32_t*>(unit + U::k_word(p, 2 * g)) = lo;
    *reinterpret_cast<uint32_t*>(unit + U::k_word(p, 2 * g + 1)) = hi;
    unit[U::k_scale(p, g)] = (uint8_t)sc;
  }
}

// ------------------------------------------------------------------------------------ gather
__device__ __forceinline__ float e2m1_f32(uint32_t code) {
  const uint32_t m = code & 7u;
  const float v = m < 4u ? 0.5f * (float)m : (m < 6u ? (float)(m - 2u) : (m == 6u ? 4.f : 6.f));
  return (code & 8u) ? -v : v;
}

template <int D>
__global__ __launch_bounds__(256) void kv_gather_kernel(moe_nvfp4_kv_cache_t c, const int32_t* __restrict__ slots,
                                                        int n, uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
  using U = KvUnit<D>;
  constexpr int NG = D / 16;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int per_token = 2 * c.kv_heads * NG;
  const long long tl = i / per_token;
  if (tl >= n) return;
  const int t = (int)tl, rest = (int)(i % per_token);
  const int g = rest % NG, h = (rest / NG) % c.kv_heads;
  const bool is_v = rest / NG >= c.kv_heads;
  uint16_t* dst = (is_v ? v : k) + ((size_t)t * c.kv_heads + h) * D + g * 16;
  const int slot = slots[t];
  uint32_t w[8];
  if (slot < 0 || slot >= c.num_pages * c.page_size) {
#pragma unroll
    for (int b = 0; b < 8; ++b) w[b] = 0x7FC07FC0u;
  } else {
    const uint8_t* unit = c.pages + kv_unit_offset<D>(c, slot, h);
    const int p = slot % kKvUnit;
    const float s = __builtin_amdgcn_cvt_f32_fp8((int)unit[is_v ? U::v_scale(p, g) : U::k_scale(p, g)], 0);
    const float d = is_v ? c.v_gscale : c.k_gscale;
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const uint32_t byte = is_v ? unit[U::v_byte(p, 8 * g + b)] : unit[U::k_word(p, 2 * g + (b >> 2)) + (b & 3)];
      w[b] = f32x2_to_bf16x2(e2m1_f32(byte & 15u) * s * d, e2m1_f32(byte >> 4) * s * d);
    }
  }
  reinterpret_cast<uint4*>(dst)[0] = uint4{w[0], w[1], w[2], w[3]};
  reinterpret_cast<uint4*>(dst)[1] = uint4{w[4], w[5], w[6], w[7]};
}

}  // namespace

moe_status_t launch_kv_plan(const int32_t* kv_lens, const int32_t* new_lens, int32_t R, int32_t page_size,
                            int32_t num_pages, const int32_t* free_pages, int32_t num_free, int32_t* block_table,
                            int32_t table_width, int32_t num_tokens, int32_t* query_offsets, int32_t* seq_lens,
                            int32_t* positions, int32_t* slots, int32_t* pages_used, hipStream_t stream) {
  const int blocks = std::max(1, (int)(((int64_t)num_tokens + kPlanThreads - 1) / kPlanThreads));
  hipLaunchKernelGGL(kv_plan_kernel, dim3(blocks), dim3(kPlanThreads), 0, stream, kv_lens, new_lens, R, page_size,
                     num_pages, free_pages, num_free, block_table, table_width, num_tokens, query_offsets, seq_lens,
                     positions, slots, pages_used);
  return launch_status();
}

moe_status_t launch_kv_append(const moe_nvfp4_kv_cache_t& c, const uint16_t* k, const uint16_t* v, int64_t k_stride,
                              int64_t v_stride, const int32_t* slots, int32_t T, hipStream_t stream) {
  const long long total = (long long)T * 2 * c.kv_heads * (c.head_dim / 16), blocks = (total + 255) / 256;
  if (blocks > 0x7FFFFFFFLL) return MOE_ERR_INVALID_ARGUMENT;
  with_head_dim(c.head_dim, [&](auto tag) {
    hipLaunchKernelGGL(kv_append_kernel<decltype(tag)::value>, dim3((unsigned)blocks), dim3(256), 0, stream, c, k, v,
                       k_stride, v_stride, slots, T);
  });
  return launch_status();
}

moe_status_t launch_kv_gather(const moe_nvfp4_kv_cache_t& c, const int32_t* slots, int32_t n, uint16_t* k,
                              uint16_t* v, hipStream_t stream) {
  const long long total = (long long)n * 2 * c.kv_heads * (c.head_dim / 16), blocks = (total + 255) / 256;
  if (blocks > 0x7FFFFFFFLL) return MOE_ERR_INVALID_ARGUMENT;
  with_head_dim(c.head_dim, [&](auto tag) {
    hipLaunchKernelGGL(kv_gather_kernel<decltype(tag)::value>, dim3((unsigned)blocks), dim3(256), 0, stream, c, slots,
                       n, k, v);
  });
  return launch_status();
}

}  // namespace moe
