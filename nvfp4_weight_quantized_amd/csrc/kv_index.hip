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
constexpr int kKeys = kKvMaxSelectPages;

// A workgroup per token and kv head: the group's rows in 8 bits, a key per page (its score as an ordered integer), and
// the largest top_k of them.
template <int D>
__global__ __launch_bounds__(256) void kv_select_kernel(KvSelectProblem p) {
  __shared__ uint32_t keys[kKeys];
  __shared__ __align__(16) int8_t rows[64][D];
  __shared__ float tops[64];
  const KvStep& s = p.step;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, h = blockIdx.y, hkv = p.index.kv_heads;
  const int t = blockIdx.x;
  int32_t* out = p.selected + ((size_t)t * hkv + h) * p.top_k;
  StepRequest q;
  int within;
  bool any = step_find(s, t - min(max(s.R > 0 ? s.offsets[0] : 0, 0), s.T), [&](const StepRequest& x) { return x.n; }, &q, &within);
  const int pos = any ? q.len - q.n + within : -1;
  if (!any || q.row0 + within != t || pos < 0) {
    for (int i = tid; i < p.top_k; i += 256) out[i] = -1;
    return;
  }
  const int own = pos / s.page_size, count = min(own + 1, s.width);
  for (int g = wave; g < p.G; g += 4) {
    constexpr int N = D / 64;
    const uint16_t* src = p.q + (int64_t)t * p.q_stride + (size_t)(h * p.G + g) * D;
    float x[N], top = 0.f;
    bool fine = true;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = bf16_to_f32(src[64 * i + lane]);
      fine &= fabsf(x[i]) <= 0x1p100f;
      top = fmaxf(top, fabsf(x[i]));
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    const bool use = __all(fine) && top >= 0x1p-100f;
    const float inv = use ? __fdiv_rn(127.f, top) : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) rows[g][64 * i + lane] = use ? (int8_t)(int)rintf(x[i] * inv) : (int8_t)0;
    if (lane == 0) tops[g] = use ? top : 0.f;
  }
  __syncthreads();
  const int32_t* table = s.table + (size_t)q.r * s.width;
  for (int j = tid; j < count; j += 256) {
    const int page = table[j];
    uint32_t key = 0;      // never chosen
    if (j < p.first || j > own - p.last) {
      key = 0xFFFFFFFFu;
    } else if (page >= 0 && page < p.index.num_pages) {
      const size_t at = (size_t)page * hkv + h;
      int code[D / 4];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const int4 x = reinterpret_cast<const int4*>(p.index.codes + at * D)[i];
        code[4 * i] = x.x, code[4 * i + 1] = x.y, code[4 * i + 2] = x.z, code[4 * i + 3] = x.w;
      }
      float most = -INFINITY;
      for (int g = 0; g < p.G; ++g) {
        int dot = 0;
#pragma unroll
        for (int i = 0; i < D / 4; ++i)
          dot = __builtin_amdgcn_sdot4(code[i], reinterpret_cast<const int*>(rows[g])[i], dot, false);
        most = fmaxf(most, (float)dot * tops[g]);
      }
      key = order_key(most * p.index.scales[at]);
    }
    keys[j] = key;
  }
  __syncthreads();
  if (wave != 0) return;
  // own pages behind the table are listed all the same: the attention makes such rows NaN
  const int beyond = min(max(own + 1 - max(s.width, own + 1 - p.last), 0), p.last);
  auto at_least = [&](uint32_t x) {
    int n = 0;
    for (int j = lane; j < count; j += 64) n += keys[j] >= x ? 1 : 0;
    return __builtin_amdgcn_readlane(wave_inclusive_scan(n), 63);
  };
  const int want = min(p.top_k - beyond, at_least(1u));
  uint32_t floor = 0;
  int above = 0;      // keys above the lowest chosen one
  if (want > 0) {
    for (int bit = 31; bit >= 0; --bit)
      if (at_least(floor | (1u << bit)) >= want) floor |= 1u << bit;
    above = floor == 0xFFFFFFFFu ? 0 : at_least(floor + 1);
  }
  int ties = want - above, filled = 0;
  for (int j0 = 0; j0 < count && filled < want; j0 += 64) {
    const uint32_t key = j0 + lane < count ? keys[j0 + lane] : 0;
    const bool tie = key == floor && key != 0;
    const uint64_t below = lane == 0 ? 0 : ~0ull >> (64 - lane), tied = __ballot(tie);
    const bool take = key > floor || (tie && __popcll(tied & below) < ties);
    const uint64_t taken = __ballot(take);
    if (take) out[filled + __popcll(taken & below)] = j0 + lane;
    filled += __popcll(taken);
    ties -= min(ties, (int)__popcll(tied));
  }
  for (int i = lane; i < p.top_k - want; i += 64) out[want + i] = i < beyond ? own + 1 - beyond + i : -1;
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
  with_head_dim(p.index.head_dim, [&](auto tag) {
    hipLaunchKernelGGL(kv_select_kernel<decltype(tag)::value>, dim3((unsigned)p.step.T, p.index.kv_heads), dim3(256), 0,
                       stream, p);
  });
  return launch_status();
}

}  // namespace moe
