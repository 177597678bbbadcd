// Attention over the paged NVFP4 key/value cache.
#include "kv_layout.h"

namespace moe {
namespace {

// Request of token t: the last r with offsets[r] <= t, or -1 where no request holds t.
__device__ __forceinline__ int kv_request_of(const int32_t* __restrict__ offsets, int R, int t) {
  if (t < offsets[0] || t >= offsets[R]) return -1;
  int lo = 0, hi = R;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (offsets[mid] <= t) lo = mid;
    else hi = mid;
  }
  return t < offsets[lo + 1] ? lo : -1;
}

// One wave per (token, query head): lane l takes the keys l, l + 64, ... in a first pass for the
// maximum, in a second for the sum, then the lanes take the output elements.
template <int D>
__global__ __launch_bounds__(64) void kv_attention_simple_kernel(KvAttentionProblem a) {
  using U = KvUnit<D>;
  const int t = blockIdx.x, hq = blockIdx.y, h = hq / a.G, lane = threadIdx.x;
  const int r = kv_request_of(a.offsets, a.R, t);
  if (r < 0) return;
  const int n = a.offsets[r + 1] - a.offsets[r];
  const int pos = a.lens[r] - n + (t - a.offsets[r]);
  const int first = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  const uint16_t* qr = a.q + t * a.q_stride + (size_t)hq * D;
  __shared__ float q[D];
  for (int d = lane; d < D; d += 64) q[d] = bf16_to_f32(qr[d]);
  __syncthreads();
  const int ps = a.cache.page_size;
  auto unit_of = [&](int j) -> const uint8_t* {
    const int b = j / ps;
    const int page = b < a.width ? a.table[(size_t)r * a.width + b] : -1;
    if (page < 0 || page >= a.cache.num_pages) return nullptr;
    return a.cache.pages + kv_unit_offset<D>(a.cache, page * ps + j % ps, h);
  };
  constexpr float kMag[8] = {0.f, 0.5f, 1.f, 1.5f, 2.f, 3.f, 4.f, 6.f};
  auto value = [&](uint32_t code) { return (code & 8u) ? -kMag[code & 7u] : kMag[code & 7u]; };
  auto score = [&](int j) -> float {
    const uint8_t* u = unit_of(j);
    if (!u) return NAN;
    const int p = j % kKvUnit;
    float s = 0.f;
    for (int g = 0; g < D / 16; ++g) {
      float x = 0.f;
      for (int e = 0; e < 16; ++e) {
        const uint8_t byte = u[U::k_word(p, 2 * g + (e >> 3)) + ((e & 7) >> 1)];
        x += q[16 * g + e] * value((e & 1) ? byte >> 4 : byte & 15u);
      }
      s += x * __builtin_amdgcn_cvt_f32_fp8((int)u[U::k_scale(p, g)], 0);
    }
    return s * a.scale;
  };
  float m = -INFINITY;
  bool bad = false;
  for (int j = first + lane; j <= pos; j += 64) {
    const float s = score(j);
    bad |= !(s == s);
    m = fmaxf(m, s);
  }
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
  bad = __any(bad);
  float o[D / 64] = {}, l = 0.f;
  if (!bad && m > -INFINITY) {
    for (int j0 = first; j0 <= pos; j0 += 64) {
      const int j = j0 + lane;
      const float pj = j <= pos ? expf(score(j) - m) : 0.f;
      l += pj;
      for (int i = 0; i < 64 && j0 + i <= pos; ++i) {
        const float w = __shfl(pj, i);
        const uint8_t* u = unit_of(j0 + i);
        const int p = (j0 + i) % kKvUnit;
        for (int e = 0; e < D / 64; ++e) {
          const int d = lane + 64 * e;
          const uint8_t byte = u[U::v_byte(p, d >> 1)];
          o[e] += w * value((d & 1) ? byte >> 4 : byte & 15u) *
                  __builtin_amdgcn_cvt_f32_fp8((int)u[U::v_scale(p, d >> 4)], 0);
        }
      }
    }
    for (int off = 32; off >= 1; off >>= 1) l += __shfl_xor(l, off);
  }
  for (int e = 0; e < D / 64; ++e)
    a.out[((size_t)t * a.Hq + hq) * D + lane + 64 * e] =
        f32_to_bf16(bad ? NAN : l > 0.f ? o[e] / l * a.cache.v_gscale : 0.f);
  if (a.lse && lane == 0) a.lse[(size_t)t * a.Hq + hq] = bad ? NAN : l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t kv_attention_workspace(int32_t, int32_t, int32_t, int32_t, int32_t) { return 0; }

moe_status_t launch_kv_attention(const KvAttentionProblem& p, void*, hipStream_t stream) {
  if (p.Hq > 65535) return MOE_ERR_INVALID_ARGUMENT;
  with_head_dim(p.cache.head_dim, [&](auto tag) {
    hipLaunchKernelGGL(kv_attention_simple_kernel<decltype(tag)::value>, dim3(p.T, p.Hq), dim3(64), 0, stream, p);
  });
  return launch_status();
}

}  // namespace moe
