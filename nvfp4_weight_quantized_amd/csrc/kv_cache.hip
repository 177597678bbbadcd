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
// the entries read (pages held) are never written.  Bound by latency: two rounds of memory, a scan over 16
// waves and a search of log2 R steps, 5.7 us for 64 requests, 6.7 us for 512 with 25000 tokens (a launch alone
// takes about 3 us); one launch, because a second one for the tokens would cost more than the prefix sums
// that every workgroup repeats.
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
// One thread per (window of W consecutive rows, head, K or V, 16-element group).  The value codes of four
// positions 4c..4c+3 share dwords, so W = 4 quantizes such a quad together and stores dwords: the thread
// takes every quad that begins among its W rows (a row whose slot is a multiple of 4 or does not follow
// the row before it), with the rows after it that continue it, also those of the next window.  W = 1
// stores bytes, row by row: for steps of few rows, where the threads of the quads would not fill the card.
// Measured with 8 heads of 128, W = 4 against W = 1, rows of one request from a position that is a multiple of 4 / from
// another / at scattered slots, where W = 4 takes its rows one after the other: 2048 rows 7.7 against 8.0 / 9.1 against
// 8.2 / 11.5 against 8.9 us, 4096 rows 10.3 against 12.3 / 11.2 against 12.4 / 14.6 against 13.3 us, 8192 rows 14.3
// against 20.0 / 15.4 against 20.2 / 30.6 against 25.8 us.  The host does not see the slots: the rule is for those of
// prompts, which such steps mostly hold.
// Bound by the vector unit and the memory one after the other: 14.3 us for 8192 rows of 8 heads of 128 (16 us with
// other work in the caches), of which about 335 instructions per group (32 of them the second quotient step) make 9 us
// and the 43 MB at the rate of a copy 8.3 us.  It is one round of four waves per SIMD, and each begins with loads of
// slots that wait for one another before its rows are asked for.  Putting whole units together in LDS and writing them
// in order took 20.8 us: the scattered stores are not what it waits for.
constexpr long long kAppendQuadThreads = 1 << 19;      // rows * groups from which quads are taken

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

template <int D, int W>
__global__ __launch_bounds__(256) void kv_append_kernel(moe_nvfp4_kv_cache_t c, const uint16_t* __restrict__ k,
                                                        const uint16_t* __restrict__ v, int64_t k_stride,
                                                        int64_t v_stride, const int32_t* __restrict__ slots, int T) {
  using U = KvUnit<D>;
  constexpr int NG = D / 16;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int per = 2 * c.kv_heads * NG;
  const long long wl = i / per;
  if (wl * W >= T) return;
  const int t0 = (int)wl * W, rest = (int)(i % per);
  const int g = rest % NG, h = (rest / NG) % c.kv_heads;
  const bool is_v = rest / NG >= c.kv_heads;
  const int cap = c.num_pages * c.page_size;
  const uint16_t* src = (is_v ? v : k) + h * D + g * 16;
  const int64_t stride = is_v ? v_stride : k_stride;
  const float d = is_v ? c.v_gscale : c.k_gscale;
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
        load_group16(src + (int64_t)(t + r) * stride, x);
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

// ------------------------------------------------------------------------------------ gather
// A workgroup takes 32 rows of the list for one head.  Where they lie in at most two units (consecutive
// positions, whatever their alignment), both units come to LDS whole and in order and every thread
// assembles 16-byte pieces of the output rows from there; otherwise the pieces are assembled from global
// memory.  Bound by memory: 32768 rows of 8 heads of 128 (172 MB) in 33.4 us, 5.16 TB/s, the rate of a copy
// (with stores that stay in the caches 36.1 us).
constexpr int kGatherRows = 32;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <int D>
__global__ __launch_bounds__(256) void kv_gather_kernel(moe_nvfp4_kv_cache_t c, const int32_t* __restrict__ slots,
                                                        int n, uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
  using U = KvUnit<D>;
  __shared__ __align__(16) uint8_t lds[2 * U::kBytes];
  __shared__ int row_slot[kGatherRows];
  const int tid = threadIdx.x, lane = tid & 63, h = blockIdx.y;
  const int t0 = blockIdx.x * kGatherRows, rows = min(kGatherRows, n - t0);
  const int cap = c.num_pages * c.page_size;
  // every wave: lane r holds row r's slot (-1 outside the cache)
  int slot = -1;
  if (lane < rows) slot = slots[t0 + lane];
  if (slot < 0 || slot >= cap) slot = -1;
  if (tid < kGatherRows) row_slot[tid] = slot;
  const uint64_t have = __ballot(slot >= 0);
  int ua = 0, ub = 0;          // units of the first and the last row inside the cache
  if (have) {
    ua = __builtin_amdgcn_readlane(slot, __ffsll((unsigned long long)have) - 1) / kKvUnit;
    ub = __builtin_amdgcn_readlane(slot, 63 - __clzll((long long)have)) / kKvUnit;
  }
  const int unit = slot / kKvUnit;
  const bool two = !__any(slot >= 0 && unit != ua && unit != ub) && rows > 1;
  if (two) {
    const uint8_t* pa = c.pages + kv_unit_offset<D>(c, ua * kKvUnit, h);
    const uint8_t* pb = c.pages + kv_unit_offset<D>(c, ub * kKvUnit, h);
    for (int i = tid; i < U::kBytes / 16; i += 256) {
      reinterpret_cast<uint4*>(lds)[i] = reinterpret_cast<const uint4*>(pa)[i];
      if (ub != ua) reinterpret_cast<uint4*>(lds + U::kBytes)[i] = reinterpret_cast<const uint4*>(pb)[i];
    }
  }
  __syncthreads();
  // pieces of eight elements: D / 8 per row of K, then of V
  constexpr int PIECES = D / 8;
  for (int i = tid; i < 2 * rows * PIECES; i += 256) {
    const bool is_v = i >= rows * PIECES;
    const int x = is_v ? i - rows * PIECES : i, r = x / PIECES, g8 = x % PIECES;
    const int s = row_slot[r];
    uint32_t w[4];
    if (s < 0) {
#pragma unroll
      for (int b = 0; b < 4; ++b) w[b] = 0x7FC07FC0u;
    } else {
      const uint8_t* u = two ? lds + (s / kKvUnit == ua ? 0 : U::kBytes) : c.pages + kv_unit_offset<D>(c, s, h);
      const int p = s % kKvUnit;
      uint32_t codes;
      if (is_v)
        codes = (uint32_t)u[U::v_byte(p, 4 * g8)] | ((uint32_t)u[U::v_byte(p, 4 * g8 + 1)] << 8) |
                ((uint32_t)u[U::v_byte(p, 4 * g8 + 2)] << 16) | ((uint32_t)u[U::v_byte(p, 4 * g8 + 3)] << 24);
      else
        codes = *reinterpret_cast<const uint32_t*>(u + U::k_word(p, g8));
      const float sc = __builtin_amdgcn_cvt_f32_fp8((int)u[is_v ? U::v_scale(p, g8 >> 1) : U::k_scale(p, g8 >> 1)], 0);
      const float d = is_v ? c.v_gscale : c.k_gscale;
      const f32x2 e[4] = {
          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1),
          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3)};
#pragma unroll
      for (int b = 0; b < 4; ++b) w[b] = f32x2_to_bf16x2(e[b][0] * sc * d, e[b][1] * sc * d);
    }
    uint16_t* dst = (is_v ? v : k) + ((size_t)(t0 + r) * c.kv_heads + h) * D + 8 * g8;
    __builtin_nontemporal_store(u32x4{w[0], w[1], w[2], w[3]}, reinterpret_cast<u32x4*>(dst));
  }
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
  const long long per = 2LL * c.kv_heads * (c.head_dim / 16);
  const bool quads = T * per >= kAppendQuadThreads;
  const long long total = (quads ? (T + 3LL) / 4 : T) * per, blocks = (total + 255) / 256;
  with_head_dim(c.head_dim, [&](auto tag) {
    constexpr int D = decltype(tag)::value;
    if (quads)
      hipLaunchKernelGGL((kv_append_kernel<D, 4>), dim3((unsigned)blocks), dim3(256), 0, stream, c, k, v, k_stride,
                         v_stride, slots, T);
    else
      hipLaunchKernelGGL((kv_append_kernel<D, 1>), dim3((unsigned)blocks), dim3(256), 0, stream, c, k, v, k_stride,
                         v_stride, slots, T);
  });
  return launch_status();
}

moe_status_t launch_kv_gather(const moe_nvfp4_kv_cache_t& c, const int32_t* slots, int32_t n, uint16_t* k,
                              uint16_t* v, hipStream_t stream) {
  with_head_dim(c.head_dim, [&](auto tag) {
    hipLaunchKernelGGL(kv_gather_kernel<decltype(tag)::value>,
                       dim3((unsigned)(((int64_t)n + kGatherRows - 1) / kGatherRows), c.kv_heads), dim3(256), 0, stream,
                       c, slots, n, k, v);
  });
  return launch_status();
}

}  // namespace moe
