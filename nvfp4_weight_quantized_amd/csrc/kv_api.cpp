// C ABI of the paged NVFP4 key/value cache: host-side validation, then the launches of kv_cache.hip
// and kv_attention.hip.  Nothing is enqueued on an error, nothing synchronises or allocates.
#include <hip/hip_runtime.h>

#include <cmath>

#include "common.h"

namespace {

using moe::al16;
using moe::check_arch;

bool valid_cache_dims(int64_t num_pages, int64_t page_size, int64_t kv_heads, int64_t head_dim) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return false;
  if (page_size <= 0 || page_size % moe::kKvUnit != 0 || page_size > 65536) return false;
  if (num_pages < 1 || kv_heads < 1 || kv_heads > 1024) return false;
  return num_pages * page_size < ((int64_t)1 << 31);
}

bool valid_gscale(float d) { return std::isfinite(d) && d >= 0x1p-64f && d <= 0x1p64f; }

bool valid_cache(const moe_nvfp4_kv_cache_t* c) {
  return c && valid_cache_dims(c->num_pages, c->page_size, c->kv_heads, c->head_dim) && valid_gscale(c->k_gscale) &&
         valid_gscale(c->v_gscale) && c->pages && al16(c->pages);
}

// A launch holds fewer than 2^32 work-items: the append one per 32 elements of the rows, up to 2^15 more, the gather 256
// per 32 rows.
constexpr int64_t kMaxAppend = (int64_t)1 << 36;
constexpr int32_t kMaxGather = (1 << 29) - 32;

bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

moe_status_t kv_attention(const moe_nvfp4_kv_cache_t* cache, const uint16_t* q, int64_t q_stride, int32_t T,
                          int32_t Hq, const int32_t* query_offsets, const int32_t* seq_lens, int32_t R,
                          const int32_t* block_table, int32_t table_width, float scale, int32_t window, uint16_t* out,
                          float* lse, bool fill, void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_cache(cache) || T < 0 || R < 0 || R > moe::kKvMaxRequests || table_width < 0)
    return MOE_ERR_INVALID_ARGUMENT;
  if (Hq < 1 || Hq % cache->kv_heads != 0 || Hq / cache->kv_heads > 64 || (int64_t)T * Hq >= ((int64_t)1 << 31))
    return MOE_ERR_INVALID_ARGUMENT;
  if ((int64_t)R * table_width >= ((int64_t)1 << 31)) return MOE_ERR_INVALID_ARGUMENT;
  if (!(std::isfinite(scale) && scale > 0.f) || window < 0) return MOE_ERR_INVALID_ARGUMENT;
  const float s = scale * cache->k_gscale;
  if (!(s >= 0x1p-126f && s <= 0x1p100f)) return MOE_ERR_INVALID_ARGUMENT;
  if (T > 1 && (q_stride < (int64_t)Hq * cache->head_dim || q_stride % 8 != 0)) return MOE_ERR_INVALID_ARGUMENT;
  if (T == 0 || (R == 0 && !fill)) return MOE_OK;
  if (!out || !al16(out)) return MOE_ERR_INVALID_ARGUMENT;
  if (R > 0 && (!q || !query_offsets || !seq_lens || !al16(q))) return MOE_ERR_INVALID_ARGUMENT;
  if (R > 0 && table_width > 0 && !block_table) return MOE_ERR_INVALID_ARGUMENT;
  const int64_t table_units = (int64_t)table_width * (cache->page_size / moe::kKvUnit);
  if (!moe::kv_attention_launchable(T, R, Hq, cache->kv_heads, cache->head_dim, table_units))
    return MOE_ERR_INVALID_ARGUMENT;
  const size_t need = moe::kv_attention_workspace(T, R, Hq, cache->kv_heads, cache->head_dim, table_units);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (need > 0 && !al16(workspace)) return MOE_ERR_INVALID_ARGUMENT;
  if (moe_status_t st = check_arch(nullptr)) return st;
  moe::KvAttentionProblem p{};
  p.cache = *cache;
  p.q = q;
  p.q_stride = q_stride;
  p.T = T;
  p.Hq = Hq;
  p.G = Hq / cache->kv_heads;
  p.offsets = query_offsets;
  p.lens = seq_lens;
  p.R = R;
  p.table = block_table;
  p.width = table_width;
  p.scale = s;
  p.window = window;
  p.out = out;
  p.lse = lse;
  p.fill = fill;
  return moe::launch_kv_attention(p, workspace, static_cast<hipStream_t>(stream));
}

}  // namespace

extern "C" {

size_t moe_nvfp4_kv_cache_bytes(int32_t num_pages, int32_t page_size, int32_t kv_heads, int32_t head_dim) {
  if (!valid_cache_dims(num_pages, page_size, kv_heads, head_dim)) return 0;
  return (size_t)num_pages * kv_heads * (page_size / moe::kKvUnit) * 36 * head_dim;
}

moe_status_t moe_kv_plan(const int32_t* kv_lens, const int32_t* new_lens, int32_t R, int32_t page_size,
                         int32_t num_pages, const int32_t* free_pages, int32_t num_free, int32_t* block_table,
                         int32_t table_width, int32_t num_tokens, int32_t* query_offsets, int32_t* seq_lens,
                         int32_t* positions, int32_t* slots, int32_t* pages_used, void* stream) {
  if (R < 0 || R > moe::kKvMaxRequests || num_tokens < 0 || num_free < 0 || table_width < 0)
    return MOE_ERR_INVALID_ARGUMENT;
  if (page_size <= 0 || page_size % moe::kKvUnit != 0 || page_size > 65536 || num_pages < 1 ||
      (int64_t)num_pages * page_size >= ((int64_t)1 << 31) || (int64_t)R * table_width >= ((int64_t)1 << 31))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!query_offsets || !pages_used || (R > 0 && (!kv_lens || !new_lens || !seq_lens)))
    return MOE_ERR_INVALID_ARGUMENT;
  if ((num_free > 0 && !free_pages) || (R > 0 && table_width > 0 && !block_table)) return MOE_ERR_INVALID_ARGUMENT;
  if (num_tokens > 0 && (!positions || !slots)) return MOE_ERR_INVALID_ARGUMENT;
  if (moe_status_t st = check_arch(nullptr)) return st;
  return moe::launch_kv_plan(kv_lens, new_lens, R, page_size, num_pages, free_pages, num_free, block_table,
                             table_width, num_tokens, query_offsets, seq_lens, positions, slots, pages_used,
                             static_cast<hipStream_t>(stream));
}

moe_status_t moe_nvfp4_kv_append(const moe_nvfp4_kv_cache_t* cache, const uint16_t* k, const uint16_t* v,
                                 int64_t k_stride, int64_t v_stride, const int32_t* slots, int32_t T, void* stream) {
  if (!valid_cache(cache) || T < 0) return MOE_ERR_INVALID_ARGUMENT;
  const int64_t row = (int64_t)cache->kv_heads * cache->head_dim;
  if (T > 1 && (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0))
    return MOE_ERR_INVALID_ARGUMENT;
  if (T * row > kMaxAppend) return MOE_ERR_INVALID_ARGUMENT;
  if (T == 0) return MOE_OK;
  if (!k || !v || !slots || !al16(k) || !al16(v) || !al4(slots)) return MOE_ERR_INVALID_ARGUMENT;
  if (moe_status_t st = check_arch(nullptr)) return st;
  return moe::launch_kv_append(*cache, k, v, k_stride, v_stride, slots, T, static_cast<hipStream_t>(stream));
}

moe_status_t moe_nvfp4_kv_gather(const moe_nvfp4_kv_cache_t* cache, const int32_t* slots, int32_t n, uint16_t* k,
                                 uint16_t* v, void* stream) {
  if (!valid_cache(cache) || n < 0 || n > kMaxGather) return MOE_ERR_INVALID_ARGUMENT;
  if (n == 0) return MOE_OK;
  if (!k || !v || !slots || !al16(k) || !al16(v) || !al4(slots)) return MOE_ERR_INVALID_ARGUMENT;
  if (moe_status_t st = check_arch(nullptr)) return st;
  return moe::launch_kv_gather(*cache, slots, n, k, v, static_cast<hipStream_t>(stream));
}

size_t moe_nvfp4_kv_attention_workspace_size(int32_t T, int32_t R, int32_t Hq, int32_t kv_heads, int32_t head_dim) {
  if (T < 0 || R < 0 || R > moe::kKvMaxRequests || Hq < 1 || kv_heads < 1 || Hq % kv_heads != 0 ||
      Hq / kv_heads > 64 || (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
      (int64_t)T * Hq >= ((int64_t)1 << 31))
    return 0;
  return moe::kv_attention_workspace(T, R, Hq, kv_heads, head_dim, INT64_MAX);      // any table
}

moe_status_t moe_nvfp4_kv_attention(const moe_nvfp4_kv_cache_t* cache, const uint16_t* q, int64_t q_stride, int32_t T,
                                    int32_t Hq, const int32_t* query_offsets, const int32_t* seq_lens, int32_t R,
                                    const int32_t* block_table, int32_t table_width, float scale, int32_t window,
                                    uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  return kv_attention(cache, q, q_stride, T, Hq, query_offsets, seq_lens, R, block_table, table_width, scale, window, out,
                      lse, false, workspace, workspace_bytes, stream);
}

moe_status_t moe_nvfp4_kv_attention_fill(const moe_nvfp4_kv_cache_t* cache, const uint16_t* q, int64_t q_stride, int32_t T,
                                         int32_t Hq, const int32_t* query_offsets, const int32_t* seq_lens, int32_t R,
                                         const int32_t* block_table, int32_t table_width, float scale, int32_t window,
                                         uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  return kv_attention(cache, q, q_stride, T, Hq, query_offsets, seq_lens, R, block_table, table_width, scale, window, out,
                      lse, true, workspace, workspace_bytes, stream);
}

}  // extern "C"
