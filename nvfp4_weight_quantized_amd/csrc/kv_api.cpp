// C ABI of the paged NVFP4 key/value cache and of rotary positions: host-side validation, then the launches of
// kv_cache.hip, rotary.hip, kv_index.hip, kv_sparse.hip and kv_attention.hip.  Nothing is enqueued on an error, nothing synchronises or allocates.
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

bool valid_index(const moe_nvfp4_kv_index_t* x) {
  return x && valid_cache_dims(x->num_pages, x->page_size, x->kv_heads, x->head_dim) && x->codes && x->scales &&
         al16(x->codes) && al4(x->scales);
}

// Offsets, lengths and table of a step of R > 0 requests.
bool valid_step(const moe::KvStep& s) {
  if (s.T < 0 || s.R < 0 || s.R > moe::kKvMaxRequests || s.width < 0) return false;
  if ((int64_t)s.R * s.width >= ((int64_t)1 << 31)) return false;
  if (s.R == 0 || s.T == 0) return true;
  return s.offsets && s.lens && (s.width == 0 || s.table) && al4(s.offsets) && al4(s.lens) && al4(s.table);
}

bool valid_rotary(const moe_rotary_t* r) {
  if (!r || r->head_dim < 16 || r->head_dim > 512 || r->head_dim % 16 != 0) return false;
  if (r->pairs < 8 || r->pairs % 8 != 0 || 2 * r->pairs > r->head_dim || r->axes < 1 || r->axes > 4) return false;
  if ((r->interleaved != 0 && r->interleaved != 1) || !std::isfinite(r->scale)) return false;
  return r->inv_freq && (reinterpret_cast<uintptr_t>(r->inv_freq) & 7) == 0 && al4(r->axis);
}

// Rows [T][heads][dim] and the token stride that reaches them.
bool valid_stride(int32_t T, int64_t stride, int64_t row) { return T <= 1 || (stride >= row && stride % 8 == 0); }

// Elements of the rows; that a launch holds fewer than 2^32 work-items is seen from the launch itself.
constexpr int64_t kMaxRotary = (int64_t)1 << 36, kMaxAppendRotary = (int64_t)1 << 35;

bool valid_rotary_rows(const moe_rotary_t& r, int64_t x_stride, int32_t T, int32_t heads, int64_t position_stride,
                       int64_t out_stride, int64_t most) {
  const int64_t row = (int64_t)heads * r.head_dim;
  if (T < 0 || heads < 1 || heads > 65536 || T * row > most || (int64_t)T >= (int64_t)1 << 24) return false;
  if (r.axes > 1 && position_stride < T) return false;
  return valid_stride(T, x_stride, row) && valid_stride(T, out_stride, row);
}

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

moe_status_t kv_sparse_attention(const moe_nvfp4_kv_cache_t* cache, const uint16_t* q, int64_t q_stride, int32_t T,
                                 int32_t Hq, const int32_t* query_offsets, const int32_t* seq_lens, int32_t R,
                                 const int32_t* block_table, int32_t table_width, const int32_t* selected,
                                 int32_t top_k, float scale, uint16_t* out, float* lse, bool fill,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_cache(cache)) return MOE_ERR_INVALID_ARGUMENT;
  const moe::KvStep step{query_offsets, seq_lens, block_table, R, T, table_width, cache->page_size};
  if (!valid_step(step)) return MOE_ERR_INVALID_ARGUMENT;
  if (Hq < 1 || Hq % cache->kv_heads != 0 || Hq / cache->kv_heads > 64 || (int64_t)T * Hq >= ((int64_t)1 << 31))
    return MOE_ERR_INVALID_ARGUMENT;
  if (top_k < 1 || top_k > moe::kKvMaxSelected) return MOE_ERR_INVALID_ARGUMENT;
  if (!(std::isfinite(scale) && scale > 0.f)) return MOE_ERR_INVALID_ARGUMENT;
  const float s = scale * cache->k_gscale;
  if (!(s >= 0x1p-126f && s <= 0x1p100f)) return MOE_ERR_INVALID_ARGUMENT;
  if (!valid_stride(T, q_stride, (int64_t)Hq * cache->head_dim)) return MOE_ERR_INVALID_ARGUMENT;
  const int32_t G = Hq / cache->kv_heads;
  if (!moe::kv_sparse_launchable(T, R, G, cache->kv_heads, cache->head_dim, cache->page_size, top_k))
    return MOE_ERR_INVALID_ARGUMENT;
  if (T == 0 || (R == 0 && !fill)) return MOE_OK;
  if (!out || !al16(out) || !al4(lse)) return MOE_ERR_INVALID_ARGUMENT;
  if (R > 0 && (!q || !al16(q) || !selected || !al4(selected))) return MOE_ERR_INVALID_ARGUMENT;
  const size_t need = moe::kv_sparse_workspace(T, R, G, cache->kv_heads, cache->head_dim, cache->page_size, top_k);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (need > 0 && !al16(workspace)) return MOE_ERR_INVALID_ARGUMENT;
  if (moe_status_t st = check_arch(nullptr)) return st;
  moe::KvSparseProblem p{};
  p.a.cache = *cache;
  p.a.q = q;
  p.a.q_stride = q_stride;
  p.a.T = T;
  p.a.Hq = Hq;
  p.a.G = G;
  p.a.offsets = query_offsets;
  p.a.lens = seq_lens;
  p.a.R = R;
  p.a.table = block_table;
  p.a.width = table_width;
  p.a.scale = s;
  p.a.out = out;
  p.a.lse = lse;
  p.a.fill = fill;
  p.selected = selected;
  p.top_k = top_k;
  return moe::launch_kv_sparse_attention(p, workspace, static_cast<hipStream_t>(stream));
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

moe_status_t moe_rotary(const moe_rotary_t* rotary, const uint16_t* x, int64_t x_stride, int32_t T, int32_t heads,
                        const int32_t* positions, int64_t position_stride, uint16_t* out, int64_t out_stride,
                        void* stream) {
  if (!valid_rotary(rotary) || !valid_rotary_rows(*rotary, x_stride, T, heads, position_stride, out_stride, kMaxRotary))
    return MOE_ERR_INVALID_ARGUMENT;
  if (T == 0) return MOE_OK;
  if (!x || !positions || !out || !al16(x) || !al16(out) || !al4(positions)) return MOE_ERR_INVALID_ARGUMENT;
  if (x == out && T > 1 && x_stride != out_stride) return MOE_ERR_INVALID_ARGUMENT;
  const moe::RotaryProblem p{*rotary, x, x_stride, T, heads, positions, position_stride, out, out_stride};
  if (!moe::rotary_launchable(p)) return MOE_ERR_INVALID_ARGUMENT;
  if (moe_status_t st = check_arch(nullptr)) return st;
  return moe::launch_rotary(p, static_cast<hipStream_t>(stream));
}

moe_status_t moe_nvfp4_kv_append_rotary(const moe_nvfp4_kv_cache_t* cache, const moe_rotary_t* rotary,
                                        const uint16_t* q, int64_t q_stride, int32_t Hq, const uint16_t* k,
                                        int64_t k_stride, const uint16_t* v, int64_t v_stride,
                                        const int32_t* positions, int64_t position_stride, const int32_t* slots,
                                        int32_t T, uint16_t* q_out, int64_t q_out_stride, void* stream) {
  if (!valid_cache(cache) || !valid_rotary(rotary) || rotary->head_dim != cache->head_dim)
    return MOE_ERR_INVALID_ARGUMENT;
  if (!valid_rotary_rows(*rotary, q_stride, T, Hq, position_stride, q_out_stride, kMaxAppendRotary))
    return MOE_ERR_INVALID_ARGUMENT;
  const int64_t row = (int64_t)cache->kv_heads * cache->head_dim;
  if (!valid_stride(T, k_stride, row) || !valid_stride(T, v_stride, row) || T * row > kMaxAppendRotary)
    return MOE_ERR_INVALID_ARGUMENT;
  if (T == 0) return MOE_OK;
  if (!q || !k || !v || !positions || !slots || !q_out) return MOE_ERR_INVALID_ARGUMENT;
  if (!al16(q) || !al16(k) || !al16(v) || !al16(q_out) || !al4(positions) || !al4(slots))
    return MOE_ERR_INVALID_ARGUMENT;
  if (q == q_out && T > 1 && q_stride != q_out_stride) return MOE_ERR_INVALID_ARGUMENT;
  const moe::RotaryProblem p{*rotary, q, q_stride, T, Hq, positions, position_stride, q_out, q_out_stride};
  if (!moe::kv_append_rotary_launchable(*cache, p)) return MOE_ERR_INVALID_ARGUMENT;
  if (moe_status_t st = check_arch(nullptr)) return st;
  return moe::launch_kv_append_rotary(*cache, p, k, v, k_stride, v_stride, slots, static_cast<hipStream_t>(stream));
}

moe_status_t moe_nvfp4_kv_index_update(const moe_nvfp4_kv_cache_t* cache, const moe_nvfp4_kv_index_t* index,
                                       const int32_t* query_offsets, const int32_t* seq_lens, int32_t R,
                                       const int32_t* block_table, int32_t table_width, int32_t T, void* stream) {
  if (!valid_cache(cache) || !valid_index(index)) return MOE_ERR_INVALID_ARGUMENT;
  if (index->num_pages != cache->num_pages || index->page_size != cache->page_size ||
      index->kv_heads != cache->kv_heads || index->head_dim != cache->head_dim)
    return MOE_ERR_INVALID_ARGUMENT;
  const moe::KvStep s{query_offsets, seq_lens, block_table, R, T, table_width, cache->page_size};
  if (!valid_step(s)) return MOE_ERR_INVALID_ARGUMENT;
  if ((T / cache->page_size + 2 * (int64_t)R) * cache->kv_heads >= (int64_t)1 << 24) return MOE_ERR_INVALID_ARGUMENT;
  if (T == 0 || R == 0 || table_width == 0) return MOE_OK;
  if (moe_status_t st = check_arch(nullptr)) return st;
  return moe::launch_kv_index_update(*cache, *index, s, static_cast<hipStream_t>(stream));
}

moe_status_t moe_nvfp4_kv_select(const moe_nvfp4_kv_index_t* index, const uint16_t* q, int64_t q_stride, int32_t T,
                                 int32_t Hq, const int32_t* query_offsets, const int32_t* seq_lens, int32_t R,
                                 const int32_t* block_table, int32_t table_width, int32_t top_k, int32_t first,
                                 int32_t last, int32_t* selected, void* stream) {
  if (!valid_index(index)) return MOE_ERR_INVALID_ARGUMENT;
  const moe::KvStep s{query_offsets, seq_lens, block_table, R, T, table_width, index->page_size};
  if (!valid_step(s) || table_width > moe::kKvMaxSelectPages) return MOE_ERR_INVALID_ARGUMENT;
  if (Hq < 1 || Hq % index->kv_heads != 0 || Hq / index->kv_heads > 64) return MOE_ERR_INVALID_ARGUMENT;
  if (!valid_stride(T, q_stride, (int64_t)Hq * index->head_dim)) return MOE_ERR_INVALID_ARGUMENT;
  if (top_k < 1 || top_k > moe::kKvMaxSelected || first < 0 || last < 1 || first > top_k || last > top_k - first)
    return MOE_ERR_INVALID_ARGUMENT;
  if ((int64_t)T * index->kv_heads > (int64_t)1 << 21) return MOE_ERR_INVALID_ARGUMENT;      // of 1024 threads each
  if (T == 0) return MOE_OK;
  if (!q || !al16(q) || !selected || !al4(selected)) return MOE_ERR_INVALID_ARGUMENT;
  if (moe_status_t st = check_arch(nullptr)) return st;
  const moe::KvSelectProblem p{*index, s, q, q_stride, Hq / index->kv_heads, top_k, first, last, selected};
  return moe::launch_kv_select(p, static_cast<hipStream_t>(stream));
}

size_t moe_nvfp4_kv_sparse_attention_workspace_size(int32_t T, int32_t R, int32_t Hq, int32_t kv_heads,
                                                    int32_t head_dim, int32_t page_size, int32_t top_k) {
  if (T < 0 || R < 0 || R > moe::kKvMaxRequests || Hq < 1 || kv_heads < 1 || Hq % kv_heads != 0 || Hq / kv_heads > 64 ||
      (int64_t)T * Hq >= ((int64_t)1 << 31) || top_k < 1 || top_k > moe::kKvMaxSelected ||
      !valid_cache_dims(1, page_size, kv_heads, head_dim))
    return 0;
  return moe::kv_sparse_workspace(T, R, Hq / kv_heads, kv_heads, head_dim, page_size, top_k);
}

moe_status_t moe_nvfp4_kv_sparse_attention(const moe_nvfp4_kv_cache_t* cache, const uint16_t* q, int64_t q_stride,
                                           int32_t T, int32_t Hq, const int32_t* query_offsets, const int32_t* seq_lens,
                                           int32_t R, const int32_t* block_table, int32_t table_width,
                                           const int32_t* selected, int32_t top_k, float scale, uint16_t* out,
                                           float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  return kv_sparse_attention(cache, q, q_stride, T, Hq, query_offsets, seq_lens, R, block_table, table_width, selected,
                             top_k, scale, out, lse, false, workspace, workspace_bytes, stream);
}

moe_status_t moe_nvfp4_kv_sparse_attention_fill(const moe_nvfp4_kv_cache_t* cache, const uint16_t* q, int64_t q_stride,
                                                int32_t T, int32_t Hq, const int32_t* query_offsets,
                                                const int32_t* seq_lens, int32_t R, const int32_t* block_table,
                                                int32_t table_width, const int32_t* selected, int32_t top_k, float scale,
                                                uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                                                void* stream) {
  return kv_sparse_attention(cache, q, q_stride, T, Hq, query_offsets, seq_lens, R, block_table, table_width, selected,
                             top_k, scale, out, lse, true, workspace, workspace_bytes, stream);
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
