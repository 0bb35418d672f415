// paged_api.cu -- the paged entry points of include/lsx.h: argument checks,
// workspace sizes and dispatch.  Every check runs before any launch.
#include "checks.h"
#include "paged.h"

namespace lsx {
namespace {

// The checks of sizes alone, which the calls share with their workspace sizes
// (those are asked for before a call is checked, with any numbers).

// pages [P, Hkv, page, D]
int check_page_sizes(const lsx_tensor& kp) {
  if (kp.B <= 0 || kp.H <= 0 || kp.N < 0 || kp.D <= 0) return LSX_ERR_SHAPE;
  if (kp.D != 64 && kp.D != 128) return LSX_ERR_UNSUPPORTED;
  if (kp.N < kMinPage || kp.N > kMaxPage || (kp.N & (kp.N - 1)) != 0) return LSX_ERR_UNSUPPORTED;
  if (kp.B >= (int64_t{1} << 31) || kp.H >= (1 << 16)) return LSX_ERR_UNSUPPORTED;
  return LSX_OK;
}

// q [B, Hq, N, D], the query heads a multiple of the cache's.
int check_query_sizes(const lsx_tensor& q, const lsx_tensor& kp) {
  if (q.B <= 0 || q.H <= 0 || q.N < 0) return LSX_ERR_SHAPE;
  if (q.D != kp.D || q.H % kp.H != 0) return LSX_ERR_SHAPE;
  const int64_t lim = int64_t{1} << 31;
  if (q.N >= lim || q.H >= (1 << 16) || q.B >= (1 << 16)) return LSX_ERR_UNSUPPORTED;
  return LSX_OK;
}

// What a table row can hold: positions, rounded up to a tile, are 32-bit.
int check_table_size(int64_t max_pages, int64_t page) {
  if (max_pages < 0) return LSX_ERR_SHAPE;
  if (max_pages >= (int64_t{1} << 31) || max_pages * page > (int64_t{1} << 31) - 2 * kMaxPage)
    return LSX_ERR_UNSUPPORTED;
  return LSX_OK;
}

int check_decode_rows(const lsx_tensor& q, const lsx_tensor& kp) {
  if (q.N < 1) return LSX_ERR_SHAPE;
  return q.H / kp.H * q.N > kMaxDecodeRows ? LSX_ERR_UNSUPPORTED : LSX_OK;
}

int check_prefix_size(int64_t prefix_len) {
  if (prefix_len < 0) return LSX_ERR_SHAPE;
  return prefix_len > (int64_t{1} << 31) - 2 * kMaxPage ? LSX_ERR_UNSUPPORTED : LSX_OK;
}

int check_prompt_sizes(const lsx_tensor& q, const lsx_tensor& kp, int64_t batch) {
  if (q.B != 1 || batch <= 0) return LSX_ERR_SHAPE;
  return batch > kMaxMapBatch || q.H / kp.H > 128 ? LSX_ERR_UNSUPPORTED : LSX_OK;
}

// keys and values in pages, bf16, the same shape.
int check_pages(const lsx_tensor* kp, const lsx_tensor* vp) {
  LSX_TRY(check_view(kp));
  LSX_TRY(check_view(vp));
  if (kp->data == nullptr || vp->data == nullptr) return LSX_ERR_NULL;
  if (kp->dtype != LSX_BF16 || vp->dtype != LSX_BF16) return LSX_ERR_DTYPE;
  if (!same_bhn_d(kp, vp)) return LSX_ERR_SHAPE;
  LSX_TRY(check_page_sizes(*kp));
  LSX_TRY(check_row_aligned(kp));
  LSX_TRY(check_row_aligned(vp));
  return LSX_OK;
}

// q, o [B, Hq, N, D] (q bf16, o bf16 or f32), lse [B, Hq, N, 1].
int check_queries(const lsx_tensor* q, const lsx_tensor* kp, const lsx_tensor* o,
                  const lsx_tensor* lse) {
  LSX_TRY(check_view(q));
  LSX_TRY(check_view(o));
  if (q->dtype != LSX_BF16) return LSX_ERR_DTYPE;
  if (!same_bhn_d(q, o)) return LSX_ERR_SHAPE;
  LSX_TRY(check_query_sizes(*q, *kp));
  LSX_TRY(check_row_aligned(q));
  LSX_TRY(check_row_aligned(o));
  if (q->N == 0) return LSX_OK;
  return check_lse(lse, q);
}

int check_ints(const void* p) {
  if (p == nullptr) return LSX_ERR_NULL;
  return reinterpret_cast<uintptr_t>(p) % 4 == 0 ? LSX_OK : LSX_ERR_ALIGN;
}

// block table [batch][max_pages], rows table_stride apart
int check_table(const int32_t* table, int64_t table_stride, int64_t max_pages, int64_t page) {
  if (table_stride < max_pages) return LSX_ERR_SHAPE;
  LSX_TRY(check_table_size(max_pages, page));
  return max_pages == 0 ? LSX_OK : check_ints(table);
}

int check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return LSX_OK;
  if (ws == nullptr || have < need) return LSX_ERR_WORKSPACE;
  return reinterpret_cast<uintptr_t>(ws) % 256 == 0 ? LSX_OK : LSX_ERR_ALIGN;
}

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a_bytes > 0 && b_bytes > 0 && x < y + static_cast<uintptr_t>(b_bytes) &&
         y < x + static_cast<uintptr_t>(a_bytes);
}

int sm_count_or(int fallback) {
  DeviceCtx ctx;
  return device_ctx(&ctx) == LSX_OK ? ctx.sm_count : fallback;
}

constexpr int kSmFallback = 152;  // sizes are asked for where no device is

}  // namespace
}  // namespace lsx

using namespace lsx;

extern "C" {

int attn_page_map(const int32_t* ctx_lens, const int32_t* new_lens, int64_t batch,
                  const int32_t* free_pages, int64_t n_free, int64_t page_size,
                  int32_t* block_table, int64_t table_stride, int64_t max_pages,
                  int64_t* slot_map, int64_t n_tokens, int32_t* cu_new, int32_t* kv_lens,
                  int32_t* taken, lsx_stream_t stream) {
  if (batch <= 0 || n_free < 0 || n_tokens < 0) return LSX_ERR_SHAPE;
  if (batch > kMaxMapBatch || n_tokens >= (int64_t{1} << 31) || n_free >= (int64_t{1} << 31))
    return LSX_ERR_UNSUPPORTED;
  if (page_size < kMinPage || page_size > kMaxPage || (page_size & (page_size - 1)) != 0)
    return LSX_ERR_UNSUPPORTED;
  LSX_TRY(check_table(block_table, table_stride, max_pages, page_size));
  LSX_TRY(check_ints(ctx_lens));
  LSX_TRY(check_ints(new_lens));
  LSX_TRY(check_ints(cu_new));
  LSX_TRY(check_ints(kv_lens));
  LSX_TRY(check_ints(taken));
  if (n_free > 0) LSX_TRY(check_ints(free_pages));
  if (n_tokens > 0) {
    if (slot_map == nullptr) return LSX_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(slot_map) % 8 != 0) return LSX_ERR_ALIGN;
  }
  // thread blocks write results while others still read the inputs
  const struct { const void* at; int64_t bytes; }
      in[] = {{ctx_lens, 4 * batch}, {new_lens, 4 * batch}, {free_pages, 4 * n_free}},
      out[] = {{block_table, 4 * ((batch - 1) * table_stride + max_pages)},
               {slot_map, 8 * n_tokens}, {cu_new, 4 * (batch + 1)}, {kv_lens, 4 * batch}, {taken, 4}};
  for (const auto& i : in)
    for (const auto& o : out)
      if (overlap(i.at, i.bytes, o.at, o.bytes)) return LSX_ERR_UNSUPPORTED;
  DeviceCtx ctx;
  LSX_TRY(device_ctx(&ctx));
  return launch_page_map(ctx_lens, new_lens, batch, free_pages, n_free, page_size, block_table,
                         table_stride, max_pages, slot_map, n_tokens, cu_new, kv_lens, taken, ctx,
                         as_stream(stream));
}

int attn_page_append(const lsx_tensor* k, const lsx_tensor* v, const int64_t* slot_map,
                     const lsx_tensor* k_pages, const lsx_tensor* v_pages, lsx_stream_t stream) {
  LSX_TRY(check_pages(k_pages, v_pages));
  LSX_TRY(check_view(k));
  LSX_TRY(check_view(v));
  if (k->dtype != v->dtype) return LSX_ERR_DTYPE;
  if (k->B != 1 || !same_bhn_d(k, v) || k->H != k_pages->H || k->D != k_pages->D)
    return LSX_ERR_SHAPE;
  if (k->N >= (int64_t{1} << 31)) return LSX_ERR_UNSUPPORTED;
  LSX_TRY(check_row_aligned(k));
  LSX_TRY(check_row_aligned(v));
  if (k->N == 0) return LSX_OK;
  if (slot_map == nullptr) return LSX_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(slot_map) % 8 != 0) return LSX_ERR_ALIGN;
  DeviceCtx ctx;
  LSX_TRY(device_ctx(&ctx));
  return launch_page_append(*k, *v, slot_map, *k_pages, *v_pages, ctx, as_stream(stream));
}

size_t attn_paged_decode_workspace_size(const lsx_tensor* q, const lsx_tensor* k_pages,
                                        int64_t max_pages, int64_t prefix_len) {
  if (q == nullptr || k_pages == nullptr || check_page_sizes(*k_pages) != LSX_OK ||
      check_query_sizes(*q, *k_pages) != LSX_OK || check_decode_rows(*q, *k_pages) != LSX_OK ||
      check_table_size(max_pages, k_pages->N) != LSX_OK || check_prefix_size(prefix_len) != LSX_OK)
    return 0;  // the call itself is refused, and says why
  return paged_decode_workspace(*q, *k_pages, max_pages, prefix_len, sm_count_or(kSmFallback));
}

int attn_paged_decode(const lsx_tensor* q, const lsx_tensor* k_pages, const lsx_tensor* v_pages,
                      const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                      const int32_t* kv_lens, const int32_t* prefix_table, int64_t prefix_len,
                      float scale, const lsx_tensor* o, const lsx_tensor* lse, void* workspace,
                      size_t workspace_bytes, lsx_stream_t stream) {
  LSX_TRY(check_pages(k_pages, v_pages));
  LSX_TRY(check_queries(q, k_pages, o, lse));
  LSX_TRY(check_decode_rows(*q, *k_pages));
  LSX_TRY(check_table(block_table, table_stride, max_pages, k_pages->N));
  LSX_TRY(check_ints(kv_lens));
  LSX_TRY(check_prefix_size(prefix_len));
  if (prefix_len > 0) LSX_TRY(check_ints(prefix_table));
  LSX_TRY(check_ws(workspace, workspace_bytes,
                   attn_paged_decode_workspace_size(q, k_pages, max_pages, prefix_len)));
  DeviceCtx ctx;
  LSX_TRY(device_ctx(&ctx));
  const PagedCache c = paged_cache(*k_pages, *v_pages, block_table, table_stride, max_pages);
  return launch_paged_decode(*q, *k_pages, *v_pages, c, kv_lens, prefix_table, prefix_len,
                             resolve_scale(scale, q->D), *o, *lse, workspace, ctx,
                             as_stream(stream));
}

size_t attn_paged_fwd_workspace_size(const lsx_tensor* q, const lsx_tensor* k_pages,
                                     int64_t batch, int64_t max_pages) {
  if (q == nullptr || k_pages == nullptr || check_page_sizes(*k_pages) != LSX_OK ||
      check_query_sizes(*q, *k_pages) != LSX_OK ||
      check_prompt_sizes(*q, *k_pages, batch) != LSX_OK ||
      check_table_size(max_pages, k_pages->N) != LSX_OK)
    return 0;  // the call itself is refused, and says why
  return paged_fwd_workspace(*q, *k_pages, batch, max_pages, sm_count_or(kSmFallback));
}

int attn_paged_fwd(const lsx_tensor* q, const lsx_tensor* k_pages, const lsx_tensor* v_pages,
                   const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                   const int32_t* kv_lens, const int32_t* cu_q, int64_t batch, float scale,
                   const lsx_tensor* o, const lsx_tensor* lse, void* workspace,
                   size_t workspace_bytes, lsx_stream_t stream) {
  LSX_TRY(check_pages(k_pages, v_pages));
  LSX_TRY(check_queries(q, k_pages, o, lse));
  LSX_TRY(check_prompt_sizes(*q, *k_pages, batch));
  LSX_TRY(check_table(block_table, table_stride, max_pages, k_pages->N));
  LSX_TRY(check_ints(kv_lens));
  LSX_TRY(check_ints(cu_q));
  if (q->N == 0) return LSX_OK;
  LSX_TRY(check_ws(workspace, workspace_bytes,
                   attn_paged_fwd_workspace_size(q, k_pages, batch, max_pages)));
  DeviceCtx ctx;
  LSX_TRY(device_ctx(&ctx));
  const PagedCache c = paged_cache(*k_pages, *v_pages, block_table, table_stride, max_pages);
  return launch_paged_fwd(*q, *k_pages, *v_pages, c, kv_lens, cu_q, batch,
                          resolve_scale(scale, q->D), *o, *lse, workspace, ctx,
                          as_stream(stream));
}

}  // extern "C"
