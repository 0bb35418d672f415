// paged.h -- what the paged-cache kernels share: the view of a cache kept in
// pages and the launchers of the paged entry points.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>

#include "internal.h"

namespace lsx {

constexpr int kMaxMapBatch = 4096;   // sequences one page map handles
constexpr int kMaxDecodeRows = 64;   // query rows per kv head and sequence
constexpr int64_t kMinPage = 16, kMaxPage = 256;

// device status: a page number outside the cache, or a length beyond the
// block table (mirrors LSX_ERR_PAGE)
constexpr int kStatusPage = -10;

// Keys and values in pages: row n of page g and kv head h starts at element
// g * sp + h * sh + n * sn.  Position i of sequence b lives in page
// table[b * table_stride + (i >> shift)], row i & (page - 1).
struct PagedCache {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t k_sp, k_sh, k_sn, v_sp, v_sh, v_sn;
  int32_t n_pages;
  int shift;
  const int32_t* table;
  int64_t table_stride;
  int32_t max_pages;
};

inline PagedCache paged_cache(const lsx_tensor& kp, const lsx_tensor& vp, const int32_t* table,
                              int64_t table_stride, int64_t max_pages) {
  PagedCache c;
  c.k = static_cast<const __nv_bfloat16*>(kp.data);
  c.v = static_cast<const __nv_bfloat16*>(vp.data);
  c.k_sp = kp.stride_b; c.k_sh = kp.stride_h; c.k_sn = kp.stride_n;
  c.v_sp = vp.stride_b; c.v_sh = vp.stride_h; c.v_sn = vp.stride_n;
  c.n_pages = static_cast<int32_t>(kp.B);
  c.shift = 0;
  while ((int64_t{1} << c.shift) < kp.N) ++c.shift;
  c.table = table;
  c.table_stride = table_stride;
  c.max_pages = static_cast<int32_t>(max_pages);
  return c;
}

// Raises a kernel's dynamic shared memory limit, once per device (`done`: a
// static of the kernel's launcher, a bit per device; setting it twice is
// harmless).
template <typename Kernel>
inline bool allow_smem(Kernel kern, int bytes, int device, std::atomic<uint64_t>& done) {
  const uint64_t bit = device < 64 ? uint64_t{1} << device : 0;
  if ((done.load(std::memory_order_acquire) & bit) != 0) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return false;
  done.fetch_or(bit, std::memory_order_release);
  return true;
}

int launch_page_map(const int32_t* ctx_lens, const int32_t* new_lens, int64_t batch,
                    const int32_t* free_pages, int64_t n_free, int64_t page_size,
                    int32_t* block_table, int64_t table_stride, int64_t max_pages,
                    int64_t* slot_map, int64_t n_tokens, int32_t* cu_new, int32_t* kv_lens,
                    int32_t* taken, const DeviceCtx& ctx, cudaStream_t s);
int launch_page_append(const lsx_tensor& k, const lsx_tensor& v, const int64_t* slot_map,
                       const lsx_tensor& k_pages, const lsx_tensor& v_pages,
                       const DeviceCtx& ctx, cudaStream_t s);

// Single-token (and draft-token) attention over the pages; prefix_table NULL
// or the pages of prefix_len keys that every sequence sees first.
size_t paged_decode_workspace(const lsx_tensor& q, const lsx_tensor& k_pages, int64_t max_pages,
                              int64_t prefix_len, int sm_count);
int launch_paged_decode(const lsx_tensor& q, const lsx_tensor& k_pages, const lsx_tensor& v_pages,
                        const PagedCache& c, const int32_t* kv_lens, const int32_t* prefix_table, int64_t prefix_len,
                        float scale, const lsx_tensor& o, const lsx_tensor& lse, void* workspace,
                        const DeviceCtx& ctx, cudaStream_t s);
// Partials of every decode query against a prefix that all of them see, on
// the prompt kernel: piece i of the row that is token (b, n) of head g of kv head
// hk is row ((b / (2 tpt) * pieces + i) * Hkv + hk) * 256 + (b / tpt % 2) * 128 +
// ((b % tpt) * Nq + n) * G + g of o [rows][D] and l [rows].  split_p: P to 16 bits
// (else bf16).
struct PrefixPlan {
  int tpt, pieces, size;  // sequences of a row tile; pieces of the prefix, key tiles each
  int64_t rows;           // of all pieces
};
PrefixPlan prefix_plan(int64_t B, int64_t per, int64_t hkv, int64_t prefix_len, int sm_count);
int launch_prefix(const lsx_tensor& q, const lsx_tensor& k_pages, const lsx_tensor& v_pages,
                  const PagedCache& prefix, int64_t prefix_len, const PrefixPlan& plan,
                  float scale, bool split_p, float* part_o, float* part_l,
                  const DeviceCtx& ctx, cudaStream_t s);
// Ragged prompt tokens, causal, over the pages.
size_t paged_fwd_workspace(const lsx_tensor& q, const lsx_tensor& k_pages, int64_t batch,
                           int64_t max_pages, int sm_count);
int launch_paged_fwd(const lsx_tensor& q, const lsx_tensor& k_pages, const lsx_tensor& v_pages,
                     const PagedCache& c, const int32_t* kv_lens, const int32_t* cu_q,
                     int64_t batch, float scale, const lsx_tensor& o, const lsx_tensor& lse,
                     void* workspace, const DeviceCtx& ctx, cudaStream_t s);

}  // namespace lsx
