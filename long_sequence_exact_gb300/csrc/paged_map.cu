// paged_map.cu -- the bookkeeping of a key/value cache kept in pages: which
// pages a step's new tokens take, where each token's row goes, and the write
// of the rows themselves.
#include <cuda_bf16.h>

#include "paged.h"
#include "ptx.cuh"

namespace lsx {
namespace {

constexpr int kMapThreads = 256;

struct MapParams {
  const int32_t* ctx;
  const int32_t* add;
  int batch;
  const int32_t* free_pages;
  int64_t n_free;
  int shift;
  int32_t* table;
  int64_t table_stride;
  int64_t max_pages;
  int64_t* slots;
  int64_t n_tokens;
  int32_t* cu;
  int32_t* kv_lens;
  int32_t* taken;
};

// A sequence's keys before and after the step: negative counts as none, and the
// sum stays where rounding it up to a page does not overflow.
constexpr int32_t kMostKeys = 0x7ffffe00;
__device__ __forceinline__ int32_t keys_before(const MapParams& p, int b) {
  const int32_t c = p.ctx[b];
  return c < 0 ? 0 : (c > kMostKeys ? kMostKeys : c);
}
__device__ __forceinline__ int32_t keys_added(const MapParams& p, int b, int32_t before) {
  const int32_t n = p.add[b];
  return n < 0 ? 0 : (n > kMostKeys - before ? kMostKeys - before : n);
}

// Last index i with start[i] <= x (start ascending, start[0] = 0).
__device__ __forceinline__ int find_seq(const int32_t* start, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// With have = ceil(ctx / page), need = ceil((ctx + new) / page) per sequence,
// the sequences take need - have pages each from free_pages, in order, and
// token j of sequence b lands in slot table[b][(ctx + j) / page] * page +
// (ctx + j) % page.  Every block scans the lengths for itself (two prefix
// sums over the batch in shared memory), so one launch does it all: a page
// that is new in this call is looked up in free_pages, one that was there
// before in the table, and no block reads what another writes.  Bound: latency.
// 64 sequences of one token each 2.8 us; 37 prompts, 663,000 slots and 10,400 pages,
// 5.6 us, 1 TB/s.
__global__ void __launch_bounds__(kMapThreads) page_map_kernel(const MapParams p) {
  extern __shared__ int32_t sm[];
  int32_t* cu = sm;                   // [batch + 1] first new token of each sequence
  int32_t* off = sm + p.batch + 1;    // [batch + 1] first page it takes
  __shared__ int32_t part[2][kMapThreads];
  const int t = threadIdx.x;
  const int per = (p.batch + kMapThreads - 1) / kMapThreads;
  const int32_t mask = (1 << p.shift) - 1;
  const int b0 = t * per < p.batch ? t * per : p.batch;
  const int b1 = b0 + per < p.batch ? b0 + per : p.batch;
  int32_t sum_new = 0, sum_take = 0;
  for (int b = b0; b < b1; ++b) {
    const int32_t c = keys_before(p, b), n = keys_added(p, b, c);
    cu[b] = sum_new;
    off[b] = sum_take;
    sum_new += n;
    sum_take += ((c + n + mask) >> p.shift) - ((c + mask) >> p.shift);
  }
  part[0][t] = sum_new;
  part[1][t] = sum_take;
  __syncthreads();
  if (t < 64) {  // warp 0 scans the token sums, warp 1 the page sums
    int32_t* row = part[t >> 5];
    const int lane = t & 31;
    int32_t v[kMapThreads / 32], run = 0;
#pragma unroll
    for (int i = 0; i < kMapThreads / 32; ++i) {
      v[i] = run;
      run += row[lane * (kMapThreads / 32) + i];
    }
    int32_t inc = run;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t o = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += o;
    }
#pragma unroll
    for (int i = 0; i < kMapThreads / 32; ++i)
      row[lane * (kMapThreads / 32) + i] = v[i] + inc - run;
    if (lane == 31) (t < 32 ? cu : off)[p.batch] = inc;
  }
  __syncthreads();
  for (int b = b0; b < b1; ++b) {
    cu[b] += part[0][t];
    off[b] += part[1][t];
  }
  __syncthreads();
  const int32_t total = cu[p.batch], pages = off[p.batch];
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kMapThreads + t;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kMapThreads;
  for (int64_t b = first; b <= p.batch; b += step) {
    p.cu[b] = cu[b];
    if (b < p.batch) {
      const int32_t c = keys_before(p, static_cast<int>(b));
      p.kv_lens[b] = c + keys_added(p, static_cast<int>(b), c);
    } else {
      *p.taken = pages;
    }
  }
  // (sums that pass 31 bits wrap: what they give is wrong then, but every place
  // that is read or written is checked)
  for (int64_t i = first; i < pages; i += step) {
    const int b = find_seq(off, p.batch, static_cast<int32_t>(i));
    const int64_t col = ((keys_before(p, b) + mask) >> p.shift) + (i - off[b]);
    if (col < p.max_pages) p.table[b * p.table_stride + col] = i < p.n_free ? p.free_pages[i] : -1;
  }
  for (int64_t i = first; i < p.n_tokens; i += step) {
    int64_t slot = -1;
    if (i < total) {
      const int b = find_seq(cu, p.batch, static_cast<int32_t>(i));
      const int32_t c = keys_before(p, b);
      const int64_t j = i - cu[b];
      const int64_t pos = c + j, col = pos >> p.shift, have = (c + mask) >> p.shift;
      int32_t page = -1;
      if (j < keys_added(p, b, c) && col < p.max_pages) {
        const int64_t at = off[b] + (col - have);
        if (col < have)
          page = p.table[b * p.table_stride + col];
        else if (at >= 0 && at < p.n_free)
          page = p.free_pages[at];
      }
      if (page >= 0) slot = (static_cast<int64_t>(page) << p.shift) + (pos & mask);
    }
    p.slots[i] = slot;
  }
}

constexpr int kAppendCtas = 32;  // per SM, at most

struct AppendParams {
  const void* k;
  const void* v;
  int64_t k_sh, k_sn, v_sh, v_sn;
  __nv_bfloat16* kp;
  __nv_bfloat16* vp;
  int64_t kp_sp, kp_sh, kp_sn, vp_sp, vp_sh, vp_sn;
  const int64_t* slots;
  int64_t n_tokens, n_slots;
  int heads, d8, shift;
  int* status;
};

template <bool kF32>
__device__ __forceinline__ uint4 load8(const void* base, int64_t off) {
  if constexpr (kF32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
    const float4 a = __ldcs(p), b = __ldcs(p + 1);
    return make_uint4(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w), pack_bf16(b.x, b.y),
                      pack_bf16(b.z, b.w));
  } else {
    return __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + off));
  }
}

// One thread per eight elements of a token's row (a 16-byte store), the
// elements of a token next to each other: with rows and pages that keep a
// token's heads together, a token is one contiguous stretch on both sides.
// Bound: HBM.  32-bit indexes where they fit (a 64-bit division a piece costs
// 8%); 40,001 fp32 rows of 8 heads x 64: 39.2 us at 8 CTAs an SM and 64-bit
// indexes, 36.0 us, 6.6 TB/s, as it is; two or four pieces of a thread in flight
// together are no faster.
template <bool kF32, typename Index>
__global__ void __launch_bounds__(256) page_append_kernel(const AppendParams p) {
  const Index per = static_cast<Index>(p.heads * p.d8);
  const Index n = static_cast<Index>(p.n_tokens) * per;
  const Index step = static_cast<Index>(gridDim.x) * 256;
  for (Index i = static_cast<Index>(blockIdx.x) * 256 + threadIdx.x; i < n; i += step) {
    const Index tok = i / per;
    const int r = static_cast<int>(i - tok * per);
    const int h = r / p.d8, e = (r - h * p.d8) * 8;
    const int64_t slot = __ldg(p.slots + tok);
    if (slot < 0) continue;
    if (slot >= p.n_slots) {
      atomicCAS(p.status, 0, kStatusPage);
      continue;
    }
    const int64_t page = slot >> p.shift, row = slot & ((1 << p.shift) - 1);
    const uint4 k = load8<kF32>(p.k, h * p.k_sh + tok * p.k_sn + e);
    const uint4 v = load8<kF32>(p.v, h * p.v_sh + tok * p.v_sn + e);
    *reinterpret_cast<uint4*>(p.kp + page * p.kp_sp + h * p.kp_sh + row * p.kp_sn + e) = k;
    *reinterpret_cast<uint4*>(p.vp + page * p.vp_sp + h * p.vp_sh + row * p.vp_sn + e) = v;
  }
}

int log2_of(int64_t x) {
  int s = 0;
  while ((int64_t{1} << s) < x) ++s;
  return s;
}

}  // namespace

int launch_page_map(const int32_t* ctx_lens, const int32_t* new_lens, int64_t batch,
                    const int32_t* free_pages, int64_t n_free, int64_t page_size,
                    int32_t* block_table, int64_t table_stride, int64_t max_pages,
                    int64_t* slot_map, int64_t n_tokens, int32_t* cu_new, int32_t* kv_lens,
                    int32_t* taken, const DeviceCtx& ctx, cudaStream_t s) {
  const MapParams p{ctx_lens, new_lens, static_cast<int>(batch), free_pages, n_free,
                    log2_of(page_size), block_table, table_stride, max_pages, slot_map,
                    n_tokens, cu_new, kv_lens, taken};
  int64_t grid = ceil_div(n_tokens > batch + 1 ? n_tokens : batch + 1, kMapThreads);
  if (grid > 4 * ctx.sm_count) grid = 4 * ctx.sm_count;
  const size_t smem = 2 * static_cast<size_t>(batch + 1) * sizeof(int32_t);
  timing_begin(kKidPageMap, s);
  page_map_kernel<<<static_cast<unsigned>(grid), kMapThreads, smem, s>>>(p);
  timing_end(kKidPageMap, s);
  return cudaGetLastError() == cudaSuccess ? LSX_OK : LSX_ERR_LAUNCH;
}

int launch_page_append(const lsx_tensor& k, const lsx_tensor& v, const int64_t* slot_map,
                       const lsx_tensor& k_pages, const lsx_tensor& v_pages,
                       const DeviceCtx& ctx, cudaStream_t s) {
  AppendParams p;
  p.k = k.data; p.v = v.data;
  p.k_sh = k.stride_h; p.k_sn = k.stride_n;
  p.v_sh = v.stride_h; p.v_sn = v.stride_n;
  p.kp = static_cast<__nv_bfloat16*>(k_pages.data);
  p.vp = static_cast<__nv_bfloat16*>(v_pages.data);
  p.kp_sp = k_pages.stride_b; p.kp_sh = k_pages.stride_h; p.kp_sn = k_pages.stride_n;
  p.vp_sp = v_pages.stride_b; p.vp_sh = v_pages.stride_h; p.vp_sn = v_pages.stride_n;
  p.slots = slot_map;
  p.n_tokens = k.N;
  p.n_slots = k_pages.B * k_pages.N;
  p.heads = static_cast<int>(k.H);
  p.d8 = static_cast<int>(k.D / 8);
  p.shift = log2_of(k_pages.N);
  p.status = ctx.status;
  const int64_t pieces = k.N * k.H * p.d8;
  int64_t grid = ceil_div(pieces, 256);
  const int64_t most = kAppendCtas * static_cast<int64_t>(ctx.sm_count);
  if (grid > most) grid = most;
  const bool small = pieces < (int64_t{1} << 31);  // (unsigned: a grid more fits too)
  timing_begin(kKidPageAppend, s);
  auto kern = k.dtype == LSX_F32
                  ? (small ? page_append_kernel<true, uint32_t> : page_append_kernel<true, int64_t>)
                  : (small ? page_append_kernel<false, uint32_t>
                           : page_append_kernel<false, int64_t>);
  kern<<<static_cast<unsigned>(grid), 256, 0, s>>>(p);
  timing_end(kKidPageAppend, s);
  return cudaGetLastError() == cudaSuccess ? LSX_OK : LSX_ERR_LAUNCH;
}

}  // namespace lsx
