// paged_simple.cu -- attention over a paged cache, one warp per query row:
// lane = key for the scores, lane = D / 32 elements for the sum over values,
// an online softmax over blocks of 32 keys.
#include <math.h>

#include "paged.h"
#include "ptx.cuh"

namespace lsx {
namespace {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct SimpleParams {
  PagedCache c;
  const __nv_bfloat16* q;
  int64_t q_sb, q_sh, q_sn;
  int64_t B, Hq, Hkv, N, batch;
  const int32_t* kv_lens;
  const int32_t* cu_q;  // NULL: decode
  const int32_t* prefix_table;
  int64_t prefix_len;
  float scale_log2;
  lsx_tensor o, lse;
  int* status;
};

template <int D>
__global__ void __launch_bounds__(128) paged_simple_kernel(const SimpleParams p) {
  __shared__ float sq[4][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + warp;
  if (row >= p.B * p.Hq * p.N) return;
  const int64_t n = row % p.N, h = row / p.N % p.Hq, b = row / (p.N * p.Hq);
  int64_t seq = b, visible;
  const int64_t cap = static_cast<int64_t>(p.c.max_pages) << p.c.shift;
  if (p.cu_q != nullptr) {
    for (seq = 0; seq < p.batch; ++seq)
      if (n >= p.cu_q[seq] && n < p.cu_q[seq + 1]) break;
    if (seq == p.batch) return;
    visible = static_cast<int64_t>(p.kv_lens[seq]) - p.cu_q[seq + 1] + n + 1;
  } else {
    visible = static_cast<int64_t>(p.kv_lens[seq]) - p.N + n + 1;
  }
  if (visible > cap) {
    visible = cap;
    if (lane == 0) atomicCAS(p.status, 0, kStatusPage);
  }
  if (visible < 0) visible = 0;
  visible += p.prefix_len;
  const __nv_bfloat16* q = p.q + b * p.q_sb + h * p.q_sh + n * p.q_sn;
  for (int d = lane; d < D; d += 32) sq[warp][d] = __bfloat162float(q[d]) * p.scale_log2;
  __syncwarp();
  const int64_t hk = h / (p.Hq / p.Hkv);
  const int32_t mask = (1 << p.c.shift) - 1;
  float m = kNegInf, l = 0.f, o[D / 32];
  for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
  for (int64_t k0 = 0; k0 < visible; k0 += 32) {
    const int64_t key = k0 + lane;
    int64_t page = -1, r = 0;
    if (key < visible) {
      const bool pre = key < p.prefix_len;
      const int64_t pos = pre ? key : key - p.prefix_len;
      page = pre ? p.prefix_table[pos >> p.c.shift]
                 : p.c.table[seq * p.c.table_stride + (pos >> p.c.shift)];
      r = pos & mask;
      if (page < 0 || page >= p.c.n_pages) {
        atomicCAS(p.status, 0, kStatusPage);
        page = -1;
      }
    }
    float s = kNegInf;
    if (page >= 0) {
      const __nv_bfloat16* k = p.c.k + page * p.c.k_sp + hk * p.c.k_sh + r * p.c.k_sn;
      s = 0.f;
      for (int d = 0; d < D; ++d) s = fmaf(sq[warp][d], __bfloat162float(k[d]), s);
    }
    float mx = s;
    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    const float m_new = fmaxf(m, mx);
    if (m_new == kNegInf) continue;
    const float alpha = ex2(m - m_new), e = ex2(s - m_new);
    float sum = e;
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    l = l * alpha + sum;
    m = m_new;
    for (int i = 0; i < D / 32; ++i) o[i] *= alpha;
    const int64_t at = page * p.c.v_sp + hk * p.c.v_sh + r * p.c.v_sn;
    for (int j = 0; j < 32; ++j) {
      const int64_t pj = __shfl_sync(0xffffffffu, page, j), aj = __shfl_sync(0xffffffffu, at, j);
      const float ej = __shfl_sync(0xffffffffu, e, j);
      if (pj < 0) continue;
      for (int i = 0; i < D / 32; ++i)
        o[i] = fmaf(ej, __bfloat162float(p.c.v[aj + lane + 32 * i]), o[i]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int64_t at = view_off(p.o, b, h, n);
  for (int i = 0; i < D / 32; ++i) {
    if (p.o.dtype == LSX_F32)
      static_cast<float*>(p.o.data)[at + lane + 32 * i] = o[i] * inv;
    else
      static_cast<__nv_bfloat16*>(p.o.data)[at + lane + 32 * i] = __float2bfloat16(o[i] * inv);
  }
  if (lane == 0)
    static_cast<float*>(p.lse.data)[view_off(p.lse, b, h, n)] =
        l > 0.f ? (m + lg2(l)) * kLn2 : kNegInf;
}

int launch_simple(const lsx_tensor& q, const PagedCache& c, int64_t hkv, const int32_t* kv_lens,
                  const int32_t* cu_q, int64_t batch, const int32_t* prefix_table,
                  int64_t prefix_len, float scale, const lsx_tensor& o, const lsx_tensor& lse,
                  const DeviceCtx& ctx, cudaStream_t s, int kid) {
  SimpleParams p{c, static_cast<const __nv_bfloat16*>(q.data), q.stride_b, q.stride_h, q.stride_n,
                 q.B, q.H, hkv, q.N, batch, kv_lens, cu_q, prefix_table, prefix_len,
                 scale * kLog2e, o, lse, ctx.status};
  const unsigned grid = static_cast<unsigned>(ceil_div(q.B * q.H * q.N, 4));
  timing_begin(kid, s);
  if (q.D == 128)
    paged_simple_kernel<128><<<grid, 128, 0, s>>>(p);
  else
    paged_simple_kernel<64><<<grid, 128, 0, s>>>(p);
  timing_end(kid, s);
  return cudaGetLastError() == cudaSuccess ? LSX_OK : LSX_ERR_LAUNCH;
}

}  // namespace

size_t paged_fwd_workspace(const lsx_tensor&, const lsx_tensor&, int64_t, int64_t, int) {
  return 0;
}

int launch_paged_fwd(const lsx_tensor& q, const lsx_tensor& k_pages, const lsx_tensor&,
                     const PagedCache& c, const int32_t* kv_lens, const int32_t* cu_q,
                     int64_t batch, float scale, const lsx_tensor& o, const lsx_tensor& lse, void*,
                     const DeviceCtx& ctx, cudaStream_t s) {
  return launch_simple(q, c, k_pages.H, kv_lens, cu_q, batch, nullptr, 0, scale, o, lse, ctx, s,
                       kKidPagedFwd);
}

}  // namespace lsx
