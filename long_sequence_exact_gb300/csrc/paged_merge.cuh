// paged_merge.cuh -- the LSE-weighted sum of one row's partials by one warp.
#pragma once

#include <cuda_bf16.h>
#include <math.h>

#include "internal.h"
#include "ptx.cuh"

namespace lsx {
namespace {

// Lane = D / 32 consecutive elements of the row.  take() adds `count` partials:
// row_of(i) is the index of partial i's row in o [rows][D] and l [rows].  The
// order of the additions is that of i, 32 partials at a time with their weights
// in the lanes, eight rows in flight.
template <int D>
struct RowMerge {
  static constexpr int E = D / 32;
  float m = -__builtin_huge_valf(), tot = 0.f, acc[E] = {};

  template <class F>
  __device__ __forceinline__ void take(const float* o, const float* l, int64_t count, int lane,
                                       F&& row_of) {
    constexpr float kNone = -__builtin_huge_valf();
    constexpr float kLog2 = 1.4426950408889634f;
    for (int64_t c0 = 0; c0 < count; c0 += 32) {
      const int n = static_cast<int>(count - c0 < 32 ? count - c0 : 32);
      float y[8][E];
      auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i0 + i < n) {
            const float* src = o + row_of(c0 + i0 + i) * D + lane * E;
            if constexpr (E == 4) {
              const float4 f = __ldcg(reinterpret_cast<const float4*>(src));
              y[i][0] = f.x; y[i][1] = f.y; y[i][2] = f.z; y[i][3] = f.w;
            } else {
              const float2 f = __ldcg(reinterpret_cast<const float2*>(src));
              y[i][0] = f.x; y[i][1] = f.y;
            }
          }
      };
      load(0);  // (in flight while the weights are formed)
      const float mine = lane < n ? __ldcg(l + row_of(c0 + lane)) : kNone;
      float mx = isnan(mine) ? -kNone : mine;  // (NaN weights, and so a NaN row)
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
      const float m_new = fmaxf(m, mx);
      if (m_new == kNone) continue;
      const float keep = m == kNone ? 0.f : ex2((m - m_new) * kLog2);
      const float w = mine == kNone ? 0.f : ex2((mine - m_new) * kLog2);
      float sum = w;
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
      tot = tot * keep + sum;
      m = m_new;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= keep;
      for (int i0 = 0; i0 < n; i0 += 8) {
        if (i0 > 0) load(i0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float wi = __shfl_sync(0xffffffffu, w, (i0 + i) & 31);
          if (i0 + i < n)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(wi, y[i][e], acc[e]);
        }
      }
    }
  }

  // The row (b, h, n) of o and lse.
  __device__ __forceinline__ void store(const lsx_tensor& o, const lsx_tensor& lse, int64_t b,
                                        int64_t h, int64_t n, int lane) const {
    const float inv = tot == 0.f ? 0.f : 1.f / tot;
    const int64_t at = view_off(o, b, h, n) + lane * E;
    if (o.dtype == LSX_F32) {
#pragma unroll
      for (int e = 0; e < E; ++e) static_cast<float*>(o.data)[at + e] = acc[e] * inv;
    } else {
#pragma unroll
      for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(o.data) + at + e) =
            pack_bf16(acc[e] * inv, acc[e + 1] * inv);
    }
    if (lane == 0)
      static_cast<float*>(lse.data)[view_off(lse, b, h, n)] =
          tot == 0.f ? -__builtin_huge_valf() : m + lg2(tot) * 0.6931471805599453f;
  }
};

}  // namespace
}  // namespace lsx
