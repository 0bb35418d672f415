// paged_decode.cu -- one or a few query tokens per sequence against a cache
// kept in pages, ragged lengths, optionally after a prefix that the batch
// shares (Lean Attention abstract: split the decode over the context and
// reduce the partials; Tree Attention abstract: tree reduction).
//
// Bound: HBM bandwidth; every visible key and value row is read once for the
// up to 64 query rows (heads of its group x query tokens) that need it.
//
// Decomposition.  A unit is (sequence, kv head): R = (Hq / Hkv) * Nq query
// rows against that sequence's keys, in steps of 64 keys.  The steps of all
// units, laid end to end, are cut into equal runs, one per CTA (two CTAs an
// SM), whatever the lengths are: no CTA has more than one step more than
// another.  A run that covers a unit whole writes its result; a unit cut
// between runs leaves normalised partials (fp32 O, LSE) in the workspace, at
// most two per CTA, and the merge kernel, launched while the first one still
// runs, combines them by the LSE rule in the order of the keys.  Which run
// holds what follows from the lengths alone, which every CTA sums for itself.
//
// A step: 128 threads copy 64 rows of K and V (cp.async, 16 bytes each, rows
// past the length and of pages that do not exist zero-filled) into one of the
// ring's stages, 96 KB an SM's half; the loads run ahead of the compute across
// unit ends.  Scores and output by warp-level bf16 MMAs: 16 query rows (padded)
// x 16 keys a time; the warps share the step's keys (and, from 17 rows on,
// the row tiles).  P enters the P V product as the sum of two bf16, so that the
// result keeps 16 bits of it: the tensor cores are idle otherwise.
#include <math.h>

#include "paged.h"
#include "paged_merge.cuh"
#include "ptx.cuh"

namespace lsx {
namespace {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 128;
constexpr int kStep = 64;       // keys per step
constexpr int kCtasPerSm = 2;

// Output rows of a call: global row gr = (b * G + g) * Nq + n within a kv head.
struct RowMap {
  int64_t B, Hq, Hkv;
  int G, Nq, per;   // per = G * Nq rows of a sequence and kv head
};

struct PartView {   // partials: slot s, row r of the unit
  float* o;         // [slots][R][D]
  float* l;         // [slots][R]
};

struct PagedDecodeParams {
  PagedCache c;
  const __nv_bfloat16* q;
  int64_t q_sb, q_sh, q_sn;
  RowMap rows;
  const int32_t* lens;  // NULL: every unit has fixed_len keys, all visible
  int64_t fixed_len;
  int64_t units_b;      // sequences, or groups of R rows against the prefix
  int R;                // rows of a unit
  float scale_log2;
  int direct;           // a unit in one run writes its result itself ...
  int64_t whole_slot0;  // ... or leaves it in this slot + the unit's number
  lsx_tensor o, lse;
  PartView part;
  int64_t* start;       // [units_b + 1] first step of each, per kv head
  int* status;
};

template <int D>
struct DecodeCfg {
  static constexpr int kTile = kStep * D * 2;          // bytes of K (or V) per stage
  static constexpr int kStages = 96 * 1024 / (2 * kTile);
  static constexpr int kXfer = 2 * 16 * D * 4;         // two warps' O, for the join
  static constexpr int kSmem = kStages * 2 * kTile + kXfer;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Keys of unit row b, clamped to what the table holds.
__device__ __forceinline__ int32_t unit_len(const PagedDecodeParams& p, int64_t b) {
  if (p.lens == nullptr) return static_cast<int32_t>(p.fixed_len);
  const int64_t cap = static_cast<int64_t>(p.c.max_pages) << p.c.shift;
  const int32_t n = __ldg(p.lens + b);
  return n < 0 ? 0 : (n > cap ? static_cast<int32_t>(cap) : n);
}
// Steps of a unit: at least one, which writes the empty result.
__device__ __forceinline__ int32_t unit_steps(int32_t len) {
  return len > 0 ? (len + kStep - 1) / kStep : 1;
}

// A place in the run: unit (b, hk), its length and steps, the step.
struct Cursor {
  int64_t b;
  int hk;
  int32_t len, steps, step;
};
__device__ __forceinline__ void advance(const PagedDecodeParams& p, Cursor& x) {
  if (++x.step < x.steps) return;
  x.step = 0;
  if (++x.hk < p.rows.Hkv) return;
  x.hk = 0;
  if (++x.b < p.units_b) {
    x.len = unit_len(p, x.b);
    x.steps = unit_steps(x.len);
  }
}

// Sums the steps of all units and finds this block's run of them, steps
// [t0, t1), and the unit that holds t0; block 0 writes the starts.
__device__ __forceinline__ void find_run(const PagedDecodeParams& p, int64_t* sums, Cursor* place,
                                         int64_t& t0, int64_t& t1) {
  const int t = threadIdx.x;
  const int64_t per = (p.units_b + kThreads - 1) / kThreads;
  const int64_t b0 = t * per < p.units_b ? t * per : p.units_b;
  const int64_t b1 = b0 + per < p.units_b ? b0 + per : p.units_b;
  int64_t mine = 0;
  for (int64_t b = b0; b < b1; ++b) mine += unit_steps(unit_len(p, b));
  int64_t inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, inc, d);
    if ((t & 31) >= d) inc += o;
  }
  if ((t & 31) == 31) sums[t >> 5] = inc;
  __syncthreads();
  int64_t before = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < (t >> 5)) before += sums[w];
    total += sums[w];
  }
  const int64_t all = total * p.rows.Hkv;
  const int64_t g = all < gridDim.x ? all : gridDim.x;  // runs: none is empty
  t0 = blockIdx.x < g ? blockIdx.x * all / g : all;
  t1 = blockIdx.x < g ? (blockIdx.x + 1) * all / g : all;
  // the thread whose sequences hold step t0 finds the unit
  const int64_t h = p.rows.Hkv;
  if (t0 >= before * h && t0 < (before + mine) * h) {
    int64_t at = before;
    for (int64_t b = b0; b < b1; ++b) {
      const int32_t len = unit_len(p, b), n = unit_steps(len);
      if (t0 < (at + n) * h) {
        const int64_t r = t0 - at * h;
        *place = Cursor{b, static_cast<int>(r / n), len, n, static_cast<int32_t>(r % n)};
        break;
      }
      at += n;
    }
  }
  if (blockIdx.x == 0) {
    int64_t at = before;
    for (int64_t b = b0; b < b1; ++b) {
      p.start[b] = at;
      at += unit_steps(unit_len(p, b));
    }
    if (t == kThreads - 1) p.start[p.units_b] = total;
    if (p.lens != nullptr) {
      const int64_t cap = static_cast<int64_t>(p.c.max_pages) << p.c.shift;
      for (int64_t b = b0; b < b1; ++b)
        if (p.lens[b] > cap) atomicCAS(p.status, 0, kStatusPage);
    }
  }
  __syncthreads();
}

// RT: 16-row tiles of a unit (1, 2 or 4).  Warp w works on row tile w % RT and
// on the keys [16 RT kg, +16 RT) of a step, kg = w / RT.
template <int D, int RT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) paged_decode_kernel(
    const PagedDecodeParams p) {
  using C = DecodeCfg<D>;
  constexpr int kS = C::kStages, kPieces = D / 8, kRowsPerPass = kThreads / kPieces;
  constexpr int kPasses = kStep / kRowsPerPass;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t sums[kThreads / 32];
  __shared__ Cursor place;
  __shared__ uint32_t pages_ok[kS];          // bit i: 16-key group i exists
  __shared__ float xm[2][16], xl[2][16];     // the join's row maxima and sums
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rt = warp % RT, kg = warp / RT;
  int64_t t0, t1;
  find_run(p, sums, &place, t0, t1);
  if (t0 >= t1) return;
  const int n_steps = static_cast<int>(t1 - t0);

  // ---- loads: the page numbers of a step's four 16-key groups, one per lane,
  // are fetched a step ahead
  Cursor ld = place;
  int ld_left = n_steps;
  auto fetch_page = [&]() -> int32_t {
    if (ld_left <= 0 || lane >= 4) return -1;
    const int32_t pos = ld.step * kStep + lane * 16;
    if (pos >= ld.len) return -1;
    return __ldg(p.c.table + ld.b * p.c.table_stride + (pos >> p.c.shift));
  };
  int32_t next_page = fetch_page();
  const uint32_t smem0 = smem_addr(smem);
  const int piece = threadIdx.x % kPieces, row0 = threadIdx.x / kPieces;
  auto issue = [&](int stage) {
    if (ld_left > 0) {
      const int32_t mine = next_page;
      const Cursor x = ld;
      advance(p, ld);
      --ld_left;
      next_page = fetch_page();
      const bool ok = mine >= 0 && mine < p.c.n_pages;
      const uint32_t mask = __ballot_sync(0xffffffffu, ok) & 15u;
      if (threadIdx.x == 0) pages_ok[stage] = mask;
      if (warp == 0 && lane < 4 && !ok && x.step * kStep + lane * 16 < x.len)
        atomicCAS(p.status, 0, kStatusPage);
      const uint32_t kd = smem0 + stage * 2 * C::kTile, vd = kd + C::kTile;
      const int64_t k_h = x.hk * p.c.k_sh + piece * 8, v_h = x.hk * p.c.v_sh + piece * 8;
      const int32_t in_page = (1 << p.c.shift) - 1;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int r = row0 + i * kRowsPerPass;
        const int32_t pos = x.step * kStep + r;
        const int64_t page = __shfl_sync(0xffffffffu, ok ? mine : -1, r >> 4);
        const bool live = pos < x.len && page >= 0;
        const int64_t g = live ? page : 0, n = pos & in_page;
        const uint32_t at = r * (D * 2) + ((piece ^ (r & 7)) << 4);
        cp_async16(kd + at, p.c.k + g * p.c.k_sp + k_h + n * p.c.k_sn, live ? 16 : 0);
        cp_async16(vd + at, p.c.v + g * p.c.v_sp + v_h + n * p.c.v_sn, live ? 16 : 0);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kS - 1; ++s) issue(s);

  // ---- compute
  Cursor x = place;
  bool whole = x.step == 0;  // the unit's keys so far are all in this run
  const int qr = lane >> 2, qc = (lane & 3) * 2;  // fragment row and column
  uint32_t qf[D / 16][4];
  float o[D / 8][4], m[2], l[2];
  int32_t last[2];  // last visible key of rows qr, qr + 8 of the tile
  auto begin_unit = [&]() {
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int r = rt * 16 + qr + 8 * hh;
      const int64_t gr = x.b * p.R + r;
      const int64_t b = gr / p.rows.per;
      const int rem = static_cast<int>(gr - b * p.rows.per), g = rem / p.rows.Nq,
                n = rem - g * p.rows.Nq;
      const bool live = r < p.R && b < p.rows.B;
      const __nv_bfloat16* q =
          p.q + b * p.q_sb + (static_cast<int64_t>(x.hk) * p.rows.G + g) * p.q_sh + n * p.q_sn;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qf[kk][hh] = live ? __ldg(reinterpret_cast<const uint32_t*>(q + kk * 16 + qc)) : 0u;
        qf[kk][2 + hh] = live ? __ldg(reinterpret_cast<const uint32_t*>(q + kk * 16 + 8 + qc)) : 0u;
      }
      // the length as given: beyond the table it still counts positions
      last[hh] = x.len - 1;
      if (p.lens != nullptr) {
        const int64_t full = __ldg(p.lens + x.b);
        const int64_t lim = full - p.rows.Nq + n;
        if (lim < last[hh]) last[hh] = lim < -1 ? -1 : static_cast<int32_t>(lim);
      }
      m[hh] = kNegInf;
      l[hh] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  };
  begin_unit();
  const uint32_t ld_row = (lane & 7), ld_mat = lane >> 3;
  float* const xo = reinterpret_cast<float*>(smem + kS * 2 * C::kTile);

  for (int it = 0; it < n_steps; ++it) {
    cp_async_wait<kS - 2>();
    __syncthreads();
    issue((it + kS - 1) % kS);
    const int stage = it % kS;
    const uint32_t kt = smem0 + stage * 2 * C::kTile, vt = kt + C::kTile;
    const uint32_t ok_mask = pages_ok[stage];
    // scores of 16 rows x 16 RT keys
    float s[2 * RT][4];
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const int key0 = (kg * RT + j) * 16;
#pragma unroll
      for (int e = 0; e < 4; ++e) s[2 * j][e] = s[2 * j + 1][e] = 0.f;
      const uint32_t r = key0 + ld_row + (ld_mat >> 1) * 8;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t kb[4];
        ldsm_x4(kt + r * (D * 2) + (((2 * kk + (ld_mat & 1)) ^ (r & 7)) << 4), kb);
        mma_16816(s[2 * j], qf[kk], kb[0], kb[1]);
        mma_16816(s[2 * j + 1], qf[kk], kb[2], kb[3]);
      }
    }
    float mx[2] = {kNegInf, kNegInf};
#pragma unroll
    for (int j = 0; j < 2 * RT; ++j) {
      const int group = kg * RT + (j >> 1);
      const bool ok = (ok_mask >> group) & 1u;
      const int32_t key = x.step * kStep + group * 16 + (j & 1) * 8 + qc;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[j][e] = ok && key + (e & 1) <= last[e >> 1] ? s[j][e] * p.scale_log2 : kNegInf;
        mx[e >> 1] = fmaxf(mx[e >> 1], s[j][e]);
      }
    }
    float mu[2];
    bool grow = false;
    float alpha[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      mx[hh] = fmaxf(mx[hh], __shfl_xor_sync(0xffffffffu, mx[hh], 1));
      mx[hh] = fmaxf(mx[hh], __shfl_xor_sync(0xffffffffu, mx[hh], 2));
      const float m_new = fmaxf(m[hh], mx[hh]);
      alpha[hh] = m_new == kNegInf ? 1.f : ex2(m[hh] - m_new);
      grow |= m_new > m[hh];
      m[hh] = m_new;
      mu[hh] = m_new == kNegInf ? 0.f : m_new;
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= alpha[0]; o[i][1] *= alpha[0];
        o[i][2] *= alpha[1]; o[i][3] *= alpha[1];
      }
      l[0] *= alpha[0];
      l[1] *= alpha[1];
    }
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const float a = ex2(s[2 * j + t][2 * hh] - mu[hh]);
          const float b = ex2(s[2 * j + t][2 * hh + 1] - mu[hh]);
          l[hh] += a + b;
          const uint32_t h = pack_bf16(a, b);
          hi[2 * t + hh] = h;
          lo[2 * t + hh] = pack_bf16(a - __uint_as_float(h << 16),
                                     b - __uint_as_float(h & 0xffff0000u));
        }
      const uint32_t r = (kg * RT + j) * 16 + ld_row + (ld_mat & 1) * 8;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t vb[4];
        ldsm_x4_t(vt + r * (D * 2) + (((2 * i + (ld_mat >> 1)) ^ (r & 7)) << 4), vb);
        mma_16816(o[2 * i], hi, vb[0], vb[1]);
        mma_16816(o[2 * i], lo, vb[0], vb[1]);
        mma_16816(o[2 * i + 1], hi, vb[2], vb[3]);
        mma_16816(o[2 * i + 1], lo, vb[2], vb[3]);
      }
    }
    const bool unit_end = x.step + 1 == x.steps;
    if (unit_end || it + 1 == n_steps) {
      // row sums over the four lanes of a row, then the join of the key groups
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 1);
        l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 2);
      }
#pragma unroll
      for (int half = 2 / RT; half >= 1; half >>= 1) {
        // key groups [half, 2 half) hand theirs to [0, half)
        const int slot = RT == 1 ? (kg & (half - 1)) : rt;
        float* buf = xo + slot * 16 * D;
        if (kg >= half && kg < 2 * half) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
              *reinterpret_cast<float2*>(buf + (qr + 8 * hh) * D + ((i * 8 + qc) ^ ((qr & 3) * 8))) =
                  make_float2(o[i][2 * hh], o[i][2 * hh + 1]);
          if ((lane & 3) == 0)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              xm[slot][qr + 8 * hh] = m[hh];
              xl[slot][qr + 8 * hh] = l[hh];
            }
        }
        __syncthreads();
        if (kg < half) {
          float wa[2], wb[2];
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const float om = xm[slot][qr + 8 * hh], ol = xl[slot][qr + 8 * hh];
            const float m_new = fmaxf(m[hh], om);
            wa[hh] = m[hh] == kNegInf ? 0.f : ex2(m[hh] - m_new);
            wb[hh] = om == kNegInf ? 0.f : ex2(om - m_new);
            l[hh] = l[hh] * wa[hh] + ol * wb[hh];
            m[hh] = m_new;
          }
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const float2 y = *reinterpret_cast<const float2*>(
                  buf + (qr + 8 * hh) * D + ((i * 8 + qc) ^ ((qr & 3) * 8)));
              o[i][2 * hh] = o[i][2 * hh] * wa[hh] + y.x * wb[hh];
              o[i][2 * hh + 1] = o[i][2 * hh + 1] * wa[hh] + y.y * wb[hh];
            }
        }
        if (half > 1) __syncthreads();
      }
      if (kg == 0) {
        const bool direct = p.direct && whole && unit_end;
        // a cut unit: the run's first slot when it began in an earlier run, its
        // second when it goes on in a later one
        const int64_t slot = whole && unit_end
                                 ? p.whole_slot0 + x.b * p.rows.Hkv + x.hk
                                 : 2 * static_cast<int64_t>(blockIdx.x) + (whole ? 1 : 0);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int r = rt * 16 + qr + 8 * hh;
          const int64_t gr = x.b * p.R + r;
          const int64_t b = gr / p.rows.per;
          if (r >= p.R || b >= p.rows.B) continue;
          const float inv = l[hh] > 0.f ? 1.f / l[hh] : 0.f;
          const float lse = l[hh] > 0.f ? (m[hh] + lg2(l[hh])) * kLn2 : kNegInf;
          if (direct) {
            const int rem = static_cast<int>(gr - b * p.rows.per), g = rem / p.rows.Nq,
                      n = rem - g * p.rows.Nq;
            const int64_t h = static_cast<int64_t>(x.hk) * p.rows.G + g;
            const int64_t at = view_off(p.o, b, h, n) + qc;
            if (p.o.dtype == LSX_F32) {
              float* dst = static_cast<float*>(p.o.data) + at;
#pragma unroll
              for (int i = 0; i < D / 8; ++i)
                *reinterpret_cast<float2*>(dst + i * 8) =
                    make_float2(o[i][2 * hh] * inv, o[i][2 * hh + 1] * inv);
            } else {
              __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o.data) + at;
#pragma unroll
              for (int i = 0; i < D / 8; ++i)
                *reinterpret_cast<uint32_t*>(dst + i * 8) =
                    pack_bf16(o[i][2 * hh] * inv, o[i][2 * hh + 1] * inv);
            }
            if ((lane & 3) == 0) static_cast<float*>(p.lse.data)[view_off(p.lse, b, h, n)] = lse;
          } else {
            float* dst = p.part.o + (slot * p.R + r) * D + qc;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
              *reinterpret_cast<float2*>(dst + i * 8) =
                  make_float2(o[i][2 * hh] * inv, o[i][2 * hh + 1] * inv);
            if ((lane & 3) == 0) p.part.l[slot * p.R + r] = lse;
          }
        }
      }
    }
    advance(p, x);
    if (unit_end) {
      whole = true;
      if (it + 1 < n_steps) begin_unit();
    }
  }
}

// The runs of one paged_decode_kernel launch, as the merge sees them.
struct RunView {
  const int64_t* start;  // [units + 1]
  int64_t units, hkv, grid, whole_slot0;
  int R;
  PartView part;
};
// Slots of unit (b, hk): those of runs first..last, run c at slot 2 c, or
// 2 c + 1 where the unit begins in it; a unit in one run has its own.
__device__ __forceinline__ void unit_runs(const RunView& v, int64_t b, int64_t hk, int64_t& first,
                                          int64_t& last, bool& begins) {
  const int64_t s0 = __ldcg(v.start + b), s1 = __ldcg(v.start + b + 1);
  const int64_t all = __ldcg(v.start + v.units) * v.hkv;
  const int64_t a = s0 * v.hkv + hk * (s1 - s0), z = a + (s1 - s0) - 1;
  // run c covers steps [c all / g, (c + 1) all / g)
  const int64_t g = all < v.grid ? all : v.grid;
  first = ((a + 1) * g - 1) / all;
  last = ((z + 1) * g - 1) / all;
  begins = a >= first * all / g;
}

struct PagedMergeParams {
  RowMap rows;
  RunView own, prefix;  // prefix.grid 0: none
  lsx_tensor o, lse;
};

// One warp per output row: the partials of a unit that was cut, in key order
// (the prefix's first); rows whose unit was whole are already written.
template <int D>
__global__ void __launch_bounds__(256) paged_merge_kernel(const PagedMergeParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= p.rows.B * p.rows.Hq * p.rows.Nq) return;
  const int64_t n = row % p.rows.Nq, h = row / p.rows.Nq % p.rows.Hq,
                b = row / (p.rows.Nq * p.rows.Hq);
  const int64_t hk = h / p.rows.G;
  const int64_t gr = (b * p.rows.G + h % p.rows.G) * p.rows.Nq + n;
  RowMerge<D> sum;
  auto take = [&](const RunView& v) {
    int64_t first, last;
    bool begins;
    const int64_t u = gr / v.R, r = gr - u * v.R;
    unit_runs(v, u, hk, first, last, begins);
    sum.take(v.part.o, v.part.l, last - first + 1, lane, [&](int64_t i) {
      const int64_t slot = first == last ? v.whole_slot0 + u * v.hkv + hk
                                         : 2 * (first + i) + (i == 0 && begins ? 1 : 0);
      return slot * v.R + r;
    });
  };
  if (p.prefix.grid > 0) {
    take(p.prefix);
  } else {
    int64_t first, last;
    bool begins;
    unit_runs(p.own, b, hk, first, last, begins);
    if (first == last) return;
  }
  take(p.own);
  sum.store(p.o, p.lse, b, h, n, lane);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace of one launch: partials of (slots + whole) x R rows, and the starts.
struct RunLayout {
  size_t o, l, start, total;
};
RunLayout run_layout(int64_t slots, int64_t R, int64_t D, int64_t units, int64_t whole) {
  slots += whole;
  RunLayout x;
  x.o = 0;
  x.l = align256(static_cast<size_t>(slots * R * D) * 4);
  x.start = x.l + align256(static_cast<size_t>(slots * R) * 4);
  x.total = x.start + align256(static_cast<size_t>(units + 1) * 8);
  return x;
}

int64_t prefix_rows(int64_t rows) { return rows < kMaxDecodeRows ? rows : kMaxDecodeRows; }

template <int D, int RT>
int launch_run(const PagedDecodeParams& p, int64_t grid, cudaStream_t s) {
  auto kern = paged_decode_kernel<D, RT>;
  constexpr int smem = DecodeCfg<D>::kSmem;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return LSX_ERR_LAUNCH;
  timing_begin(kKidPagedDecode, s);
  kern<<<static_cast<unsigned>(grid), kThreads, smem, s>>>(p);
  timing_end(kKidPagedDecode, s);
  return cudaGetLastError() == cudaSuccess ? LSX_OK : LSX_ERR_LAUNCH;
}

int launch_run(const PagedDecodeParams& p, int64_t d, int64_t grid, cudaStream_t s) {
  const int rt = p.R <= 16 ? 1 : (p.R <= 32 ? 2 : 4);
  if (d == 128)
    return rt == 1 ? launch_run<128, 1>(p, grid, s)
                   : (rt == 2 ? launch_run<128, 2>(p, grid, s) : launch_run<128, 4>(p, grid, s));
  return rt == 1 ? launch_run<64, 1>(p, grid, s)
                 : (rt == 2 ? launch_run<64, 2>(p, grid, s) : launch_run<64, 4>(p, grid, s));
}

}  // namespace

size_t paged_decode_workspace(const lsx_tensor& q, const lsx_tensor& k_pages, int64_t,
                              int64_t prefix_len, int sm_count) {
  const int64_t slots = 2 * kCtasPerSm * static_cast<int64_t>(sm_count);
  const int64_t per = q.H / k_pages.H * q.N;
  if (prefix_len <= 0) return run_layout(slots, per, q.D, q.B, 0).total;
  const int64_t R = prefix_rows(q.B * per), groups = ceil_div(q.B * per, R);
  return run_layout(slots, per, q.D, q.B, q.B * k_pages.H).total +
         run_layout(slots, R, q.D, groups, groups * k_pages.H).total;
}

int launch_paged_decode(const lsx_tensor& q, const PagedCache& c, int64_t hkv,
                        const int32_t* kv_lens, const int32_t* prefix_table, int64_t prefix_len,
                        float scale, const lsx_tensor& o, const lsx_tensor& lse, void* workspace,
                        const DeviceCtx& ctx, cudaStream_t s) {
  PagedDecodeParams p;
  p.c = c;
  p.q = static_cast<const __nv_bfloat16*>(q.data);
  p.q_sb = q.stride_b; p.q_sh = q.stride_h; p.q_sn = q.stride_n;
  const int64_t per = q.H / hkv * q.N;
  p.rows = RowMap{q.B, q.H, hkv, static_cast<int>(q.H / hkv), static_cast<int>(q.N),
                  static_cast<int>(per)};
  p.scale_log2 = scale * kLog2e;
  p.o = o; p.lse = lse;
  p.status = ctx.status;
  const int64_t slots = 2 * kCtasPerSm * static_cast<int64_t>(ctx.sm_count);
  // at most one CTA per possible step
  auto runs = [&](int64_t units, int64_t most_keys) {
    const int64_t steps = units * hkv * (most_keys > kStep ? ceil_div(most_keys, kStep) : 1);
    return steps < slots / 2 ? steps : slots / 2;
  };
  PagedMergeParams mp;
  mp.rows = p.rows; mp.o = o; mp.lse = lse;
  char* ws = static_cast<char*>(workspace);
  auto place = [&](int64_t R, int64_t units, int64_t grid) {
    const RunLayout x = run_layout(slots, R, q.D, units, prefix_len > 0 ? units * hkv : 0);
    p.part = PartView{reinterpret_cast<float*>(ws + x.o), reinterpret_cast<float*>(ws + x.l)};
    p.start = reinterpret_cast<int64_t*>(ws + x.start);
    p.units_b = units;
    p.whole_slot0 = slots;
    p.R = static_cast<int>(R);
    ws += x.total;
    return RunView{p.start, units, hkv, grid, slots, static_cast<int>(R), p.part};
  };
  mp.prefix = RunView{};
  if (prefix_len > 0) {
    const int64_t R = prefix_rows(q.B * per), units = ceil_div(q.B * per, R);
    const int64_t grid = runs(units, prefix_len);
    mp.prefix = place(R, units, grid);
    p.c.table = prefix_table;
    p.c.table_stride = 0;
    p.c.max_pages = static_cast<int32_t>(ceil_div(prefix_len, int64_t{1} << c.shift));
    p.lens = nullptr;
    p.fixed_len = prefix_len;
    p.direct = 0;
    const int rc = launch_run(p, q.D, grid, s);
    if (rc != LSX_OK) return rc;
    p.c = c;
  }
  const int64_t grid = runs(q.B, static_cast<int64_t>(c.max_pages) << c.shift);
  mp.own = place(per, q.B, grid);
  p.lens = kv_lens;
  p.fixed_len = 0;
  p.direct = prefix_len > 0 ? 0 : 1;
  const int rc = launch_run(p, q.D, grid, s);
  if (rc != LSX_OK) return rc;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(q.B * q.H * q.N, 8)));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  timing_begin(kKidPagedMerge, s);
  const cudaError_t e = q.D == 128 ? cudaLaunchKernelEx(&cfg, paged_merge_kernel<128>, mp)
                                   : cudaLaunchKernelEx(&cfg, paged_merge_kernel<64>, mp);
  timing_end(kKidPagedMerge, s);
  return e == cudaSuccess ? LSX_OK : LSX_ERR_LAUNCH;
}

}  // namespace lsx
