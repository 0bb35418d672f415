// paged_decode.cu -- one or a few query tokens per sequence against a cache
// kept in pages, ragged lengths, optionally after a prefix that the batch
// shares (Lean Attention abstract: split the decode over the context and
// reduce the partials; Tree Attention abstract: tree reduction).
//
// Bound: HBM bandwidth; every visible key and value row is read once for the
// up to 64 query rows (heads of its group x query tokens) that need it.
//
// Decomposition.  A unit is (sequence, kv head): R = (Hq / Hkv) * Nq query
// rows against that sequence's keys, in steps of 64 or 128 keys.  The steps of all
// units, laid end to end, are cut into runs of equal cost, one per CTA (two CTAs
// an SM), whatever the lengths are.  A run that covers a unit whole writes its
// result; a unit cut between runs leaves normalised partials (fp32 O, LSE) in the
// workspace, at most two per CTA, and the merge kernel, launched while the first
// one still runs, combines them by the LSE rule in the order of the keys.  Which
// run holds what follows from the lengths alone, which every CTA sums for itself.
//
// A step is 16 KB of keys and 16 KB of values (64 keys of 128, 128 keys of 64),
// loaded page by page with TMA into one of three stages by a warp of its own,
// which runs ahead across unit ends; pages past the length and pages that do not
// exist come from outside the tensor map and read as zeros.  Scores and output
// by warp-level bf16 MMAs, 16 query rows (padded) x 16 keys a time; the four
// compute warps share the step's keys (and, from 17 rows on, the row tiles).  P
// enters the P V product as the sum of two bf16, so that the result keeps 16
// bits of it (up to 16 rows the tensor pipe is a quarter busy with it; each doubling
// of the rows doubles that).
//
// Measured (8 kv heads of 128 under 32 query heads, ragged): 64 sequences of up
// to 8192 keys 183 us, 6.5 TB/s, of up to 2048 keys 56 us; eight of 131072 keys,
// four drafts, 16 heads of 64, 330 us, 6.7 TB/s; one of 2049 keys 9.6 us.  The 64
// sequences of up to 8192 keys with 4, 32, 40 and 64 rows a key head: 185, 222, 384 and
// 398 us.  From 33 rows on each warp multiplies every key of a step for its 16 rows,
// and the warp MMAs (tensor pipe 51% busy, HBM 42%) set the time.
#include <math.h>

#include "paged.h"
#include "paged_decode.cuh"
#include "paged_merge.cuh"
#include "ptx.cuh"
#include "tma_host.h"

namespace lsx {
namespace {

constexpr int kWarps = 4;                       // compute warps
constexpr int kThreads = 32 * (kWarps + 1);     // and the loader
template <int D>
struct DecodeCfg {
  static constexpr int kStep = step_keys(D, false);    // keys per step
  static constexpr int kSub = D / 64;                  // 64-column (128 B) boxes
  static constexpr int kTile = kStep * D * 2;          // bytes of K (or V) per stage
  static constexpr int kStages = 3;
  static constexpr int kXfer = 2 * 16 * D * 4;         // two warps' O, for the join
};

// What a CTA keeps in shared memory behind the stages and the join's buffer.
struct Shared {
  int64_t sums[kThreads / 32];
  Run run;
  uint64_t full[3], empty[3];
  uint32_t pages_ok[3];     // bit i: 16-key group i of the stage exists
  int abort;
  float xm[2][16], xl[2][16];  // the join's row maxima and sums
};

// The compute warps alone.
__device__ __forceinline__ void compute_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
}

// RT: 16-row tiles of a unit (1, 2 or 4).  Warp w works on row tile w % RT and
// on the keys [16 RT kg, +16 RT) of a step, kg = w / RT.
// CL > 1: few short units.  A cluster of CL CTAs takes one unit, a CL-th of its
// steps each, and joins the parts through its shared memory: no sums over the
// lengths, no partials in memory, no second launch.
template <int D, int RT, int CL>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const PagedDecodeParams p) {
  using C = DecodeCfg<D>;
  constexpr int kS = C::kStages, kStep = C::kStep;
  constexpr int KB = RT * kStep / 64;  // 16-key blocks of a warp and step
  extern __shared__ __align__(128) uint8_t smem[];
  float* const xo = reinterpret_cast<float*>(smem + kS * 2 * C::kTile);
  Shared& sh = *reinterpret_cast<Shared*>(smem + kS * 2 * C::kTile + C::kXfer);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rt = warp % RT, kg = warp / RT;
  const WaitGuard guard{p.status, p.wait_ns, &sh.abort};
  if (threadIdx.x == 0) {
    sh.abort = 0;
    for (int i = 0; i < kS; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kWarps);
    }
    fence_barrier_init();
    tma_prefetch_map(&tm_k);
    tma_prefetch_map(&tm_v);
  }
  int n_steps;
  const uint32_t rank = CL > 1 ? cluster_rank() : 0;
  Cursor x;
  if constexpr (CL > 1) {
    const int32_t unit = blockIdx.x / CL, hkv = static_cast<int32_t>(p.rows.Hkv);
    x.b = unit / hkv;
    x.hk = unit - x.b * hkv;
    x.len = unit_len(p, x.b);
    x.steps = unit_steps<kStep>(x.len);
    x.step = static_cast<int32_t>(static_cast<int64_t>(x.steps) * rank / CL);
    n_steps = static_cast<int32_t>(static_cast<int64_t>(x.steps) * (rank + 1) / CL) - x.step;
    if (threadIdx.x == 0 && rank == 0 &&
        __ldg(p.lens + x.b) > static_cast<int64_t>(p.c.max_pages) << p.c.shift)
      atomicCAS(p.status, 0, kStatusPage);
    __syncthreads();  // the barriers
  } else {
    find_run<kStep, kThreads>(p, sh.sums, &sh.run);
    x = sh.run.from;  // (of no use to a block without steps)
    n_steps = static_cast<int>(sh.run.s1 - sh.run.s0);
  }
  const uint32_t smem0 = smem_addr(smem);

  const int qr = lane >> 2, qc = (lane & 3) * 2;  // fragment row and column
  // (a CTA of a cluster that has no step leaves these as its part: no keys)
  float o[D / 8][4] = {}, m[2] = {kNegInf, kNegInf}, l[2] = {};
  if (warp == kWarps) {
    // ---- loader: the page numbers of a step's 16-key groups, one per lane, are
    // fetched a step ahead; then one box per page, 64-column half and tensor
    constexpr int kGroups = kStep / 16;
    constexpr int kLog = kStep == 64 ? 6 : 7;
    const int boxes = p.c.shift >= kLog ? 1 : kStep >> p.c.shift;
    const int rows = kStep / boxes, per = kGroups / boxes;
    const int box = lane % boxes, sub = lane / boxes % C::kSub, kv = lane / (boxes * C::kSub);
    const CUtensorMap* map = kv == 0 ? &tm_k : &tm_v;
    Cursor ld = x;
    auto fetch = [&](int left) -> int32_t {
      if (left <= 0 || lane >= kGroups) return -1;
      const int32_t pos = ld.step * kStep + lane * 16;
      return pos < ld.len ? __ldg(p.c.table + ld.b * p.c.table_stride + (pos >> p.c.shift)) : -1;
    };
    int32_t next = fetch(n_steps);
    int issued = 0;
    for (int it = 0; it < n_steps; ++it) {
      const int32_t mine = next, pos = ld.step * kStep;
      const int hk = ld.hk;
      const bool exists = mine >= 0 && mine < p.c.n_pages;
      if (lane < kGroups && !exists && pos + lane * 16 < ld.len)
        atomicCAS(p.status, 0, kStatusPage);
      advance<kStep>(p, ld);
      next = fetch(n_steps - it - 1);
      if (ld.step == 0 && it + 1 < n_steps) {  // the next unit's queries
        for (int r = lane; r < p.R; r += 32) {
          int64_t b, h, n;
          if (out_row(p, ld.b, ld.hk, r, b, h, n)) {
            const __nv_bfloat16* q = p.q + b * p.q_sb + h * p.q_sh + n * p.q_sn;
#pragma unroll
            for (int i = 0; i < D; i += 64)
              asm volatile("prefetch.global.L1 [%0];" ::"l"(q + i));
          }
        }
      }
      const uint32_t mask = __ballot_sync(0xffffffffu, exists);
      const int page = __shfl_sync(0xffffffffu, exists ? mine : p.c.n_pages, (box * per) & 31);
      const int stage = it % kS;
      int ok = 1;
      if (lane == 0) {
        ok = it < kS || mbar_wait(&sh.empty[stage], ((it / kS) & 1) ^ 1, guard);
        if (ok) {
          sh.pages_ok[stage] = mask;
          mbar_arrive_expect_tx(&sh.full[stage], 2 * C::kTile);
        }
      }
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      if (kv < 2)
        tma_load_4d(smem + (2 * stage + kv) * C::kTile + sub * kStep * 128 + box * rows * 128, map,
                    &sh.full[stage], sub * 64, p.c.shift > kLog ? pos & ((1 << p.c.shift) - 1) : 0,
                    hk, page);
      ++issued;
    }
    if (issued < n_steps && lane == 0)  // gave up: wait for what is in flight
      for (int i = issued > kS ? issued - kS : 0; i < issued; ++i) {
        const uint64_t since = global_timer_ns();
        while (!mbar_try_wait(&sh.full[i % kS], (i / kS) & 1))
          if (global_timer_ns() - since > p.wait_ns) break;
      }
  }

  // ---- compute (the loader's threads take part in the barriers only)
  const bool computes = warp < kWarps;
  bool whole = x.step == 0;  // the unit's keys so far are all in this run
  uint32_t qf[D / 16][4];
  int32_t last[2];  // last visible key of rows qr, qr + 8 of the tile
  auto begin_unit = [&]() {
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      int64_t b, h, n = 0;
      const bool live = out_row(p, x.b, x.hk, rt * 16 + qr + 8 * hh, b, h, n);
      const __nv_bfloat16* q = live ? p.q + b * p.q_sb + h * p.q_sh + n * p.q_sn : p.q;
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
  if (computes && n_steps > 0) begin_unit();
  // ldmatrix rows of this lane: for K, 8 keys x 16 bytes of d per matrix, keys
  // 8..15 in the upper two; for V (transposed), keys 8..15 in the odd ones.  A
  // 128-byte line's 16-byte pieces are permuted by its address bits 7..9.
  const uint32_t k_row = (lane & 7) + (lane >> 4) * 8, k_piece = (lane >> 3) & 1;
  const uint32_t v_row = (lane & 7) + ((lane >> 3) & 1) * 8, v_piece = lane >> 4;
  const uint32_t sw0 = smem0 >> 7;

  for (int it = 0; computes && it < n_steps; ++it) {
    const int stage = it % kS;
    // (past a wait that ran out every wait returns at once: the run ends with
    // the status set, all barriers met)
    mbar_wait(&sh.full[stage], (it / kS) & 1, guard);
    const uint32_t kt = smem0 + stage * 2 * C::kTile, vt = kt + C::kTile;
    const uint32_t ok_mask = *const_cast<volatile uint32_t*>(&sh.pages_ok[stage]);
    // scores of 16 rows x 16 KB keys
    float s[2 * KB][4];
#pragma unroll
    for (int j = 0; j < KB; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[2 * j][e] = s[2 * j + 1][e] = 0.f;
      const uint32_t r = (kg * KB + j) * 16 + k_row;
      const uint32_t line = kt + r * 128, sw = (sw0 + r) & 7;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t kb[4];
        ldsm_x4(line + (kk >> 2) * kStep * 128 + (((2 * (kk & 3) + k_piece) ^ sw) << 4), kb);
        mma_16816(s[2 * j], qf[kk], kb[0], kb[1]);
        mma_16816(s[2 * j + 1], qf[kk], kb[2], kb[3]);
      }
    }
    float mx[2] = {kNegInf, kNegInf};
#pragma unroll
    for (int j = 0; j < 2 * KB; ++j) {
      const int group = kg * KB + (j >> 1);
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
    // rows of V past the last key may hold anything: cleared (0 * NaN is NaN)
    const bool ragged = (x.step + 1) * kStep > x.len;
#pragma unroll
    for (int j = 0; j < KB; ++j) {
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
      const uint32_t r = (kg * KB + j) * 16 + v_row;
      const uint32_t line = vt + r * 128, sw = (sw0 + r) & 7;
      uint32_t keep[2] = {~0u, ~0u};
      if (ragged) {
        const int32_t left = x.len - (x.step * kStep + (kg * KB + j) * 16 + qc);
#pragma unroll
        for (int t = 0; t < 2; ++t)
          keep[t] = (left > 8 * t ? 0xffffu : 0u) | (left > 8 * t + 1 ? 0xffff0000u : 0u);
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t vb[4];
        ldsm_x4_t(line + (i >> 2) * kStep * 128 + (((2 * (i & 3) + v_piece) ^ sw) << 4), vb);
        if (ragged) {
          vb[0] &= keep[0]; vb[1] &= keep[1];
          vb[2] &= keep[0]; vb[3] &= keep[1];
        }
        mma_16816(o[2 * i], hi, vb[0], vb[1]);
        mma_16816(o[2 * i + 1], hi, vb[2], vb[3]);
        mma_16816(o[2 * i], lo, vb[0], vb[1]);
        mma_16816(o[2 * i + 1], lo, vb[2], vb[3]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.empty[stage]);
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
              sh.xm[slot][qr + 8 * hh] = m[hh];
              sh.xl[slot][qr + 8 * hh] = l[hh];
            }
        }
        compute_sync();
        if (kg < half) {
          float wa[2], wb[2];
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const float om = sh.xm[slot][qr + 8 * hh], ol = sh.xl[slot][qr + 8 * hh];
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
        compute_sync();  // (the buffer is free for the next round, or unit)
      }
      if constexpr (CL > 1) break;  // (the cluster's one unit: joined below)
      if (kg == 0) {
        const bool direct = p.direct && whole && unit_end;
        // a cut unit: the run's first slot when it began in an earlier run, its
        // second when it goes on in a later one
        const int64_t slot = whole && unit_end
                                 ? p.whole_slot0 + static_cast<int64_t>(x.b) * p.rows.Hkv + x.hk
                                 : 2 * static_cast<int64_t>(blockIdx.x) + (whole ? 1 : 0);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int r = rt * 16 + qr + 8 * hh;
          int64_t b, h, n;
          if (!out_row(p, x.b, x.hk, r, b, h, n)) continue;
          // (a row without keys has l = 0; a NaN score stays)
          const float inv = l[hh] == 0.f ? 0.f : 1.f / l[hh];
          const float lse = l[hh] == 0.f ? kNegInf : (m[hh] + lg2(l[hh])) * kLn2;
          if (direct) {
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
    advance<kStep>(p, x);
    if (unit_end) {
      whole = true;
      if (it + 1 < n_steps) begin_unit();
    }
  }
  if constexpr (CL > 1) {
    // every CTA leaves its rows (sums over its keys) in its shared memory, and
    // each takes every CL-th piece of four output elements from all of them
    float* const part = reinterpret_cast<float*>(smem);  // [16 RT][D], stages now idle
    float* const part_m = xo;
    float* const part_l = xo + 16 * RT;
    __syncthreads();
    if (kg == 0 && computes) {
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int r = rt * 16 + qr + 8 * hh;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<float2*>(part + r * D + i * 8 + qc) =
              make_float2(o[i][2 * hh], o[i][2 * hh + 1]);
        if ((lane & 3) == 0) {
          part_m[r] = m[hh];
          part_l[r] = l[hh];
        }
      }
    }
    cluster_sync();
    for (int i = threadIdx.x * CL + rank; i < p.R * (D / 4); i += kThreads * CL) {
      const int r = i / (D / 4), e = (i - r * (D / 4)) * 4;
      float pm[CL], pl[CL];
      float4 po[CL];
#pragma unroll
      for (int c = 0; c < CL; ++c) {
        pm[c] = ld_cluster(sibling(smem_addr(part_m + r), c));
        pl[c] = ld_cluster(sibling(smem_addr(part_l + r), c));
        po[c] = ld_cluster4(sibling(smem_addr(part + r * D + e), c));
      }
      float mm = kNegInf, tot = 0.f;
#pragma unroll
      for (int c = 0; c < CL; ++c) mm = fmaxf(mm, pm[c]);
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < CL; ++c) {
        const float w = pm[c] == kNegInf ? 0.f : ex2(pm[c] - mm);
        tot += pl[c] * w;
        s.x += po[c].x * w; s.y += po[c].y * w;
        s.z += po[c].z * w; s.w += po[c].w * w;
      }
      const float inv = tot == 0.f ? 0.f : 1.f / tot;
      int64_t b, h, n;
      if (out_row(p, x.b, x.hk, r, b, h, n)) {
        const int64_t at = view_off(p.o, b, h, n) + e;
        if (p.o.dtype == LSX_F32)
          *reinterpret_cast<float4*>(static_cast<float*>(p.o.data) + at) =
              make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv);
        else
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o.data) + at) =
              make_uint2(pack_bf16(s.x * inv, s.y * inv), pack_bf16(s.z * inv, s.w * inv));
        if (e == 0)
          static_cast<float*>(p.lse.data)[view_off(p.lse, b, h, n)] =
              tot == 0.f ? kNegInf : (mm + lg2(tot)) * kLn2;
      }
    }
    cluster_sync();  // no CTA leaves while its rows are read
  } else {
    // a prefix launch that this one overlaps with (nothing of it is read here)
    // has ended before this one has: the merge waits for this one alone
    asm volatile("griddepcontrol.wait;" ::: "memory");
  }
}

// The runs of one paged_decode_kernel launch, as the merge sees them.
struct RunView {
  const int64_t* start;  // [units + 1]
  int64_t units, hkv, grid, whole_slot0;
  int R;
  PartView part;
  bool by_head;
};
// Slots of unit (b, hk): those of runs first..last; the unit begins in the first,
// slot 2 first + 1, and goes on in the others, slot 2 c (of their blocks' numbers).  A
// unit in one run has its own.
__device__ __forceinline__ void unit_runs(const RunView& v, int64_t b, int64_t hk, int64_t& first,
                                          int64_t& last) {
  const int64_t s0 = __ldcg(v.start + b), n = __ldcg(v.start + b + 1) - s0;
  const int64_t h = v.by_head ? 1 : v.hkv, grid = v.by_head ? v.grid / v.hkv : v.grid;
  const int64_t total = __ldcg(v.start + v.units), extra = unit_extra(total, h, grid);
  const int64_t all = (total + extra * v.units) * h, g = run_count(all, grid);
  const int64_t a = (s0 + extra * b) * h + (v.by_head ? 0 : hk * (n + extra)) + extra;
  const int64_t z = a + n - 1;
  first = ((a + 1) * g - 1) / all;
  last = ((z + 1) * g - 1) / all;
}

// The prompt kernel's partials of a shared prefix (pieces 0: none).
struct TileView {
  int tpt, pieces;
  const float* o;
  const float* l;
};

struct PagedMergeParams {
  RowMap rows;
  RunView own, prefix;  // prefix.grid 0: none
  TileView tiles;
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
    const int64_t u = gr / v.R, r = gr - u * v.R;
    unit_runs(v, u, hk, first, last);
    sum.take(v.part.o, v.part.l, last - first + 1, lane, [&](int64_t i) {
      const int64_t block = v.by_head ? (first + i) * v.hkv + hk : first + i;
      const int64_t slot = first == last ? v.whole_slot0 + u * v.hkv + hk
                                         : 2 * block + (i == 0 ? 1 : 0);
      return slot * v.R + r;
    });
  };
  if (p.tiles.pieces > 0) {
    const TileView& v = p.tiles;
    const int64_t unit = b / (2 * v.tpt);
    const int64_t at = (b / v.tpt % 2) * 128 +
                       ((b % v.tpt) * p.rows.Nq + n) * p.rows.G + h % p.rows.G;
    sum.take(v.o, v.l, v.pieces, lane,
             [&](int64_t i) { return ((unit * v.pieces + i) * p.rows.Hkv + hk) * 256 + at; });
  } else if (p.prefix.grid > 0) {
    take(p.prefix);
  } else {
    int64_t first, last;
    unit_runs(p.own, b, hk, first, last);
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

// A prefix under more query rows of a key head than these goes to the prompt kernel.
// 131072 keys under 32, 36 and 64 rows, heads of 128: 105, 175 and 179 us here, 124
// there (36 and 64), 162 with P to 16 bits; of 64: 64, 119 and 122 us here, 97 and
// 140 there.  4096 keys differ by 2 us at most.
// 8 bits, heads of 128: 36 and 64 rows 171 and 176 us here, 147 there (f32 results: 224 and
// 231, 189 and 198); of 64: 110 here, 132 there (135 and 140, 166).
constexpr int64_t most_warp_rows(int64_t d, bool q8) { return q8 && d == 64 ? 64 : 32; }

template <int D>
constexpr int kSmem =
    DecodeCfg<D>::kStages * 2 * DecodeCfg<D>::kTile + DecodeCfg<D>::kXfer + static_cast<int>(sizeof(Shared));
// two CTAs, each with the system's 1 KB, on an SM's 228 KB
static_assert(2 * (kSmem<128> + 1024) <= 228 * 1024, "shared memory of two CTAs");

// Units a cluster each: all of them on the device at once, and short (the
// table's width bounds the keys; the lengths are not known here, so that a short
// sequence behind a wide table takes runs: 2049 keys 13.8 us instead of 9.6).  8 units of
// 128: 2048 keys 8.6 us, 13.6 us as runs; 8192 keys 20.0 and 17.1 us; of 64: 8192 keys 10.0
// and 13.5 us, 16384 keys 15.7 and 15.1 us.
// 8-bit caches: up to 12288 keys.  Of 128, one sequence of 2049 keys 13.4 us, 19.6 as runs; of
// 12000 23.6 and 27.8; four of 12000 28.8 and 36.0; of 64, one of 12000 19.6 and 25.7.
constexpr int64_t kClusterSteps = 12;  // of a CTA, at most
bool fits_clusters(int64_t units, int64_t most_keys, int64_t d, bool q8, int sm_count) {
  return units * kCluster <= kCtasPerSm * static_cast<int64_t>(sm_count) &&
         most_keys <= kCluster * kClusterSteps * (q8 ? 128 : step_keys(d, false));
}

// A line for each kv head (8-bit caches), where that leaves few blocks without work.
// 64 sequences of up to 12000 keys, 8 heads of 128 in 16-token pages, a token's heads
// together: 148 us, one line for all heads 209; 8 of up to 131072 keys, 16 heads of 64, a
// head's together: 177, 187.
bool use_head_lines(int64_t hkv, int64_t grid) {
  return hkv > 1 && grid >= hkv && grid % hkv <= grid / 16;
}

template <int D, int RT>
int launch_clusters(const PageMaps& maps, const PagedDecodeParams& p, int device, cudaStream_t s) {
  auto kern = paged_decode_kernel<D, RT, kCluster>;
  constexpr int smem = kSmem<D>;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(kern, smem, device, done)) return LSX_ERR_LAUNCH;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.units_b * p.rows.Hkv * kCluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {kCluster, 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  timing_begin(kKidPagedDecode, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, maps.k, maps.v, p);
  timing_end(kKidPagedDecode, s);
  return e == cudaSuccess ? LSX_OK : LSX_ERR_LAUNCH;
}

int launch_clusters(const PageMaps& maps, const PagedDecodeParams& p, int64_t d, int dev,
                    cudaStream_t s) {
  if (p.ks != nullptr) return launch_clusters_q8(maps, p, d, dev, s);
  const int rt = p.R <= 16 ? 1 : (p.R <= 32 ? 2 : 4);
  if (d == 128)
    return rt == 1   ? launch_clusters<128, 1>(maps, p, dev, s)
           : rt == 2 ? launch_clusters<128, 2>(maps, p, dev, s)
                     : launch_clusters<128, 4>(maps, p, dev, s);
  return rt == 1   ? launch_clusters<64, 1>(maps, p, dev, s)
         : rt == 2 ? launch_clusters<64, 2>(maps, p, dev, s)
                   : launch_clusters<64, 4>(maps, p, dev, s);
}

// early: the launch before is the shared prefix's; this one may start while
// that one drains.
template <int D, int RT>
int launch_run(const PageMaps& maps, const PagedDecodeParams& p, int64_t grid, bool early,
               int device, cudaStream_t s) {
  auto kern = paged_decode_kernel<D, RT, 1>;
  constexpr int smem = kSmem<D>;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(kern, smem, device, done)) return LSX_ERR_LAUNCH;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = early ? 1 : 0;
  timing_begin(kKidPagedDecode, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, maps.k, maps.v, p);
  timing_end(kKidPagedDecode, s);
  return e == cudaSuccess ? LSX_OK : LSX_ERR_LAUNCH;
}

int launch_run(const PageMaps& maps, const PagedDecodeParams& p, int64_t d, int64_t grid,
               bool early, int dev, cudaStream_t s) {
  if (p.ks != nullptr) return launch_run_q8(maps, p, d, grid, early, dev, s);
  const int rt = p.R <= 16 ? 1 : (p.R <= 32 ? 2 : 4);
  if (d == 128)
    return rt == 1   ? launch_run<128, 1>(maps, p, grid, early, dev, s)
           : rt == 2 ? launch_run<128, 2>(maps, p, grid, early, dev, s)
                     : launch_run<128, 4>(maps, p, grid, early, dev, s);
  return rt == 1   ? launch_run<64, 1>(maps, p, grid, early, dev, s)
         : rt == 2 ? launch_run<64, 2>(maps, p, grid, early, dev, s)
                   : launch_run<64, 4>(maps, p, grid, early, dev, s);
}

}  // namespace

size_t paged_decode_workspace(const lsx_tensor& q, const lsx_tensor& k_pages, int64_t max_pages,
                              int64_t prefix_len, bool q8, int sm_count) {
  const int64_t slots = 2 * kCtasPerSm * static_cast<int64_t>(sm_count);
  const int64_t per = q.H / k_pages.H * q.N;
  if (prefix_len <= 0 && fits_clusters(q.B * k_pages.H, max_pages * k_pages.N, q.D, q8, sm_count))
    return 0;
  if (prefix_len <= 0) return run_layout(slots, per, q.D, q.B, 0).total;
  const size_t own = run_layout(slots, per, q.D, q.B, q.B * k_pages.H).total;
  const int64_t R = q.B * per;
  if (R <= most_warp_rows(q.D, q8)) return own + run_layout(slots, R, q.D, 1, k_pages.H).total;
  const size_t rows = static_cast<size_t>(
      prefix_plan(q.B, per, k_pages.H, prefix_len, sm_count).rows);
  return own + align256(rows * 4) + align256(rows * static_cast<size_t>(q.D) * 4);
}

int launch_paged_decode(const lsx_tensor& q, const lsx_tensor& k_pages, const lsx_tensor& v_pages,
                        const PagedCache& c, const PagedCache8* c8, const int32_t* kv_lens,
                        const int32_t* prefix_table, int64_t prefix_len, float scale,
                        const lsx_tensor& o, const lsx_tensor& lse, void* workspace,
                        const DeviceCtx& ctx, cudaStream_t s) {
  PagedDecodeParams p;
  p.c = c;
  p.q = static_cast<const __nv_bfloat16*>(q.data);
  p.q_sb = q.stride_b; p.q_sh = q.stride_h; p.q_sn = q.stride_n;
  const int64_t hkv = k_pages.H, per = q.H / hkv * q.N;
  p.rows = RowMap{q.B, q.H, hkv, static_cast<int>(q.H / hkv), static_cast<int>(q.N),
                  static_cast<int>(per)};
  p.scale_log2 = scale * kLog2e;
  p.o = o; p.lse = lse;
  p.status = ctx.status;
  p.wait_ns = ctx.wait_ns;
  const bool q8 = c8 != nullptr;
  p.ks = p.vs = nullptr;
  if (q8) {
    p.ks = c8->ks; p.ks_sp = c8->ks_sp; p.ks_sh = c8->ks_sh;
    p.vs = c8->vs; p.vs_sp = c8->vs_sp; p.vs_sh = c8->vs_sh;
    p.split = o.dtype == LSX_F32;
  }
  const int64_t slots = 2 * kCtasPerSm * static_cast<int64_t>(ctx.sm_count);
  // at most one CTA per possible step
  auto runs = [&](int64_t units, int64_t most_keys) {
    const int64_t steps =
        units * hkv * (most_keys > 0 ? ceil_div(most_keys, step_keys(q.D, q8)) : 1);
    return steps < slots / 2 ? steps : slots / 2;
  };
  const uint32_t box = static_cast<uint32_t>(
      k_pages.N < step_keys(q.D, q8) ? k_pages.N : step_keys(q.D, q8));
  auto encode = [&](CUtensorMap* map, const lsx_tensor& t) {
    return q8 ? make_map_u8_4d(map, t.data, t.B, t.H, t.N, t.D, t.stride_b, t.stride_h, t.stride_n,
                               box, t.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                               : CU_TENSOR_MAP_SWIZZLE_64B)
              : make_map_bf16_4d(map, t.data, t.B, t.H, t.N, t.D, t.stride_b, t.stride_h,
                                 t.stride_n, box);
  };
  PageMaps maps;
  if (!encode(&maps.k, k_pages) || !encode(&maps.v, v_pages)) return LSX_ERR_LAUNCH;
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
    p.by_head = q8 && use_head_lines(hkv, grid);
    return RunView{p.start, units, hkv, grid, slots, static_cast<int>(R), p.part, p.by_head};
  };
  mp.prefix = RunView{};
  mp.tiles = TileView{};
  if (prefix_len > 0) {
    p.c.table = prefix_table;
    p.c.table_stride = 0;
    p.c.max_pages = static_cast<int32_t>(ceil_div(prefix_len, int64_t{1} << c.shift));
    int rc;
    if (q.B * per <= most_warp_rows(q.D, q8)) {
      const int64_t grid = runs(1, prefix_len);
      mp.prefix = place(q.B * per, 1, grid);
      p.lens = nullptr;
      p.fixed_len = prefix_len;
      p.direct = 0;
      rc = launch_run(maps, p, q.D, grid, false, ctx.device, s);
    } else {
      const PrefixPlan plan = prefix_plan(q.B, per, hkv, prefix_len, ctx.sm_count);
      float* part_l = reinterpret_cast<float*>(ws);
      ws += align256(static_cast<size_t>(plan.rows) * 4);
      float* part_o = reinterpret_cast<float*>(ws);
      ws += align256(static_cast<size_t>(plan.rows * q.D) * 4);
      mp.tiles = TileView{plan.tpt, plan.pieces, part_o, part_l};
      rc = launch_prefix(q, k_pages, v_pages, p.c, c8, prefix_len, plan, scale, o.dtype == LSX_F32,
                         part_o, part_l, ctx, s);
    }
    if (rc != LSX_OK) return rc;
    p.c = c;
  }
  const int64_t most_keys = static_cast<int64_t>(c.max_pages) << c.shift;
  if (prefix_len == 0 && fits_clusters(q.B * hkv, most_keys, q.D, q8, ctx.sm_count)) {
    p.lens = kv_lens;
    p.fixed_len = 0;
    p.units_b = q.B;
    p.R = static_cast<int>(per);
    p.direct = 1;
    p.start = nullptr;
    p.by_head = false;
    p.part = PartView{};
    p.whole_slot0 = 0;
    return launch_clusters(maps, p, q.D, ctx.device, s);
  }
  const int64_t grid = runs(q.B, most_keys);
  mp.own = place(per, q.B, grid);
  p.lens = kv_lens;
  p.fixed_len = 0;
  p.direct = prefix_len > 0 ? 0 : 1;
  const int rc = launch_run(maps, p, q.D, grid, prefix_len > 0, ctx.device, s);
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
