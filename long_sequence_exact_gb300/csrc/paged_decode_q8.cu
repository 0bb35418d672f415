// paged_decode_q8.cu -- the decode kernel of the 8-bit cache (paged_q8.cu has the
// format): units, runs, clusters, partials and their merge are those of the bf16 one
// (paged_decode.cu).
//
// Bound: HBM bandwidth, at half the bytes a key; so twice the keys a second have to go
// through the warps, and each value is converted on its way.
//
// f16 holds an e4m3 exactly (one conversion instruction for two), so the products are
// of f16, and the rows' powers of two go elsewhere: a key's into its scores, a value's
// into its weight.
// - Q.  A row enters as f16 times a power of two that brings its largest element to
//   [2^12, 2^13): its 8 significant bits are kept exactly down to 2^-29 of that, and to
//   half of f16's last step, 2^-37 of it, below.
// - P.  A weight p enters as f16(p 2^(e - E + kPBits)), e the exponent of its value's row
//   and E the largest so far (O is rescaled when it grows, as under a maximum): 11 bits,
//   and never further off than 2^-36 of the largest that 2^E allows.  For f32 results its
//   remainder is a second f16: 22 bits.
// - The softmax's reference m moves only where a weight under it would pass 2^4 (the
//   quotient is the same under any m), to the row's maximum.  So that a block of keys
//   needs a vote and no maximum over the lanes as a rule.
//
// The products are transposed: S^T = K Q^T with 16 keys as the rows of an m16n8k16 and
// eight query rows as its columns, O^T += V^T P^T with 16 columns of V as the rows.  So
// a unit of up to eight query rows (a group of eight heads, or four heads with two
// tokens) fills the products that 16 rows would half fill, with half the registers: 32
// for O and 16 for Q with heads of 128.
//
// Fragments.  The 16 columns of a product's step may come in any order, as long as Q
// and K agree: a lane's four neighbouring bytes of a key row (ldmatrix of 8 keys x 16
// bytes) are its columns {2c, 2c + 1, 2c + 8, 2c + 9}, two registers of one operand.
// V, transposed by ldmatrix in units of two bytes, comes with columns 2n and 2n + 1 of
// two keys in one register: O's rows n and n + 8.  P^T as an operand is S^T's result
// with keys and rows exchanged between the lanes: one movmatrix for 8 keys.
//
// Steps of 16 KB of keys and 16 KB of values (128 keys of 128, 256 of 64: with 128 of 64
// a call of long contexts took 205 us instead of 179), three stages, 288 threads at 96
// registers (up to 8 rows), two CTAs an SM.  Neighbouring blocks work on neighbouring heads
// of the same keys (use_head_lines), whose rows share the lines that L2 fetches; exponents
// come by 16-byte copies of the loader's lanes.
//
// Measured, 8 kv heads under 32: 64 sequences of up to 12000 keys of 128 145 us for 0.88
// GB, 6.0 TB/s (tensor pipe 16%, issue 44%); 8 of up to 131072, 16 heads of 64, four drafts,
// f32 results 177 us for 1.13 GB, 6.4 TB/s (issue 57%).  64 sequences of up to 8192 keys with
// 8, 16, 32 and 64 rows a key head: of 128 128, 144, 216 and 392 us (the bf16 cache: 210, 214,
// 239 and 407), of 64 83, 97, 138 and 239 us (155, 159, 167 and 279): from 17 rows on the
// warp MMAs and the conversions for them set the time, as there.
#include <math.h>

#include "paged.h"
#include "paged_decode.cuh"
#include "ptx.cuh"
#include "q8.cuh"

namespace lsx {
namespace {

constexpr uint32_t kPBits = 11;  // weights are at most 2^(4 + 11) (f16 ends at 2^16)
constexpr float kMostLog = 4.f;
constexpr float kNoKeys = -3.402823466e38f;  // m of a row without keys so far

// NT: query rows of a warp, in eights.  One: eight compute warps, two: four, which
// have the registers for it.
template <int D, int NT>
struct CfgQ8 {
  static constexpr int kWarps = NT == 1 ? 8 : 4;
  static constexpr int kThreads = 32 * (kWarps + 1);  // and the loader
  static constexpr int kStep = step_keys(D, true);
  static constexpr int kTile = kStep * D;             // bytes of K (or V) per stage
  static constexpr int kStages = 3;
};

template <int D, int NT>
struct SharedQ8 {
  using C = CfgQ8<D, NT>;
  alignas(16) uint8_t exps[C::kStages][2][C::kStep];  // of a stage's keys and values
  int64_t sums[C::kThreads / 32];
  Run run;
  uint64_t full[C::kStages], empty[C::kStages];
  uint32_t pages_ok[C::kStages];  // bit i: 16-key group i of the stage exists
  int abort;
  float m[C::kWarps][8 * NT], l[C::kWarps][8 * NT];  // the warps' row maxima and sums
  float part_m[64], part_l[64];                      // the block's, for its cluster
};
template <int D, int NT>
constexpr int kSmemQ8 =
    CfgQ8<D, NT>::kStages * 2 * CfgQ8<D, NT>::kTile + static_cast<int>(sizeof(SharedQ8<D, NT>));
// two CTAs, each with the system's 1 KB, on an SM's 228 KB
static_assert(2 * (kSmemQ8<128, 1> + 1024) <= 228 * 1024, "shared memory of two CTAs");
static_assert(2 * (kSmemQ8<64, 1> + 1024) <= 228 * 1024, "shared memory of two CTAs");

// The lane's part of one query row (columns 16 kk + 4 (lane % 4) of each step kk, four
// of them) as operands, and the power of two that they were divided by.
template <int D>
__device__ __forceinline__ float load_row(const __nv_bfloat16* q, bool live,
                                          uint32_t (&qf)[D / 16][2]) {
  uint2 w[D / 16];
  float top = 0.f;
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    w[kk] = live ? __ldg(reinterpret_cast<const uint2*>(q + kk * 16)) : make_uint2(0u, 0u);
    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[kk].x << 16)),
                           fabsf(__uint_as_float(w[kk].x & 0xffff0000u))));
    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[kk].y << 16)),
                           fabsf(__uint_as_float(w[kk].y & 0xffff0000u))));
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  int e = static_cast<int>(__float_as_uint(top) >> 23) - 127 - 12;
  if (e < -126) e = -126;
  const float f = q8_power(-e);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    qf[kk][0] = pack_f16(__uint_as_float(w[kk].x << 16) * f,
                         __uint_as_float(w[kk].x & 0xffff0000u) * f);
    qf[kk][1] = pack_f16(__uint_as_float(w[kk].y << 16) * f,
                         __uint_as_float(w[kk].y & 0xffff0000u) * f);
  }
  return q8_power(e);
}

// RT: row tiles of 8 NT rows of a unit, each with warps of its own; warp w works on
// row tile w % RT and on the 16-key blocks [KB kg, + KB) of a step, kg = w / RT.
// CL > 1: few short units, a cluster each (paged_decode.cu).
// Split: P in two f16 (f32 results).
template <int D, int NT, int RT, int CL, bool Split>
__global__ void __launch_bounds__(CfgQ8<D, NT>::kThreads, kCtasPerSm)
    paged_decode_q8_kernel(const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const PagedDecodeParams p) {
  using C = CfgQ8<D, NT>;
  using Sh = SharedQ8<D, NT>;
  constexpr int kS = C::kStages, kW = C::kWarps, kT = C::kThreads, kStep = C::kStep;
  constexpr int kParts = kW / RT;                // warps of a row tile
  constexpr int KB = kStep / 16 / kParts;        // 16-key blocks of a warp and step
  // of them at a time (16 rows of 128 have no registers for two: 64 sequences of up to
  // 8192 keys with 16, 32 and 64 rows 151, 243 and 409 us instead of 144, 216 and 392)
  constexpr int kN = KB < 2 || (D == 128 && NT == 2) ? 1 : 2;
  extern __shared__ __align__(128) uint8_t smem[];
  Sh& sh = *reinterpret_cast<Sh*>(smem + kS * 2 * C::kTile);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rt = warp % RT, kg = warp / RT;
  const WaitGuard guard{p.status, p.wait_ns, &sh.abort};
  if (threadIdx.x == 0) {
    sh.abort = 0;
    for (int i = 0; i < kS; ++i) {
      mbar_init(&sh.full[i], 1 + 32);  // the tiles' bytes, and every lane's copies
      mbar_init(&sh.empty[i], kW);
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
    find_run<kStep, kT>(p, sh.sums, &sh.run);
    x = sh.run.from;  // (of no use to a block without steps)
    n_steps = static_cast<int>(sh.run.s1 - sh.run.s0);
  }
  const uint32_t smem0 = smem_addr(smem);

  if (warp == kW) {
    // ---- loader, as that of the bf16 cache: the rows' exponents from lanes of their own
    constexpr int kGroups = kStep / 16;
    constexpr int kLog = kStep == 128 ? 7 : 8;
    const int boxes = p.c.shift >= kLog ? 1 : kStep >> p.c.shift;
    const int rows = kStep / boxes, per = kGroups / boxes;
    const int box = lane % boxes, part = lane / boxes;  // 0, 1: K, V
    const CUtensorMap* map = part == 0 ? &tm_k : &tm_v;
    // a lane each for the exponents of a 16-key group (copies of 16 bytes: as bulk
    // copies they would take as long as tiles, some 56 cycles each)
    const bool v_exp = (lane & kGroups) != 0;
    const uint8_t* const exps = v_exp ? p.vs : p.ks;
    const int64_t exp_sp = v_exp ? p.vs_sp : p.ks_sp, exp_sh = v_exp ? p.vs_sh : p.ks_sh;
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
      if (part < 2)
        tma_load_4d(smem + (2 * stage + part) * C::kTile + box * rows * D, map, &sh.full[stage], 0,
                    p.c.shift > kLog ? pos & ((1 << p.c.shift) - 1) : 0, hk, page);
      const int group = lane & (kGroups - 1);
      const int32_t its = __shfl_sync(0xffffffffu, mine, group);
      if (lane < 2 * kGroups && ((mask >> group) & 1u) != 0)
        cp_async16(&sh.exps[stage][v_exp ? 1 : 0][group * 16],
                   exps + its * exp_sp + hk * exp_sh + ((pos + group * 16) & ((1 << p.c.shift) - 1)));
      cp_async_arrive(&sh.full[stage]);
      ++issued;
    }
    if (issued < n_steps && lane == 0)  // gave up: wait for what is in flight
      for (int i = issued > kS ? issued - kS : 0; i < issued; ++i) {
        const uint64_t since = global_timer_ns();
        while (!mbar_try_wait(&sh.full[i % kS], (i / kS) & 1))
          if (global_timer_ns() - since > p.wait_ns) break;
      }
  }

  // ---- compute (the loader's threads take part in the block's barriers only)
  auto compute_sync = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kW) : "memory"); };
  const bool computes = warp < kW;
  const int g = lane >> 2, c2 = (lane & 3) * 2;  // the lane's key, and its query rows c2, c2 + 1
  bool whole = x.step == 0;  // the unit's keys so far are all in this run
  uint32_t qf[NT][D / 16][2];
  float q_scale[NT][2];  // of the rows' scores
  int32_t last[NT][2];   // their last visible keys
  // O^T: o[c][t] is columns 16 c + 2 g (first two) and 16 c + 2 g + 1 of rows
  // 8 t + c2, 8 t + c2 + 1, in units of 2^(v_ref - 127 - kPBits)
  float o[D / 16][NT][4], m[NT][2], l[NT][2];
  float l_rest[NT][2];  // f32 results: what l's roundings left (a row's sum over 131072
                        // keys, most of them far below it, was off by up to 2e-6 without)
  uint32_t v_ref = 0;
  auto begin_unit = [&]() {
    v_ref = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      int64_t b, h, n = 0;
      const int row0 = rt * 8 * NT + t * 8;
      const bool live = out_row(p, x.b, x.hk, row0 + g, b, h, n);
      const __nv_bfloat16* q = live ? p.q + b * p.q_sb + h * p.q_sh + n * p.q_sn : p.q;
      const float unit = load_row<D>(q + 2 * c2, live, qf[t]) * p.scale_log2;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        q_scale[t][i] = __shfl_sync(0xffffffffu, unit, (c2 + i) * 4);
        // the length as given: beyond the table it still counts positions
        last[t][i] = x.len - 1;
        n = 0;
        if (p.lens != nullptr) {
          out_row(p, x.b, x.hk, row0 + c2 + i, b, h, n);
          const int64_t lim = static_cast<int64_t>(__ldg(p.lens + x.b)) - p.rows.Nq + n;
          if (lim < last[t][i]) last[t][i] = lim < -1 ? -1 : static_cast<int32_t>(lim);
        }
        m[t][i] = kNoKeys;
        l[t][i] = 0.f;
        if constexpr (Split) l_rest[t][i] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[c][t][e] = 0.f;
    }
  };
  // Where this lane's rows of a block are for ldmatrix, from the tile: keys 0..7 and
  // 8..15 in matrices 0 and 1, the next 16 columns' in 2 and 3.  The 16-byte pieces of
  // a row are permuted by address bits 7 and up, three of them for rows of 128 bytes and
  // two for rows of 64; the piece 2 c after the first is where 32 c is XORed.
  const uint32_t row0 = (lane & 15) * D;
  const uint32_t first =
      row0 + (((lane >> 4) ^ (((smem0 + row0) >> 7) & (D == 128 ? 7 : 3))) << 4);
  // 16 kN keys of a step, from block g0 on
  auto block = [&](uint32_t kt, uint32_t vt, const uint8_t* k_exp, const uint8_t* v_exp,
                   uint32_t ok_mask, int g0) {
    const int32_t key0 = x.step * kStep + g0 * 16;
    // all keys there, and visible to all query tokens
    constexpr uint32_t kAll = (1u << kN) - 1u;
    const bool all = key0 + kN * 16 < x.len + 2 - p.rows.Nq && ((ok_mask >> g0) & kAll) == kAll;
    float s[kN][NT][4];
    uint32_t ke[kN][2], ve[kN][2];  // exponent bytes of the lane's keys and values
#pragma unroll
    for (int j = 0; j < kN; ++j) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][t][e] = 0.f;
      const uint32_t row = kt + first + (g0 + j) * 16 * D;
#pragma unroll
      for (int kk = 0; kk < D / 16; kk += 2) {
        uint32_t w[4];
        ldsm_x4(row ^ (kk << 4), w);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t a[4];
          e4m3_f16x4(w[2 * i], a[0], a[2]);
          e4m3_f16x4(w[2 * i + 1], a[1], a[3]);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma_16816_f16(s[j][t], a, qf[t][kk + i][0], qf[t][kk + i][1]);
        }
      }
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int at = (g0 + j) * 16 + 8 * hh + g;
        ke[j][hh] = *const_cast<const volatile uint8_t*>(k_exp + at);
        ve[j][hh] = *const_cast<const volatile uint8_t*>(v_exp + at);
      }
    }
    if (!all) {
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const bool ok = (ok_mask >> (g0 + j)) & 1u;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int32_t key = key0 + j * 16 + 8 * hh + g;
          if (!ok || key >= x.len) ke[j][hh] = ve[j][hh] = 0u;  // (they may be anything)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (!ok || key > last[t][i]) s[j][t][2 * hh + i] = kNegInf;
        }
      }
    }
    // what a score is multiplied with (never 0, which would make -infinity a NaN; a
    // score that it holds up is 0 all the same)
    auto factor = [&](int j, int hh, int t, int i) {
      return fmaxf(q_scale[t][i] * q8_scale(ke[j][hh]), 1.17549435e-38f);
    };
    // scores less m, in log2
    float a[kN][NT][4];
    float most = kNegInf;
    uint32_t v_top = 0;
#pragma unroll
    for (int j = 0; j < kN; ++j)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        v_top = max(v_top, ve[j][hh]);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float& v = a[j][t][2 * hh + i];
            v = fmaf(s[j][t][2 * hh + i], factor(j, hh, t, i), -m[t][i]);
            most = fmaxf(most, v);
          }
      }
    if (__any_sync(0xffffffffu, most > kMostLog || v_top > v_ref)) {
      float mx[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mx[t][i] = kNegInf;
#pragma unroll
          for (int j = 0; j < kN; ++j)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
              mx[t][i] = fmaxf(mx[t][i], s[j][t][2 * hh + i] * factor(j, hh, t, i));
        }
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        v_top = max(v_top, __shfl_xor_sync(0xffffffffu, v_top, d));
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            mx[t][i] = fmaxf(mx[t][i], __shfl_xor_sync(0xffffffffu, mx[t][i], d));
      }
      float unit = 1.f;
      if (v_top > v_ref) {
        const uint32_t up = v_top - v_ref;
        unit = up < 127 ? q8_power(-static_cast<int>(up)) : 0.f;
        v_ref = v_top;
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float m_new = fmaxf(m[t][i], mx[t][i]);
          const float alpha = ex2(m[t][i] - m_new);  // (0 for the first keys)
          m[t][i] = m_new;
          l[t][i] *= alpha;
          if constexpr (Split) l_rest[t][i] *= alpha;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            o[c][t][i] *= alpha * unit;
            o[c][t][2 + i] *= alpha * unit;
          }
#pragma unroll
          for (int j = 0; j < kN; ++j)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
              a[j][t][2 * hh + i] = fmaf(s[j][t][2 * hh + i], factor(j, hh, t, i), -m_new);
        }
    }
    uint32_t hi[kN][NT][2], lo[kN][NT][2];
    float part[NT][2] = {};  // f32 results: the block's row sums
#pragma unroll
    for (int j = 0; j < kN; ++j)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const uint32_t e = ve[j][hh] + 127u + kPBits;
        const float vf = e > v_ref ? __uint_as_float((e - v_ref) << 23) : 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float w0 = ex2(a[j][t][2 * hh]), w1 = ex2(a[j][t][2 * hh + 1]);
          if constexpr (Split) {
            part[t][0] += w0;
            part[t][1] += w1;
          } else {
            l[t][0] += w0;
            l[t][1] += w1;
          }
          const uint32_t w = pack_f16(w0 * vf, w1 * vf);
          hi[j][t][hh] = transpose_8x8(w);
          if constexpr (Split) {
            const float2 back = unpack_f16(w);
            lo[j][t][hh] = transpose_8x8(pack_f16(w0 * vf - back.x, w1 * vf - back.y));
          }
        }
      }
    if constexpr (Split) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float both = l[t][i] + part[t][i], got = both - l[t][i];
          l_rest[t][i] += (l[t][i] - (both - got)) + (part[t][i] - got);
          l[t][i] = both;
        }
    }
    // rows of V past the last key may hold anything: cleared (0 * NaN is NaN)
    const bool ragged = key0 + kN * 16 > x.len;
#pragma unroll
    for (int c = 0; c < D / 16; c += 2) {
      // (f32 results: a block's products are added up apart and then to O, rounded to
      // the nearest; the tensor cores cut off what does not fit, so that a long chain of
      // them loses 2^-24 of O a link: 6.6e-6 instead of 1e-6 over 131072 keys)
      float sum[2][NT][4] = {};
      uint32_t v[kN][4];  // keys 0..7 and 8..15 of columns 16 c, and of the next 16
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        ldsm_x4_t((vt + first + (g0 + j) * 16 * D) ^ (c << 4), v[j]);
        if (ragged) {
          const int32_t left = x.len - (key0 + j * 16 + c2);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint32_t keep =
                (left > 8 * t ? 0xffffu : 0u) | (left > 8 * t + 1 ? 0xffff0000u : 0u);
            v[j][t] &= keep;
            v[j][2 + t] &= keep;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t b[kN][4];
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          e4m3_f16x4(__byte_perm(v[j][2 * i], 0, 0x3120), b[j][0], b[j][1]);
          e4m3_f16x4(__byte_perm(v[j][2 * i + 1], 0, 0x3120), b[j][2], b[j][3]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if constexpr (Split) {  // (the small ones first, which lose next to nothing)
#pragma unroll
            for (int j = 0; j < kN; ++j) mma_16816_f16(sum[i][t], b[j], lo[j][t][0], lo[j][t][1]);
          }
#pragma unroll
          for (int j = 0; j < kN; ++j)
            mma_16816_f16(Split ? sum[i][t] : o[c + i][t], b[j], hi[j][t][0], hi[j][t][1]);
        }
      }
      if constexpr (Split) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[c + i][t][e] += sum[i][t][e];
      }
    }
  };
  // The warps' rows and sums into `buf` [warp][8 NT][D] and sh.m, sh.l.
  auto leave = [&](float* buf) {
    const float f = v_ref > kPBits ? __uint_as_float((v_ref - kPBits) << 23) : 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (Split) l[t][i] += l_rest[t][i];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], d);
        const int r = t * 8 + c2 + i;
        if (g == 0) {
          sh.m[warp][r] = m[t][i] == kNoKeys ? kNegInf : m[t][i];
          sh.l[warp][r] = l[t][i];
        }
        // (rows of a power of two bytes: the pieces of 16 columns change places, so that
        // the four rows of a store fall on different banks)
        float* dst = buf + (warp * 8 * NT + r) * D;
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
          *reinterpret_cast<float2*>(dst + ((c ^ (c2 >> 1 & 1)) * 16) + 2 * g) =
              make_float2(o[c][t][i] * f, o[c][t][2 + i] * f);
      }
  };
  // Columns e .. e + 3 of unit row r, summed over the warps: the numerator, its
  // maximum and its denominator.
  auto sum_row = [&](const float* buf, int r, int e, float4& s, float& mm, float& tot) {
    const int tile = r / (8 * NT), in = r - tile * 8 * NT;
    mm = kNegInf;
#pragma unroll
    for (int k = 0; k < kParts; ++k) mm = fmaxf(mm, sh.m[k * RT + tile][in]);
    s = make_float4(0.f, 0.f, 0.f, 0.f);
    tot = 0.f;
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      const float mk = sh.m[k * RT + tile][in];
      const float w = mk == kNegInf ? 0.f : ex2(mk - mm);
      const float4 y = *reinterpret_cast<const float4*>(
          buf + ((k * RT + tile) * 8 * NT + in) * D + (e ^ ((in >> 1 & 1) * 16)));
      tot += sh.l[k * RT + tile][in] * w;
      s.x += y.x * w; s.y += y.y * w;
      s.z += y.z * w; s.w += y.w * w;
    }
  };
  auto store = [&](int r, int e, const float4& s, float mm, float tot, int64_t slot, bool direct) {
    // (a row without keys has tot = 0; a NaN score stays)
    int64_t b, h, n;
    if (!out_row(p, x.b, x.hk, r, b, h, n)) return;
    const float inv = tot == 0.f ? 0.f : 1.f / tot;
    const float lse = tot == 0.f ? kNegInf : (mm + lg2(tot)) * kLn2;
    const float4 y = make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv);
    if (!direct) {
      *reinterpret_cast<float4*>(p.part.o + (slot * p.R + r) * D + e) = y;
      if (e == 0) p.part.l[slot * p.R + r] = lse;
      return;
    }
    const int64_t at = view_off(p.o, b, h, n) + e;
    if (p.o.dtype == LSX_F32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.o.data) + at) = y;
    else
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o.data) + at) =
          make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
    if (e == 0) static_cast<float*>(p.lse.data)[view_off(p.lse, b, h, n)] = lse;
  };

  if (computes && n_steps > 0) begin_unit();
  for (int it = 0; computes && it < n_steps; ++it) {
    const int stage = it % kS;
    // (past a wait that ran out every wait returns at once: the run ends with
    // the status set, all barriers met)
    mbar_wait(&sh.full[stage], (it / kS) & 1, guard);
    const uint32_t kt = smem0 + stage * 2 * C::kTile, vt = kt + C::kTile;
    const uint32_t ok_mask = *const_cast<volatile uint32_t*>(&sh.pages_ok[stage]);
#pragma unroll 1
    for (int j = 0; j < KB; j += kN)
      block(kt, vt, sh.exps[stage][0], sh.exps[stage][1], ok_mask, kg * KB + j);
    const bool unit_end = x.step + 1 == x.steps;
    if (unit_end || it + 1 == n_steps) {
      // the stage that has just been used takes the warps' rows; it is free for the
      // loader when they have been summed
      float* const buf = reinterpret_cast<float*>(smem + stage * 2 * C::kTile);
      compute_sync();
      leave(buf);
      compute_sync();
      if constexpr (CL > 1) break;  // (the cluster's one unit: joined below)
      const bool direct = p.direct && whole && unit_end;
      // a cut unit: the run's first slot when it began in an earlier run, its
      // second when it goes on in a later one
      const int64_t slot = whole && unit_end
                               ? p.whole_slot0 + static_cast<int64_t>(x.b) * p.rows.Hkv + x.hk
                               : 2 * static_cast<int64_t>(blockIdx.x) + (whole ? 1 : 0);
      for (int i = threadIdx.x; i < p.R * (D / 4); i += 32 * kW) {
        const int r = i / (D / 4), e = (i - r * (D / 4)) * 4;
        float4 s;
        float mm, tot;
        sum_row(buf, r, e, s, mm, tot);
        store(r, e, s, mm, tot, slot, direct);
      }
      fence_proxy_async_smem();
      compute_sync();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.empty[stage]);
    advance<kStep>(p, x);
    if (unit_end) {
      whole = true;
      if (it + 1 < n_steps) begin_unit();
    }
  }
  if constexpr (CL > 1) {
    // every CTA leaves its rows (sums over its keys) in its shared memory, and each
    // takes every CL-th piece of four output elements from all of them
    __syncthreads();
    // (the last stage has the warps' rows; the one after it takes the block's)
    const float* const buf =
        reinterpret_cast<const float*>(smem + (n_steps > 0 ? (n_steps - 1) % kS : 0) * 2 * C::kTile);
    float* const part = reinterpret_cast<float*>(smem + n_steps % kS * 2 * C::kTile);
    for (int i = threadIdx.x; i < p.R * (D / 4); i += kT) {
      const int r = i / (D / 4), e = (i - r * (D / 4)) * 4;
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      float mm = kNegInf, tot = 0.f;
      if (n_steps > 0) sum_row(buf, r, e, s, mm, tot);
      *reinterpret_cast<float4*>(part + r * D + e) = s;
      if (e == 0) {
        sh.part_m[r] = mm;
        sh.part_l[r] = tot;
      }
    }
    // (the siblings' rows may lie in another stage than this block's)
    if (threadIdx.x == 0) sh.pages_ok[0] = n_steps % kS;
    cluster_sync();
    uint32_t at[CL];
#pragma unroll
    for (int c = 0; c < CL; ++c)
      at[c] = sibling(smem0, c) + __float_as_uint(ld_cluster(sibling(smem_addr(&sh.pages_ok[0]), c))) *
                                      (2 * C::kTile);
    for (int i = threadIdx.x * CL + rank; i < p.R * (D / 4); i += kT * CL) {
      const int r = i / (D / 4), e = (i - r * (D / 4)) * 4;
      float pm[CL], pl[CL];
      float4 po[CL];
#pragma unroll
      for (int c = 0; c < CL; ++c) {
        pm[c] = ld_cluster(sibling(smem_addr(sh.part_m + r), c));
        pl[c] = ld_cluster(sibling(smem_addr(sh.part_l + r), c));
        po[c] = ld_cluster4(at[c] + (r * D + e) * 4);
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
      store(r, e, s, mm, tot, 0, true);
    }
    cluster_sync();  // no CTA leaves while its rows are read
  } else {
    // a prefix launch that this one overlaps with (nothing of it is read here)
    // has ended before this one has: the merge waits for this one alone
    asm volatile("griddepcontrol.wait;" ::: "memory");
  }
}

template <int D, int NT, int RT, int CL, bool Split>
int launch(const PageMaps& maps, const PagedDecodeParams& p, int64_t grid, bool early, int device,
           cudaStream_t s) {
  auto kern = paged_decode_q8_kernel<D, NT, RT, CL, Split>;
  constexpr int smem = kSmemQ8<D, NT>;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(kern, smem, device, done)) return LSX_ERR_LAUNCH;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(CfgQ8<D, NT>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  if (CL > 1) {
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {CL, 1, 1};
  } else {
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = &attr;
  cfg.numAttrs = CL > 1 || early ? 1 : 0;
  timing_begin(kKidPagedDecode, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, maps.k, maps.v, p);
  timing_end(kKidPagedDecode, s);
  return e == cudaSuccess ? LSX_OK : LSX_ERR_LAUNCH;
}

template <int D, int CL, bool Split>
int launch_rows(const PageMaps& maps, const PagedDecodeParams& p, int64_t grid, bool early,
                int device, cudaStream_t s) {
  return p.R <= 8    ? launch<D, 1, 1, CL, Split>(maps, p, grid, early, device, s)
         : p.R <= 16 ? launch<D, 2, 1, CL, Split>(maps, p, grid, early, device, s)
         : p.R <= 32 ? launch<D, 2, 2, CL, Split>(maps, p, grid, early, device, s)
                     : launch<D, 2, 4, CL, Split>(maps, p, grid, early, device, s);
}
template <int CL>
int launch_heads(const PageMaps& maps, const PagedDecodeParams& p, int64_t d, int64_t grid,
                 bool early, int device, cudaStream_t s) {
  return d == 128 ? (p.split ? launch_rows<128, CL, true>(maps, p, grid, early, device, s)
                             : launch_rows<128, CL, false>(maps, p, grid, early, device, s))
                  : (p.split ? launch_rows<64, CL, true>(maps, p, grid, early, device, s)
                             : launch_rows<64, CL, false>(maps, p, grid, early, device, s));
}

}  // namespace

// early: the launch before is the shared prefix's; this one may start while that
// one drains.
int launch_run_q8(const PageMaps& maps, const PagedDecodeParams& p, int64_t d, int64_t grid,
                  bool early, int device, cudaStream_t s) {
  return launch_heads<1>(maps, p, d, grid, early, device, s);
}
int launch_clusters_q8(const PageMaps& maps, const PagedDecodeParams& p, int64_t d, int device,
                       cudaStream_t s) {
  return launch_heads<kCluster>(maps, p, d, p.units_b * p.rows.Hkv * kCluster, false, device, s);
}

}  // namespace lsx
