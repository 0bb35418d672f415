// paged_fwd.cu -- tcgen05 attention of many query tokens against a cache kept
// in pages: ragged prompts, causal (attn_paged_fwd), and the queries of a
// decode batch against the prefix they share (attn_paged_decode).  The online
// softmax of the dense forward (BurstAttention, method section: local attention
// computation), with pages in the place of chunks.
//
// Bound: the tensor cores (4 D operations per visible (query, key) pair), for
// few tokens the cache's bytes.  32 query and 8 kv heads of 128, replayed from a
// graph: 12345 tokens 0.778 ms, 1.60 PFLOP/s (0.82 after some seconds, when the power
// cap lowers the clock); 32768 tokens 5.43 to 5.61 ms, 1.62 to 1.57 PFLOP/s; 512 tokens
// after 65536 keys 0.364 to 0.383 ms, of which the partials' merge 0.011; heads of
// 64, 32768 tokens 4.36 ms, 1.01 PFLOP/s.  With heads of 128 the tensor pipe is busy
// 66% of the time; with heads of 64, half the products for the same weights, it and
// the exponentials' pipe are at 39% and issue slots at 44%: the softmax's chain,
// two warps a scheduler, sets the time.
//
// Rows.  The heads that share a key head are rows of one tile: row r of a
// 128-row query tile is head r % G of token r / G, floor(128 / G) tokens a tile,
// so that K and V are read once for the whole group.  A TMA box with the head
// dimension between d and the tokens lays the rows out that way.
//
// Work.  A unit is two query tiles (a pair) of one sequence, for every kv head;
// units with more key tiles come first.  Where the units times kv heads are
// fewer than two per SM, they are cut along the keys into pieces of equal
// length; the piece count is the one whose rounds over the SMs, partial writes
// and merge reads cost least (plan_kernel, from the lengths on the device).
// A cut unit leaves fp32 partials (O, LSE), merged by the LSE rule at the end.
//
// CTA roles (384 threads, one CTA an SM): warp 0 loads queries and keys and hands
// the decoded items on, warp 3 loads values (TMA, one lane per page and 64-column
// half), warp 1 lane 0 issues the MMAs, warp 2 clears the value rows past a
// sequence's last key, warps 4..7 and 8..11 do the softmax of query tile 0 and 1
// (thread = row = TMEM lane).
// TMEM: S_0 [0,128), S_1 [128,256), O_0 [256,256+D), O_1 [384,384+D); P_t (bf16)
// replaces S_t's first half.  The MMA order per key tile j is P_0 V_j, S_0(j+1), P_1 V_j,
// S_1(j+1): each tile's softmax runs under two products of the other.
//
// Bits of P.  It is rounded to bf16 once, as in the dense forward (the row sums
// are of the weights before that): the error this leaves in O is below that of a
// bf16 O itself.  A shared prefix whose results are f32 keeps 16 bits, as decode does
// everywhere else, so that their accuracy does not depend on how many others are
// in the batch: P = bf16(P) + bf16(P - bf16(P)), the second half behind the first
// in S_t's columns and multiplied with V as well.  131072 keys under 128 rows, a
// call: heads of 128 124 us with one product, 161 with both, of 64 98 and 141.
//
// The issuing thread and the softmax take turns in setting the pace, so both are
// kept short (times of the 12345 tokens above, one after the other):
// - What is consumed together arrives together: a step of the ring holds V of
//   tile j and K of tile j + 1, one barrier when both are in and one when both
//   are free; a barrier looked at costs the issuing thread about 150 cycles
//   (980 -> 928 us).
// - The tiles that both query tiles take go through a loop without conditions,
//   descriptors move by their low words (919 -> 833 us).
// - The softmax takes no maximum of a tile as a rule (833 -> 789 us, heads of 64
//   5.0 -> 4.3 ms at 32768 tokens): the weights exp2(s - m) of any m give the same
//   quotient as long as neither they nor their products with V overflow or vanish.
//   m starts at 0; where a tile's sum reaches 2^15 (128 weights of 2^8: as far as
//   the dense forward lets them go) or a row's is not above 1/2, the tile's
//   maximum is formed, m moved to the size of the sum, O rescaled and the tile's
//   weights formed again.  So |O| stays below 2^15 max |v| a tile, and a small V
//   keeps all but a bit of the range that weights under a maximum leave it (a
//   window up to 2^8 instead: prompts 2.6% slower).  Rows that end in their first
//   tile take its maximum all the same: their largest weight is then exactly 1, and
//   a row with one key is that key's value.
// - Query tile 1's first scores wait for tile 0's first softmax: the two stay out
//   of step, each softmax under the other's products (789 -> 776 us).
// Measured and not kept: P published in halves (a wait more: +7%, and nothing
// once the rest was short), O's barrier once per item (+2%), scores read from
// TMEM in parts between the exponentials (+7% to +14%), the next tile prefetched
// into L2 (+1% to +50%; -3% where a prefix streams from HBM), an issuing thread per
// query tile (+28%, heads of 64 +22%: the tiles' products interleave, and each
// waits for both), for heads of 64 the next scores beside the weights, in TMEM
// that heads of 128 do not have left (-1% ahead of the tile's product, +8% as soon
// as the scores before are read).
//
// Pages.  A tile of 128 keys is 128 / page boxes of a page each (one for pages
// of 128 and more).  A page past the length or one that does not exist is
// loaded from a coordinate outside the tensor map, which fills zeros, and its
// keys are masked by a word per tile that the loader leaves in a ring.  Rows of
// the last page past the length may hold anything: keys there are masked, and
// values are cleared in shared memory before the product (0 * NaN is NaN).
#include <cuda_bf16.h>
#include <math.h>

#include "paged.h"
#include "paged_merge.cuh"
#include "ptx.cuh"
#include "tma_host.h"

namespace lsx {
namespace {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMostSum = 32768.f;  // 2^15 (see the softmax)
constexpr float kLeastSum = 0.5f;
constexpr int kOkRing = 8;       // >= stages + 2 (see the loader)
constexpr int kItems = 4;        // items handed to the other roles ahead
constexpr int kMinPiece = 4;     // key tiles
constexpr int kPiecesPerSm = 4;  // at most, over all units and kv heads
constexpr int kPlanThreads = 512;

// What a CTA works on: tokens [tok0, tok0 + ntok) of sequence b (rows of up to
// two tiles) against key tiles [j0, j0 + size); the first token's last visible
// key is lim0 (causal; each next token sees one more) and there are len keys.
struct __align__(16) Entry {
  int32_t b, tok0, ntok, j0, size, len, lim0, slot;  // slot < 0: the whole row range
};
struct Item {
  Entry e;
  int hk;    // < 0: no more items
  int n[2];  // key tiles of query tile t
  int pad;
};

template <int D>
struct Cfg {
  static constexpr int kStages = (D == 128) ? 2 : 4;
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kSub = D / 64;  // 64-column (128 B) boxes
};

template <int D>
struct __align__(1024) Smem {
  __nv_bfloat16 q[2][128 * D];
  __nv_bfloat16 k[Cfg<D>::kStages][128 * D];
  __nv_bfloat16 v[Cfg<D>::kStages][128 * D];
  uint64_t q_full, q_empty, final_bar;
  uint64_t v_tail, v_fixed;  // the tile with a sequence's last key is in; its dead rows are cleared
  uint64_t full[Cfg<D>::kStages];   // a step: K of a tile and V of the one before
  uint64_t empty[Cfg<D>::kStages];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t item_full[kItems], item_empty[kItems];
  Item item[kItems];
  uint32_t keys_ok[kOkRing];  // bit g: keys [16 g, 16 g + 16) of the tile exist
  uint32_t tail_stage;
  uint32_t tmem_base;
  int abort;
};

// A cut unit for the merge: pieces first, .., first + n - 1.
struct __align__(16) CutUnit {
  int32_t tok0, ntok, first, n;
};
struct Header {
  int32_t n_entries, n_cut;
};

struct FwdParams {
  PagedCache c;
  int64_t Hkv;
  int G, per, tpt;  // heads of a group; rows of a token; tokens of a tile
  const Header* header;
  const Entry* entries;  // NULL: the uniform pieces below (a shared prefix)
  int32_t u_tokens, u_len, u_pieces, u_size;
  float scale_log2;
  lsx_tensor o, lse;
  bool wide;      // the rows of o are 32-byte aligned
  float* part_o;  // [slot][Hkv][256][D]
  float* part_l;  // [slot][Hkv][256]
  int* status;
  uint64_t wait_ns;
};

__device__ __forceinline__ int64_t item_count(const FwdParams& p) {
  const int64_t n = p.entries == nullptr
                        ? static_cast<int64_t>((p.u_tokens + 2 * p.tpt - 1) / (2 * p.tpt)) * p.u_pieces
                        : __ldcg(&p.header->n_entries);
  return n * p.Hkv;
}

// Tokens of tile t of an entry.
__device__ __forceinline__ int tile_tokens(const FwdParams& p, const Entry& e, int t) {
  const int n = e.ntok - t * p.tpt;
  return n < 0 ? 0 : (n > p.tpt ? p.tpt : n);
}
// Last visible key of token i of an entry (the queries of a shared prefix have
// no order: all see all of it).
__device__ __forceinline__ int last_key(const FwdParams& p, const Entry& e, int i) {
  const int lim = p.entries == nullptr ? e.lim0 : e.lim0 + i;
  return lim < e.len - 1 ? lim : e.len - 1;
}

// Item `it` of the list: entry rank, kv head.
__device__ __forceinline__ Item get_item(const FwdParams& p, int64_t it, int64_t n_entries) {
  Item x;
  int64_t rank, hk;
  banded_item(it, n_entries, p.Hkv, &rank, &hk);
  x.hk = static_cast<int>(hk);
  if (p.entries != nullptr) {
    const int4* src = reinterpret_cast<const int4*>(p.entries + rank);
    const int4 a = __ldcg(src), b = __ldcg(src + 1);  // (written by the launch before)
    x.e = Entry{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  } else {  // piece-major: the pairs of one key range run together
    const int pairs = static_cast<int>(n_entries) / p.u_pieces;
    const int piece = static_cast<int>(rank) / pairs, pair = static_cast<int>(rank) % pairs;
    const int tok0 = pair * 2 * p.tpt, left = p.u_tokens - tok0;
    x.e = Entry{0, tok0, left < 2 * p.tpt ? left : 2 * p.tpt, piece * p.u_size, p.u_size,
                p.u_len, p.u_len - 1, pair * p.u_pieces + piece};
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int cnt = tile_tokens(p, x.e, t);
    const int last = cnt > 0 ? last_key(p, x.e, t * p.tpt + cnt - 1) : -1;
    const int n = (last >= 0 ? (last >> 7) + 1 : 0) - x.e.j0;
    x.n[t] = n < 0 ? 0 : (n > x.e.size ? x.e.size : n);
  }
  return x;
}

// Position (within the entry's tiles) of the tile whose value rows past the
// last key have to be cleared, -1 when there is none.
__device__ __forceinline__ int tail_tile(const FwdParams& p, const Entry& e, int nkv) {
  if ((e.len & ((1 << p.c.shift) - 1)) == 0) return -1;
  const int j = (e.len >> 7) - e.j0;
  return j >= 0 && j < nkv ? j : -1;
}

// The products with the low word of a descriptor given apart: the step along K is
// added to it alone (the address field does not carry out of it).
__device__ __forceinline__ void mma_ss_lo(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                          uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts_lo(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// N words of a row, 32 bytes a store (16 where the row is only so aligned).
template <int N>
__device__ __forceinline__ void store_row(void* dst, const uint32_t (&w)[N], bool wide) {
  uint32_t* p = static_cast<uint32_t*>(dst);
  if (wide) {
#pragma unroll
    for (int i = 0; i < N; i += 8)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + i),
                   "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]),
                   "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<uint4*>(p + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  }
}

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > limit_ns) break;
  }
}

template <int D, bool kSplitP>
__global__ void __launch_bounds__(384, 1)
    paged_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const FwdParams p) {
  using C = Cfg<D>;
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                            ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const WaitGuard guard{p.status, p.wait_ns, &sm.abort};

  if (threadIdx.x == 0) {
    sm.abort = 0;
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    mbar_init(&sm.final_bar, 1);
    mbar_init(&sm.v_tail, 1);
    mbar_init(&sm.v_fixed, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&sm.item_full[i], 1);
      mbar_init(&sm.item_empty[i], 11);  // MMA thread, warps 2 and 3, 8 softmax warps
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.s_full[t], 1);
      mbar_init(&sm.p_full[t], 128);
      mbar_init(&sm.o_full[t], 1);
    }
    fence_barrier_init();
    tma_prefetch_map(&tm_q);
    tma_prefetch_map(&tm_k);
    tma_prefetch_map(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan
  const int64_t n_items = item_count(p);
  const int64_t n_entries = n_items / p.Hkv;
  const int64_t grid = gridDim.x, c = blockIdx.x;
  // registers: 128 * 104 + 256 * 200 = 128 * 88 + 256 * 208 = 64,512 = 384 * 168.
  // 32768 tokens: heads of 128 6.32 ms (88 / 208: 6.35), of 64 5.31 ms (104 / 200: 5.73)
  if (warp < 4) {
    regs_dec<D == 64 ? 88 : 104>();
    // Loads: a box per page and 64-column half, each from a lane of its own; the
    // 16-key groups of a tile are in lanes 0..7, a tile ahead.
    const int boxes = p.c.shift >= 7 ? 1 : 128 >> p.c.shift;  // per 64-column half
    const int rows = 128 / boxes;
    const int box = lane % boxes, sub = lane / boxes;
    const int at = sub * 128 * 64 + box * rows * 64;  // where it goes in a tile
    auto group_page = [&](const Item& x, int j, int nkv) -> int32_t {
      const int pos = (x.e.j0 + j) * 128 + lane * 16;
      return j < nkv && lane < 8 && pos < x.e.len
                 ? __ldg(p.c.table + x.e.b * p.c.table_stride + (pos >> p.c.shift))
                 : -1;
    };
    auto box_page = [&](int32_t mine) {
      const bool exists = mine >= 0 && mine < p.c.n_pages;
      return __shfl_sync(0xffffffffu, exists ? mine : p.c.n_pages, (box * (8 / boxes)) & 7);
    };
    auto page_row = [&](const Item& x, int j) {
      return p.c.shift > 7 ? (x.e.j0 + j) * 128 & ((1 << p.c.shift) - 1) : 0;
    };
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
      int ok = 1;
      if (lane == 0) ok = mbar_wait(bar, parity, guard);
      return __shfl_sync(0xffffffffu, ok, 0) != 0;
    };
    if (warp == 0) {
      // --------------------------------------- items, queries and keys
      uint32_t stage = 0, phase = 0, qe_phase = 0;
      uint32_t count = 0, steps = 0;  // key tiles and steps loaded
      const uint32_t q_bytes = 2 * C::kSub * p.per * p.tpt * 128;
      for (int64_t r = 0;; ++r) {
        // (decoded here, ahead of time, and handed to the other roles in a slot)
        const int64_t it = snake_item(c, r, grid);
        const int slot = static_cast<int>(r % kItems);
        Item x;
        if (it < n_items) x = get_item(p, it, n_entries);
        else x.hk = -1;
        if (r >= kItems && !wait_all(&sm.item_empty[slot], ((r / kItems) & 1) ^ 1)) break;
        if (lane == 0) {
          sm.item[slot] = x;
          mbar_arrive(&sm.item_full[slot]);
        }
        if (x.hk < 0) break;
        const int nkv = x.n[0] > x.n[1] ? x.n[0] : x.n[1];
        int32_t next = group_page(x, 0, nkv);
        if (!wait_all(&sm.q_empty, qe_phase ^ 1)) break;
        qe_phase ^= 1;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sm.q_full, q_bytes);
          for (int t = 0; t < 2; ++t)
            for (int s = 0; s < C::kSub; ++s) {
              const int tok = x.e.tok0 + t * p.tpt;
              tma_load_4d(&sm.q[t][s * 128 * 64], &tm_q, &sm.q_full, s * 64, x.hk * p.G,
                          p.entries != nullptr ? tok : 0, p.entries != nullptr ? 0 : tok);
            }
        }
        bool ok = true;
        for (int j = 0; j <= nkv && nkv > 0; ++j) {  // step j: K of tile j, V of tile j - 1
          const int32_t mine = next;
          next = group_page(x, j + 1, nkv);
          const bool exists = mine >= 0 && mine < p.c.n_pages;
          if (j < nkv && lane < 8 && !exists && (x.e.j0 + j) * 128 + lane * 16 < x.e.len)
            atomicCAS(p.status, 0, kStatusPage);
          const uint32_t mask = __ballot_sync(0xffffffffu, exists) & 255u;
          const int page = box_page(mine);
          if (!wait_all(&sm.empty[stage], phase ^ 1)) { ok = false; break; }
          if (lane == 0) {
            // (the word of 8 tiles ago: its readers are done, for the S product
            // of the tile `stages` ago has been taken after their P)
            if (j < nkv) *const_cast<volatile uint32_t*>(&sm.keys_ok[count % kOkRing]) = mask;
            mbar_arrive_expect_tx(&sm.full[stage], (j > 0 && j < nkv ? 2 : 1) * C::kTileBytes);
          }
          __syncwarp();
          if (j < nkv && lane < boxes * C::kSub)
            tma_load_4d(&sm.k[stage][at], &tm_k, &sm.full[stage], sub * 64, page_row(x, j), x.hk,
                        page);
          if (j < nkv) ++count;
          ++steps;
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
      }
      if (lane == 0 && *guard.abort != 0) {
        // gave up: the copies in flight land before the block ends
        drain_wait(&sm.q_full, qe_phase ^ 1, p.wait_ns);
        for (uint32_t i = steps > kStages ? steps - kStages : 0; i < steps; ++i)
          drain_wait(&sm.full[i % kStages], (i / kStages) & 1, p.wait_ns);
      }
    } else if (warp == 3) {
      // ----------------------------------------------------------- values
      // (the step's barrier is armed for both tiles by warp 0)
      uint32_t stage = 0, phase = 0;
      for (uint32_t r = 0;; ++r) {
        if (!wait_all(&sm.item_full[r % kItems], (r / kItems) & 1)) break;
        const Item x = sm.item[r % kItems];
        if (x.hk < 0) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.item_empty[r % kItems]);
        const int nkv = x.n[0] > x.n[1] ? x.n[0] : x.n[1];
        int32_t next = group_page(x, 0, nkv);
        bool ok = true;
        for (int j = 0; j <= nkv && nkv > 0; ++j) {
          if (j > 0) {
            const int page = box_page(next);
            next = group_page(x, j, nkv);
            if (!wait_all(&sm.empty[stage], phase ^ 1)) { ok = false; break; }
            if (lane < boxes * C::kSub)
              tma_load_4d(&sm.v[stage][at], &tm_v, &sm.full[stage], sub * 64, page_row(x, j - 1),
                          x.hk, page);
          }
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
      }
    } else if (warp == 1 && lane == 0) {
      // ------------------------------------------------------ MMA issuer
      constexpr uint32_t kIdS = idesc_bf16_f32(128, 128, 0, 0);
      constexpr uint32_t kIdO = idesc_bf16_f32(128, D, 0, 1);
      // S_t(j+1) overwrites the columns of P_t(j); issued right after P_t(j) V_j
      // by this thread, whose products execute in order.
      uint32_t st = 0, ph = 0, q_phase = 0, fix_phase = 0;
      uint32_t p_phase[2] = {0, 0};
      bool issued = false;
      // operand descriptors: the low words move, with the tile and the step along K
      constexpr uint32_t kTileDesc = C::kTileBytes >> 4;
      const uint64_t q_desc = sdesc_sw128(smem_addr(sm.q[0]), 16, 1024);
      const uint64_t v_desc = sdesc_sw128(smem_addr(sm.v[0]), 128 * 128, 1024);
      const uint32_t q_lo = static_cast<uint32_t>(q_desc);
      const uint32_t k_lo = static_cast<uint32_t>(sdesc_sw128(smem_addr(sm.k[0]), 16, 1024));
      const uint32_t v_lo = static_cast<uint32_t>(v_desc);
      const uint32_t qk_hi = static_cast<uint32_t>(q_desc >> 32);
      const uint32_t v_hi = static_cast<uint32_t>(v_desc >> 32);
      auto issue_s = [&](int t, uint32_t stage) {
        const uint32_t q0 = q_lo + t * kTileDesc, k0 = k_lo + stage * kTileDesc;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss_lo(tmem + t * 128, q0 + static_cast<uint32_t>(kmajor_step(kk, 128)), qk_hi,
                    k0 + static_cast<uint32_t>(kmajor_step(kk, 128)), qk_hi, kIdS,
                    kk > 0 ? 1u : 0u);
        mma_commit(&sm.s_full[t]);
      };
      auto issue_pv = [&](int t, uint32_t stage, uint32_t acc0) {
        const uint32_t v0 = v_lo + stage * kTileDesc;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts_lo(tmem + 256 + t * 128, tmem + t * 128 + kk * 8,
                    v0 + static_cast<uint32_t>(mnmajor_step(kk)), v_hi, kIdO, kk > 0 ? 1u : acc0);
        if constexpr (kSplitP) {  // what P's rounding left out, from the columns behind
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts_lo(tmem + 256 + t * 128, tmem + t * 128 + 64 + kk * 8,
                      v0 + static_cast<uint32_t>(mnmajor_step(kk)), v_hi, kIdO, 1u);
        }
        mma_commit(&sm.o_full[t]);
      };
      for (uint32_t r = 0;; ++r) {
        if (!mbar_wait(&sm.item_full[r % kItems], (r / kItems) & 1, guard)) break;
        const Item& x = sm.item[r % kItems];
        if (x.hk < 0) break;
        const int n0 = x.n[0], n1 = x.n[1];
        const int nkv = n0 > n1 ? n0 : n1;
        const int tail = tail_tile(p, x.e, nkv);
        mbar_arrive(&sm.item_empty[r % kItems]);
        if (!mbar_wait(&sm.q_full, q_phase, guard)) break;
        q_phase ^= 1;
        tc_fence_after();
        bool ok = true;
        if (nkv > 0) {  // S_t(0)
          if (!mbar_wait(&sm.full[st], ph, guard)) break;
          tc_fence_after();
          if (n0 > 0) issue_s(0, st);
          issued = true;
          // the other tile's scores once this one's softmax is done
          if (n0 > 1 && n1 > 1 && !mbar_wait(&sm.p_full[0], p_phase[0], guard)) break;
          if (n1 > 0) issue_s(1, st);
          mma_commit(&sm.empty[st]);
          if (++st == kStages) { st = 0; ph ^= 1; }
        }
        // Q is free for the next item once the last S products are done
        if (nkv <= 1) mma_commit(&sm.q_empty);
        int j = 0;
        for (const int both = (n0 < n1 ? n0 : n1) - 2; j < both; ++j) {
          // both query tiles take this tile and the next two: no conditions
          if (!mbar_wait(&sm.full[st], ph, guard)) { ok = false; break; }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!mbar_wait(&sm.p_full[t], p_phase[t], guard)) { ok = false; break; }
            p_phase[t] ^= 1;
            tc_fence_after();
            issue_pv(t, st, j > 0 ? 1u : 0u);
            issue_s(t, st);
          }
          if (!ok) break;
          mma_commit(&sm.empty[st]);
          if (++st == kStages) { st = 0; ph ^= 1; }
        }
        if (!ok) break;
        for (; j < nkv; ++j) {
          // V of this tile and K of the next
          if (!mbar_wait(&sm.full[st], ph, guard)) { ok = false; break; }
          if (j == tail) {
            sm.tail_stage = st;
            mbar_arrive(&sm.v_tail);
            if (!mbar_wait(&sm.v_fixed, fix_phase, guard)) { ok = false; break; }
            fix_phase ^= 1;
          }
          tc_fence_after();
          for (int t = 0; t < 2; ++t) {
            const int nt = t == 0 ? n0 : n1;
            if (j < nt) {
              if (!mbar_wait(&sm.p_full[t], p_phase[t], guard)) { ok = false; break; }
              p_phase[t] ^= 1;
              tc_fence_after();
              issue_pv(t, st, j > 0 ? 1u : 0u);
            }
            if (j + 1 < nt) issue_s(t, st);
          }
          if (!ok) break;
          if (j + 2 == nkv) mma_commit(&sm.q_empty);
          mma_commit(&sm.empty[st]);
          if (++st == kStages) { st = 0; ph ^= 1; }
        }
        if (!ok) break;
      }
      if (issued) {  // every product has completed before TMEM is released
        mma_commit(&sm.final_bar);
        drain_wait(&sm.final_bar, 0, p.wait_ns);
      }
    } else if (warp == 2) {
      // --------------------------------- value rows past the last key
      // (when the MMA thread asks for it: it knows the stage, and waits)
      uint32_t phase = 0;
      for (uint32_t r = 0;; ++r) {
        int ok = 1;
        if (lane == 0) ok = mbar_wait(&sm.item_full[r % kItems], (r / kItems) & 1, guard);
        if (!__shfl_sync(0xffffffffu, ok, 0)) break;
        const Item x = sm.item[r % kItems];
        if (x.hk < 0) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.item_empty[r % kItems]);
        if (tail_tile(p, x.e, x.n[0] > x.n[1] ? x.n[0] : x.n[1]) >= 0) {
          if (lane == 0) ok = mbar_wait(&sm.v_tail, phase, guard);
          if (!__shfl_sync(0xffffffffu, ok, 0)) break;
          phase ^= 1;
          const uint32_t st = *const_cast<volatile uint32_t*>(&sm.tail_stage);
          // rows [len, end of its page) of the tile; pages after it are zeros
          const int r0 = x.e.len & 127;
          const int r1e = (x.e.len | ((1 << p.c.shift) - 1)) + 1 - (x.e.len & ~127);
          const int r1 = r1e < 128 ? r1e : 128;
          uint4* base = reinterpret_cast<uint4*>(sm.v[st]);
          for (int i = r0 * 8 + lane; i < r1 * 8; i += 32)
#pragma unroll
            for (int s = 0; s < C::kSub; ++s) base[s * 128 * 8 + i] = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.v_fixed);
        }
      }
    }
  } else {
    regs_inc<D == 64 ? 208 : 200>();
    // ----------------------------------------------------------- softmax
    const int t = (warp - 4) >> 2;
    const int row = threadIdx.x - 128 * (1 + t);  // 0..127 == TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + t * 128;
    const uint32_t tO = tS + 256;
    // The loop over key tiles holds 128 scores in registers (to the end: their
    // weights may have to be formed again): little else lives across it.  s_phase:
    // parity of the s_full completions seen, which is that of the P tiles
    // published, too.  live: a row that is written (others may hold anything).
    uint32_t s_phase = 0;
    uint32_t tile = 0;  // key tiles taken (by either query tile), for keys_ok
    const float sl2 = p.scale_log2;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return mbar_wait(bar, parity, WaitGuard{p.status, p.wait_ns, &sm.abort});
    };
    for (uint32_t r = 0;; ++r) {
      if (!wait(&sm.item_full[r % kItems], (r / kItems) & 1)) break;
      int left, last;  // key tiles left; the row's last key within the next one
      bool live;
      {
        const Item& x = sm.item[r % kItems];
        if (x.hk < 0) break;
        left = x.n[t];
        last = last_key(p, x.e, t * p.tpt + row / p.per) - x.e.j0 * 128;
        live = row / p.per < tile_tokens(p, x.e, t);
      }
      float m = 0.f, l = 0.f;
      bool ok = true, first = true;
      for (; left > 0; --left, ++tile, last -= 128) {
        if (!wait(&sm.s_full[t], s_phase)) { ok = false; break; }
        s_phase ^= 1;
        tc_fence_after();
        const uint32_t okm = *const_cast<volatile uint32_t*>(&sm.keys_ok[tile % kOkRing]);
        float s[128];
        {
          uint32_t u0[32], u1[32], u2[32], u3[32];
          tmem_ld32(tS, u0);
          tmem_ld32(tS + 32, u1);
          tmem_ld32(tS + 64, u2);
          tmem_ld32(tS + 96, u3);
          tmem_ld_wait32(u0);
          reg_fence32(u1);
          reg_fence32(u2);
          reg_fence32(u3);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            s[i] = __uint_as_float(u0[i]);
            s[32 + i] = __uint_as_float(u1[i]);
            s[64 + i] = __uint_as_float(u2[i]);
            s[96 + i] = __uint_as_float(u3[i]);
          }
        }
        if (last < 127) {
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i > last) s[i] = kNegInf;
        }
        if (okm != 255u) {
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (((okm >> (i / 16)) & 1u) == 0) s[i] = kNegInf;
        }
        auto weights = [&]() -> float {
          const float2 sc2 = make_float2(sl2, sl2);
          const float2 nm2 = make_float2(-m, -m);
          float2 la = make_float2(0.f, 0.f), lb = make_float2(0.f, 0.f);
          if constexpr (kSplitP) {
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
              uint32_t hi[16], lo[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 arg =
                    __ffma2_rn(make_float2(s[cc * 32 + 2 * i], s[cc * 32 + 2 * i + 1]), sc2, nm2);
                const float2 e = make_float2(ex2(arg.x), ex2(arg.y));
                if (i & 1) lb = __fadd2_rn(lb, e); else la = __fadd2_rn(la, e);
                hi[i] = pack_bf16(e.x, e.y);
                lo[i] = pack_bf16(e.x - __uint_as_float(hi[i] << 16),
                                  e.y - __uint_as_float(hi[i] & 0xffff0000u));
              }
              tmem_st16(tS + cc * 16, hi);
              tmem_st16(tS + 64 + cc * 16, lo);
            }
          } else {
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float2 arg =
                  __ffma2_rn(make_float2(s[cc * 64 + 2 * i], s[cc * 64 + 2 * i + 1]), sc2, nm2);
              const float2 e = make_float2(ex2(arg.x), ex2(arg.y));
              if (i & 1) lb = __fadd2_rn(lb, e); else la = __fadd2_rn(la, e);
              pk[i] = pack_bf16(e.x, e.y);
            }
            tmem_st32(tS + cc * 32, pk);
          }
          }
          return (la.x + la.y) + (lb.x + lb.y);
        };
        float part = weights();  // the tile's row sum under m
        const bool few = first && last < 127;  // the row ends in this tile
        if (__any_sync(0xffffffffu, live && (few || !(part < kMostSum && l + part > kLeastSum)))) {
          float mx0 = s[0], mx1 = s[1], mx2 = s[2], mx3 = s[3];
#pragma unroll
          for (int i = 4; i < 124; i += 8) {
            mx0 = fmax3(mx0, s[i], s[i + 1]);
            mx1 = fmax3(mx1, s[i + 2], s[i + 3]);
            mx2 = fmax3(mx2, s[i + 4], s[i + 5]);
            mx3 = fmax3(mx3, s[i + 6], s[i + 7]);
          }
          mx0 = fmax3(mx0, s[124], s[125]);
          mx1 = fmax3(mx1, s[126], s[127]);
          const float mx = fmax3(fmaxf(mx0, mx1), mx2, mx3);
          // m to the size of what the row has, or gets: alpha is at most 1 / l
          float m_new = fmaxf(l > 0.f ? m + lg2(l) : kNegInf, mx * sl2);
          if (!(m_new > kNegInf)) m_new = m;
          // the weights stored first have landed before others follow them
          tmem_st_wait();
          if (!first) {
            // O_t must hold the finished P_t V of the previous key tile
            if (!wait(&sm.o_full[t], s_phase)) { ok = false; break; }
            tc_fence_after();
            const float alpha = l > 0.f ? ex2(m - m_new) : 0.f;
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t u[32];
              tmem_ld32(tO + cc * 32, u);
              tmem_ld_wait32(u);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                u[i] = __float_as_uint(__uint_as_float(u[i]) * alpha);
              tmem_st32(tO + cc * 32, u);
            }
            tmem_st_wait();
            l *= alpha;
          }
          m = m_new;
          part = weights();
        }
        l += part;
        first = false;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&sm.p_full[t]);
      }
      if (!ok) break;
      // ------------------------------------------------------- epilogue
      const Item& x = sm.item[r % kItems];
      const int nkv = x.n[t];
      if (x.n[1 - t] > nkv) tile += x.n[1 - t] - nkv;
      const int tok = row / p.per, rem = row - tok * p.per;
      const bool valid = tok < tile_tokens(p, x.e, t);
      if (nkv > 0) {
        if (!wait(&sm.o_full[t], s_phase ^ 1)) break;
        tc_fence_after();
      }
      // (a row without keys has l = 0; a NaN score stays)
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const float lse = l == 0.f ? kNegInf : (m + lg2(l)) * kLn2;
      const bool part = x.e.slot >= 0;
      const int64_t prow =
          (static_cast<int64_t>(x.e.slot) * p.Hkv + x.hk) * 256 + t * 128 + row;
      const int64_t token = x.e.tok0 + t * p.tpt + tok;
      const int64_t h = static_cast<int64_t>(x.hk) * p.G + rem;  // (direct: rem is the head)
      // 32-byte stores where the rows allow it: a whole sector per lane and store
      const bool wide = part || p.wide;
      float* f32 = part ? p.part_o + prow * D
                        : (p.o.dtype == LSX_F32
                               ? static_cast<float*>(p.o.data) + view_off(p.o, 0, h, token)
                               : nullptr);
      __nv_bfloat16* b16 = static_cast<__nv_bfloat16*>(p.o.data) + view_off(p.o, 0, h, token);
#pragma unroll
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t u[32];
        if (nkv > 0) {
          tmem_ld32(tO + cc * 32, u);
          tmem_ld_wait32(u);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) u[i] = 0u;
        }
        if (!valid) continue;
        float ov[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) ov[i] = l == 0.f ? 0.f : __uint_as_float(u[i]) * inv;
        if (f32 != nullptr) {
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(ov[i]);
          store_row(f32 + cc * 32, w, wide);
        } else {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = pack_bf16(ov[2 * i], ov[2 * i + 1]);
          store_row(b16 + cc * 32, w, wide);
        }
      }
      if (valid) {
        if (part)
          p.part_l[prow] = lse;
        else
          static_cast<float*>(p.lse.data)[view_off(p.lse, 0, h, token)] = lse;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_empty[r % kItems]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------- plan
struct PlanParams {
  const int32_t* kv_lens;
  const int32_t* cu_q;
  int batch;
  int64_t n_tokens, cap;  // packed tokens; keys a table row can hold
  int64_t Hkv;
  int tpt, sm_count;
  int max_entries, max_slots;  // room in the workspace (slots per kv head)
  Header* header;
  Entry* entries;
  CutUnit* cut;
  int* status;
};

struct Seq {
  int32_t q0, n, len;
};
__device__ __forceinline__ Seq plan_seq(const PlanParams& p, int b) {
  Seq s;
  const int64_t T = p.n_tokens;
  int64_t q0 = p.cu_q[b], q1 = p.cu_q[b + 1];
  q0 = q0 < 0 ? 0 : (q0 > T ? T : q0);
  q1 = q1 < q0 ? q0 : (q1 > T ? T : q1);
  s.q0 = static_cast<int32_t>(q0);
  s.n = static_cast<int32_t>(q1 - q0);
  s.len = p.kv_lens[b] < 0 ? 0 : p.kv_lens[b];
  return s;
}

// Key tiles of a pair whose last token is the i-th of its sequence.
__device__ __forceinline__ int32_t pair_tiles(int64_t cap, const Seq& s, int32_t i) {
  int64_t vis = static_cast<int64_t>(s.len) - s.n + i + 1;
  if (vis > cap) vis = cap;
  return vis > 0 ? static_cast<int32_t>((vis + 127) >> 7) : 0;
}

constexpr int kCutUnits = kPlanThreads;  // pairs that the cutting handles (two per SM is below)
constexpr int kBuckets = 64;

// What cutting costs, in the time of a key tile (1.6 us).  `big` items of about w
// tiles set the rounds over the SMs, all of them the work to be spread; an item
// costs kItemTiles besides its tiles (its first tile's chain, its result), and
// partials a merge (54 of 128 KB in a tile's time, 4 to start).
constexpr float kItemTiles = 4.f;
__host__ __device__ inline float cut_cost(float big, float w, float items, float tiles,
                                          float partials, int sm_count) {
  const float each = 1.f / sm_count;
  const float rounds = ceilf((big - 0.5f) * each) * (w + kItemTiles);
  const float spread = (tiles + kItemTiles * items) * each;
  return (rounds > spread ? rounds : spread) + (partials > 0 ? 4.f + partials * (1.f / 54.f) : 0.f);
}
// Numbers of pieces that are tried: 1 to 16, then about a fifth more each time.
constexpr int kCandidates = 32;
__device__ __forceinline__ int candidate(int i) {
  return i < 16 ? i + 1 : static_cast<int>(16.f * ex2(0.263034406f * (i - 15)));
}

// One block: the units of all sequences, whether and how to cut them, and the
// list of work, longest pieces first.  Latency-bound: 5 to 7 us; the next
// launch's set-up runs meanwhile.
__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PlanParams p) {
  extern __shared__ int32_t start[];  // [batch + 1] first pair of each sequence
  Seq* const seqs = reinterpret_cast<Seq*>(start + p.batch + 1);
  __shared__ int64_t wsum[kPlanThreads / 32];
  __shared__ int32_t tiles[kCutUnits], slot0[kCutUnits];
  __shared__ int32_t hist[kBuckets + 1];
  __shared__ unsigned long long best;
  __shared__ int32_t longest;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t = threadIdx.x, lane = t & 31;
  if (t == 0) { longest = 0; best = ~0ull; }
  if (t <= kBuckets) hist[t] = 0;
  const int pair_tok = 2 * p.tpt;
  // pairs of each sequence, exclusive sums
  const int per = (p.batch + kPlanThreads - 1) / kPlanThreads;
  const int b0 = t * per < p.batch ? t * per : p.batch;
  const int b1 = b0 + per < p.batch ? b0 + per : p.batch;
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) {
    const Seq s = plan_seq(p, b);
    seqs[b] = s;
    mine += (s.n + pair_tok - 1) / pair_tok;
    if (s.len > p.cap && s.n > 0) atomicCAS(p.status, 0, kStatusPage);
  }
  int64_t inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) wsum[t >> 5] = inc;
  __syncthreads();
  int64_t before = inc - mine, all_pairs = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < (t >> 5)) before += wsum[w];
    all_pairs += wsum[w];
  }
  // (more pairs than the workspace has room for: only if cu_q does not ascend)
  const int32_t n_pairs = static_cast<int32_t>(all_pairs < p.max_entries ? all_pairs : p.max_entries);
  for (int b = b0; b < b1; ++b) {
    start[b] = static_cast<int32_t>(before < n_pairs ? before : n_pairs);
    before += (seqs[b].n + pair_tok - 1) / pair_tok;
  }
  if (t == 0) start[p.batch] = n_pairs;
  __syncthreads();
  auto unit = [&](int i, Seq& s, int32_t& first) -> int32_t {
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= i) lo = mid; else hi = mid;
    }
    s = seqs[lo];
    first = (i - start[lo]) * pair_tok;
    return lo;
  };
  const bool may_cut = p.max_slots > 0 && n_pairs <= kCutUnits &&
                       n_pairs * p.Hkv < 2 * static_cast<int64_t>(p.sm_count);
  int32_t top = 0;
  for (int i = t; i < n_pairs; i += kPlanThreads) {
    Seq s;
    int32_t first;
    unit(i, s, first);
    const int32_t last = (first + pair_tok < s.n ? first + pair_tok : s.n) - 1;
    const int32_t n = pair_tiles(p.cap, s, last);
    if (may_cut) tiles[i] = n;
    top = n > top ? n : top;
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0 && top > 0) atomicMax(&longest, top);
  __syncthreads();
  int32_t piece = longest > 0 ? longest : 1;
  if (may_cut && longest >= 2 * kMinPiece) {
    // candidate k: the longest unit in k pieces, a warp each
    int64_t all_tiles = 0;
    for (int i = lane; i < n_pairs; i += 32) all_tiles += tiles[i];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) all_tiles += __shfl_xor_sync(0xffffffffu, all_tiles, d);
    for (int c = t >> 5; c < kCandidates; c += kPlanThreads / 32) {
      const int k = candidate(c);
      const int32_t w = (longest + k - 1) / k;
      if (k > 1 && w < kMinPiece) break;
      int32_t n = 0, big = 0, slots = 0;  // pieces, those over half of w, those with partials
      for (int i = lane; i < n_pairs; i += 32) {
        const int32_t q = tiles[i] > w ? (tiles[i] + w - 1) / w : 1;
        n += q;
        if (2 * tiles[i] > w * q) big += q;
        if (q > 1) slots += q;
      }
      n = __reduce_add_sync(0xffffffffu, n);
      big = __reduce_add_sync(0xffffffffu, big);
      slots = __reduce_add_sync(0xffffffffu, slots);
      if (k > 1 && slots > p.max_slots) continue;
      const float h = p.Hkv, cost = cut_cost(big * h, w, n * h, all_tiles * h, slots * h, p.sm_count);
      if (lane == 0)
        atomicMin(&best, (static_cast<unsigned long long>(cost * 16.f) << 32) |
                             static_cast<unsigned>(w));
    }
    __syncthreads();
    piece = static_cast<int32_t>(best & 0xffffffffu);
  }
  // pieces of each unit: equal, at most `piece` tiles
  auto cut = [&](int32_t n, int32_t& size) -> int32_t {
    const int32_t k = n > piece ? (n + piece - 1) / piece : 1;
    size = (n + k - 1) / k;
    return size > 0 ? (n + size - 1) / size : 1;
  };
  int32_t n_cut = 0;
  if (may_cut) {  // slots and list of the cut units, unit t in thread t
    int32_t size;
    const int32_t k = t < n_pairs ? cut(tiles[t], size) : 0;
    const int32_t need = k > 1 ? (1 << 16) + k : 0;  // (a unit, its slots)
    int32_t sum = need;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t o = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += o;
    }
    __syncthreads();  // (wsum was read above)
    if (lane == 31) wsum[t >> 5] = sum;
    __syncthreads();
    int32_t all = 0, ahead = sum - need;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < (t >> 5)) ahead += static_cast<int32_t>(wsum[w]);
      all += static_cast<int32_t>(wsum[w]);
    }
    n_cut = all >> 16;
    if (t < n_pairs) {
      slot0[t] = k > 1 ? ahead & 0xffff : -1;
      if (k > 1) {
        Seq s;
        int32_t first;
        unit(t, s, first);
        p.cut[ahead >> 16] = CutUnit{
            s.q0 + first, s.n - first < pair_tok ? s.n - first : pair_tok, ahead & 0xffff, k};
      }
    }
  }
  __syncthreads();
  const int32_t widest = piece > 0 ? piece : 1;
  auto bucket = [&](int32_t size) {  // 0: the longest
    const int32_t x = size * (kBuckets - 1) / widest;  // (fewer than 2^24 tiles)
    return kBuckets - 1 - (x < kBuckets ? x : kBuckets - 1);
  };
  // Every piece, piece-major, by whole warps: f(its bucket, -1 for none, the
  // lanes of the warp with the same one, the piece as an entry).
  const int rounds = longest > piece ? (longest + piece - 1) / piece : 1;  // a unit's most pieces
  auto each = [&](auto&& f) {
    const int32_t count = rounds * n_pairs;  // (rounds > 1: few pairs, few pieces)
    for (int32_t at = t; at - lane < count; at += kPlanThreads) {
      int32_t key = -1;
      Entry e{};
      if (at < count) {
        const int j = at / n_pairs, i = at - j * n_pairs;
        Seq s;
        int32_t first, size;
        e.b = unit(i, s, first);
        e.tok0 = s.q0 + first;
        e.ntok = s.n - first < pair_tok ? s.n - first : pair_tok;
        const int32_t n = pair_tiles(p.cap, s, first + e.ntok - 1);
        const int32_t k = cut(n, size);
        e.j0 = j * size;
        e.size = n - e.j0 < size ? n - e.j0 : size;
        e.len = static_cast<int32_t>(s.len > p.cap ? p.cap : s.len);
        e.lim0 = s.len - s.n + first;
        e.slot = k > 1 ? slot0[i] + j : -1;
        if (j < k) key = bucket(e.size);
      }
      f(key, __match_any_sync(0xffffffffu, key), e);
    }
  };
  each([&](int32_t key, uint32_t same, const Entry&) {
    if (key >= 0 && lane == __ffs(same) - 1) atomicAdd(&hist[key + 1], __popc(same));
  });
  __syncthreads();
  if (t < 32) {
    int32_t a = hist[1 + 2 * lane], b = hist[2 + 2 * lane];
    int32_t sum = a + b;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t o = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += o;
    }
    hist[1 + 2 * lane] = sum - b;
    hist[2 + 2 * lane] = sum;
  }
  __syncthreads();
  const int32_t total = hist[kBuckets];
  each([&](int32_t key, uint32_t same, const Entry& e) {
    const int leader = __ffs(same) - 1;
    int32_t at = 0;
    if (key >= 0 && lane == leader) at = atomicAdd(&hist[key], __popc(same));
    at = __shfl_sync(0xffffffffu, at, leader) + __popc(same & ((1u << lane) - 1u));
    if (key >= 0 && at < p.max_entries) p.entries[at] = e;
  });
  if (t == 0) *p.header = Header{total < p.max_entries ? total : p.max_entries, n_cut};
}

// ------------------------------------------------------------------ merge
struct FwdMergeParams {
  const Header* header;
  const CutUnit* cut;
  int64_t Hkv;
  int G, tpt;
  const float* part_o;
  const float* part_l;
  lsx_tensor o, lse;
};

// One warp per row of a cut unit, three blocks an SM (448 pieces of 128 KB 16.0 us
// with the events around the launch, at two blocks 19.0; four blocks take 1.8 us
// more for few rows).
template <int D>
__global__ void __launch_bounds__(256, 3) paged_fwd_merge_kernel(const FwdMergeParams p) {
  const int lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t rows = __ldcg(&p.header->n_cut) * p.Hkv * 256;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5; i < rows;
       i += step) {
    const int row = static_cast<int>(i & 255), t = row >> 7;
    const int64_t hk = (i >> 8) % p.Hkv;
    const int4 u = __ldcg(reinterpret_cast<const int4*>(p.cut) + (i >> 8) / p.Hkv);
    const CutUnit x{u.x, u.y, u.z, u.w};
    const int tok = (row & 127) / p.G;
    if (tok >= p.tpt || t * p.tpt + tok >= x.ntok) continue;
    RowMerge<D> sum;
    sum.take(p.part_o, p.part_l, x.n, lane,
             [&](int64_t c) { return ((x.first + c) * p.Hkv + hk) * 256 + row; });
    sum.store(p.o, p.lse, 0, hk * p.G + (row & 127) - tok * p.G, x.tok0 + t * p.tpt + tok, lane);
  }
}

// ------------------------------------------------------------------- host
size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// bf16 map with dims (innermost first) {D, n1, n2, n3}, element strides, box
// {64, b1, b2, b3}, 128-byte swizzle; elements outside read as zero.
bool encode4(CUtensorMap* map, const void* base, int64_t D, const int64_t (&n)[3],
             int64_t s1, int64_t s2, int64_t s3, uint32_t b1, uint32_t b2, uint32_t b3) {
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  // the stride of an extent-1 dimension is never used; give it a legal value
  if (n[0] == 1) s1 = D;
  if (n[1] == 1) s2 = s1 * n[0];
  if (n[2] == 1) s3 = s2 * n[1];
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)n[0], (cuuint64_t)n[1], (cuuint64_t)n[2]};
  cuuint64_t str[3] = {(cuuint64_t)(s1 * 2), (cuuint64_t)(s2 * 2), (cuuint64_t)(s3 * 2)};
  cuuint32_t box[4] = {64u, b1, b2, b3};
  cuuint32_t one[4] = {1u, 1u, 1u, 1u};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, str, box,
             one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_pages(CUtensorMap* map, const lsx_tensor& t) {
  return encode4(map, t.data, t.D, {t.N, t.H, t.B}, t.stride_n, t.stride_h, t.stride_b,
                 static_cast<uint32_t>(t.N < 128 ? t.N : 128), 1, 1);
}

template <int D, bool kSplitP>
int launch_tiles(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                 const FwdParams& p, int64_t grid, bool early, int device, cudaStream_t s) {
  const size_t smem = sizeof(Smem<D>) + 1024;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(paged_fwd_kernel<D, kSplitP>, static_cast<int>(smem), device, done)) return LSX_ERR_LAUNCH;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(384);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = early ? 1 : 0;
  timing_begin(kKidPagedFwd, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_fwd_kernel<D, kSplitP>, tq, tk, tv, p);
  timing_end(kKidPagedFwd, s);
  return e == cudaSuccess ? LSX_OK : LSX_ERR_LAUNCH;
}

struct FwdLayout {
  int64_t max_entries, max_slots;
  size_t entries, cut, part_l, part_o, total;
};
FwdLayout fwd_layout(const lsx_tensor& q, const lsx_tensor& kp, int64_t batch, int64_t max_pages,
                     int sm_count) {
  FwdLayout x;
  const int64_t G = q.H / kp.H, tpt = G <= 128 ? 128 / G : 1;
  const int64_t tiles = ceil_div(max_pages * kp.N, 128);
  x.max_slots = tiles >= 2 * kMinPiece ? kPiecesPerSm * sm_count / kp.H : 0;
  if (x.max_slots < 2) x.max_slots = 0;
  x.max_entries = ceil_div(q.N, 2 * tpt) + batch + x.max_slots;
  x.entries = 256;
  x.cut = x.entries + align256(static_cast<size_t>(x.max_entries) * sizeof(Entry));
  x.part_l = x.cut + align256(kCutUnits * sizeof(CutUnit));
  const size_t rows = static_cast<size_t>(x.max_slots * kp.H) * 256;
  x.part_o = x.part_l + align256(rows * 4);
  x.total = x.part_o + align256(rows * static_cast<size_t>(q.D) * 4);
  return x;
}

}  // namespace

PrefixPlan prefix_plan(int64_t B, int64_t per, int64_t hkv, int64_t prefix_len, int sm_count) {
  PrefixPlan x;
  // few sequences: both row tiles get half of them, so that each one's softmax
  // runs under the other's products
  x.tpt = static_cast<int>(128 / per);
  if (B < 2 * x.tpt) x.tpt = static_cast<int>(ceil_div(B, 2));
  const int64_t units = ceil_div(B, 2 * x.tpt), tiles = ceil_div(prefix_len, 128);
  auto cost = [&](int64_t k) {
    const float n = static_cast<float>(units * hkv * k);
    return cut_cost(n, static_cast<float>(ceil_div(tiles, k)), n,
                    static_cast<float>(units * hkv * tiles), n, sm_count);
  };
  int64_t best = 1;
  float least = cost(1);
  for (int64_t k = 2; units * hkv * k <= kPiecesPerSm * sm_count && ceil_div(tiles, k) >= kMinPiece;
       ++k) {
    const float c = cost(k);
    if (c < least) { best = k; least = c; }
  }
  x.size = static_cast<int>(ceil_div(tiles, best));
  x.pieces = static_cast<int>(ceil_div(tiles, x.size));
  x.rows = units * x.pieces * hkv * 256;
  return x;
}

int launch_prefix(const lsx_tensor& q, const lsx_tensor& k_pages, const lsx_tensor& v_pages,
                  const PagedCache& prefix, int64_t prefix_len, const PrefixPlan& plan,
                  float scale, bool split_p, float* part_o, float* part_l,
                  const DeviceCtx& ctx, cudaStream_t s) {
  FwdParams p;
  p.c = prefix;
  p.Hkv = k_pages.H;
  p.G = static_cast<int>(q.H / k_pages.H);
  p.per = static_cast<int>(p.G * q.N);
  p.tpt = plan.tpt;
  p.header = nullptr;
  p.entries = nullptr;
  p.u_tokens = static_cast<int32_t>(q.B);
  p.u_len = static_cast<int32_t>(prefix_len);
  p.u_pieces = plan.pieces;
  p.u_size = plan.size;
  p.scale_log2 = scale * kLog2e;
  p.o = q;  // (not written: every row goes to the partials)
  p.lse = q;
  p.wide = false;
  p.part_o = part_o;
  p.part_l = part_l;
  p.status = ctx.status;
  p.wait_ns = ctx.wait_ns;
  CUtensorMap tq, tk, tv;
  if (!encode4(&tq, q.data, q.D, {q.H, q.N, q.B}, q.stride_h, q.stride_n, q.stride_b,
               static_cast<uint32_t>(p.G), static_cast<uint32_t>(q.N),
               static_cast<uint32_t>(p.tpt)) ||
      !encode_pages(&tk, k_pages) || !encode_pages(&tv, v_pages))
    return LSX_ERR_LAUNCH;
  const int64_t items = plan.rows / 256;
  const int64_t grid = items < ctx.sm_count ? items : ctx.sm_count;
  auto launch = q.D == 128 ? (split_p ? launch_tiles<128, true> : launch_tiles<128, false>)
                           : (split_p ? launch_tiles<64, true> : launch_tiles<64, false>);
  return launch(tq, tk, tv, p, grid, false, ctx.device, s);
}

size_t paged_fwd_workspace(const lsx_tensor& q, const lsx_tensor& k_pages, int64_t batch,
                           int64_t max_pages, int sm_count) {
  return fwd_layout(q, k_pages, batch, max_pages, sm_count).total;
}

int launch_paged_fwd(const lsx_tensor& q, const lsx_tensor& k_pages, const lsx_tensor& v_pages,
                     const PagedCache& c, const int32_t* kv_lens, const int32_t* cu_q,
                     int64_t batch, float scale, const lsx_tensor& o, const lsx_tensor& lse,
                     void* workspace, const DeviceCtx& ctx, cudaStream_t s) {
  const FwdLayout x = fwd_layout(q, k_pages, batch, c.max_pages, ctx.sm_count);
  char* ws = static_cast<char*>(workspace);
  FwdParams p;
  p.c = c;
  p.Hkv = k_pages.H;
  p.G = static_cast<int>(q.H / k_pages.H);
  p.per = p.G;
  p.tpt = 128 / p.G;
  p.header = reinterpret_cast<Header*>(ws);
  p.entries = reinterpret_cast<Entry*>(ws + x.entries);
  p.u_tokens = p.u_len = p.u_pieces = p.u_size = 0;
  p.scale_log2 = scale * kLog2e;
  p.o = o; p.lse = lse;
  const int64_t unit = o.dtype == LSX_F32 ? 8 : 16;  // elements of 32 bytes
  p.wide = reinterpret_cast<uintptr_t>(o.data) % 32 == 0 && o.stride_h % unit == 0 &&
           o.stride_n % unit == 0;
  p.part_o = reinterpret_cast<float*>(ws + x.part_o);
  p.part_l = reinterpret_cast<float*>(ws + x.part_l);
  p.status = ctx.status;
  p.wait_ns = ctx.wait_ns;
  CUtensorMap tq, tk, tv;
  if (!encode4(&tq, q.data, q.D, {q.H, q.N, 1}, q.stride_h, q.stride_n, 0,
               static_cast<uint32_t>(p.G), static_cast<uint32_t>(p.tpt), 1) ||
      !encode_pages(&tk, k_pages) || !encode_pages(&tv, v_pages))
    return LSX_ERR_LAUNCH;
  PlanParams pp;
  pp.kv_lens = kv_lens;
  pp.cu_q = cu_q;
  pp.batch = static_cast<int>(batch);
  pp.n_tokens = q.N;
  pp.cap = static_cast<int64_t>(c.max_pages) << c.shift;
  pp.Hkv = p.Hkv;
  pp.tpt = p.tpt;
  pp.sm_count = ctx.sm_count;
  pp.max_entries = static_cast<int>(x.max_entries);
  pp.max_slots = static_cast<int>(x.max_slots);
  pp.header = reinterpret_cast<Header*>(ws);
  pp.entries = reinterpret_cast<Entry*>(ws + x.entries);
  pp.cut = reinterpret_cast<CutUnit*>(ws + x.cut);
  pp.status = ctx.status;
  timing_begin(kKidPagedPlan, s);
  const int plan_smem = static_cast<int>((batch + 1) * sizeof(int32_t) + batch * sizeof(Seq));
  static std::atomic<uint64_t> done{0};
  if (plan_smem > 40 * 1024 &&
      !allow_smem(paged_plan_kernel, kMaxMapBatch * 16 + 16, ctx.device, done))
    return LSX_ERR_LAUNCH;
  paged_plan_kernel<<<1, kPlanThreads, plan_smem, s>>>(pp);
  timing_end(kKidPagedPlan, s);
  if (cudaGetLastError() != cudaSuccess) return LSX_ERR_LAUNCH;
  const int64_t most = x.max_entries * p.Hkv;
  const int64_t grid = most < ctx.sm_count ? most : ctx.sm_count;
  const int rc = q.D == 128 ? launch_tiles<128, false>(tq, tk, tv, p, grid, true, ctx.device, s)
                            : launch_tiles<64, false>(tq, tk, tv, p, grid, true, ctx.device, s);
  if (rc != LSX_OK || x.max_slots == 0) return rc;
  const FwdMergeParams mp{pp.header, pp.cut, p.Hkv, p.G, p.tpt, p.part_o, p.part_l, o, lse};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(3 * ctx.sm_count));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  timing_begin(kKidPagedMerge, s);
  const cudaError_t e = q.D == 128 ? cudaLaunchKernelEx(&cfg, paged_fwd_merge_kernel<128>, mp)
                                   : cudaLaunchKernelEx(&cfg, paged_fwd_merge_kernel<64>, mp);
  timing_end(kKidPagedMerge, s);
  return e == cudaSuccess ? LSX_OK : LSX_ERR_LAUNCH;
}

}  // namespace lsx
