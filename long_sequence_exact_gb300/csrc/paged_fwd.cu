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
// call: heads of 128 124 us with one product, 161 with both, of 64 98 and 141.  Over an
// 8-bit cache the same holds for prompts whose results are f32, by way of a bf16 copy;
// tiles widened in place keep 11 and 22 bits (below), so that there the bits follow from
// the number of rows, and a workspace without room for the copy keeps the more of them.
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

#include <type_traits>

#include "paged.h"
#include "paged_merge.cuh"
#include "ptx.cuh"
#include "q8.cuh"
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

// 8-bit caches: tiles as they come, the exponent bytes of their rows, and what the
// softmax needs of each tile.
struct TileInfo {
  float factor;  // of its scores
  float shift;   // its weights are 2^shift of what the row sums count; NaN: kShift, and
                 // O's unit is another than before
  float unit;    // what O is in units of
  float grow;    // the unit before in terms of it
};
template <int D, bool Q8>
struct RawTiles {};
template <int D>
struct RawTiles<D, true> {
  static constexpr int kRaw = 1;          // tiles ahead, of keys and of values (more: no faster)
  static constexpr int kExps = kRaw + 2;  // (a tile's are read again with its values)
  static constexpr int kInfos = Cfg<D>::kStages + 2;
  alignas(1024) uint8_t k[kRaw][128 * D];
  uint8_t v[kRaw][128 * D];
  alignas(16) uint8_t exps[kExps][2][128];
  alignas(16) TileInfo info[kInfos];
  float top[4];      // largest |q| that the warps found
  uint64_t q_top;    // all four are in `top`
  uint64_t q_ready;  // Q in f16
  uint64_t k_full[kRaw], k_empty[kRaw], v_full[kRaw], v_empty[kRaw];
};

template <int D, bool Q8>
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
  RawTiles<D, Q8> raw;
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
  const uint8_t *ks, *vs;  // 8-bit caches: the rows' exponent bytes
  int64_t ks_sp, ks_sh, vs_sp, vs_sh;
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

// ------------------------------------------------------------ 8-bit caches
// Few query rows a key, and shared prefixes: the tiles are loaded as they are and widened
// on their way to the products (many rows: see dense_rows).  The products are of f16, which
// holds an e4m3 exactly; a warpgroup of its own (512 threads in all: warps 12..15, which
// also turn Q into f16 in place and clear the values past the last key) widens the tiles,
// one conversion and one multiplication for two values.  Warps 0 and 3 load into a ring of
// raw tiles, and the ring of steps is filled by the widening warps.
//
// Bound: the chain load, widen, product, softmax; no pipe is above 50%.  The roles share
// the instruction cache: with the bf16 kernel's softmax (128 scores in registers, all
// unrolled) its hit rate was 0.80 instead of 0.92 and every role slower, so here the
// softmax goes over TMEM twice, 32 scores a turn, for the maximum and for the weights.
// 12 sequences' 150 tokens after up to 9000 keys, 24 heads over 8 of 64: 97 us
// (105 before; bf16, twice the bytes: 76), tensor pipe 20%, issue 47%; 131072 keys under
// 256 rows, 8 heads of 128: 125 us (147; bf16 108), tensor pipe 46%.
// The rows' powers of two stay out of the softmax's loop:
// - A tile's rows become value * 2^(e - E + kRise), E the largest exponent of the tile's
//   rows: at most 448 * 2^7, an f16 still, exact down to e = E - 22, and below that to
//   half of f16's last step, 2^(E - 32) in all (a row's largest value is above 224 * 2^e).
//   For keys 2^(E - kRise) is a factor of all the tile's scores, for values an exponent of
//   all its weights.
// - Q becomes f16 times a power of two that brings the largest element of an item's
//   rows to [2^14, 2^15): 8 bits are kept exactly down to 2^-31 of it.
// - P is kept as f16, 11 bits.  The weights that are stored are 2^(kShift + E - E_ref) of
//   what the row sums count, E_ref the exponent of O's unit: below f16's normal range they
//   are off by up to 2^-33 of the row's largest, times 448 2^E_ref.  E_ref is the first
//   tile's E (that has rows), and a later one's where it is above that by more than kSlack:
//   O is then divided by as much, and the row sums stay as they are (with one unit for an
//   item, m had to make up for it: sums and LSE lost bits where values grew by 2^100).  An E
//   further than kFar below E_ref counts as that much, so that the sums, taken of the
//   weights as they are stored before they are f16, stay in range.  m starts at the first
//   tile's maximum and moves where a weight would be stored as more than 2^15.  f32
//   results: a weight's remainder is a second f16.
constexpr int kShift = 8;
constexpr int kRise = 7;
constexpr int kSlack = 6;
constexpr int kFar = 64;

// A tile [128][D] of e4m3 (rows of 128 bytes with the 128-byte swizzle, of 64 without)
// to the f16 tile that the products read; thread t of 128.  `there`: a bit for each of the
// thread's four rows; `clear`: those that are not become zeros.  A quarter of a warp's
// 16-byte accesses have to fall on different banks, in the 8-bit tile (16 values of four
// columns' pieces in a row) and in the f16 one (two pieces): its eight threads take half a
// row each of two rows that differ in bits 0 and 2 (heads of 64: in bit 0).
//
// A row's power of two is an f16 factor.  f16 has those down to 2^-24 and the smallest
// value is 2^-9, so that the first product stops at 2^-14, where it is exact; rows below
// that (rare: 2^22 smaller than the tile's largest) are multiplied once more, where the one
// rounding is.
template <int D>
__device__ __forceinline__ int widen_row(int t) {
  const int pair = (t >> 3) & 3, sel = (t >> 2) & 1;
  return (t >> 5) * 32 + (D == 128 ? (sel ? pair ^ 5 : pair) : 2 * pair + sel);
}
template <int D>
__device__ __forceinline__ void widen_tile(const uint8_t* src, const uint8_t* exps, int top,
                                           uint32_t there, bool clear, __nv_bfloat16* dst,
                                           int t) {
  const int c = t & 3, r = widen_row<D>(t), sw = r & 7;
  const uint8_t* in = src + r * D;
  uint8_t* out = reinterpret_cast<uint8_t*>(dst) + r * 128;
  const int at0 = ((2 * c) ^ sw) << 4, at1 = ((2 * c + 1) ^ sw) << 4;
  int least = 1;
#pragma unroll
  for (int i = 0; i < 4; ++i, in += 8 * D, out += 8 * 128, there >>= 1) {
    uint4 x[D / 64];
#pragma unroll
    for (int half = 0; half < D / 64; ++half)
      x[half] = *reinterpret_cast<const uint4*>(in + ((D == 128 ? (half * 4 + c) ^ sw : c) << 4));
    // (two f16 powers by their exponent fields; a row that is not there has any)
    const int field = static_cast<int>(exps[r + 8 * i]) - top + kRise + 15;
    if ((there & 1u) != 0) least = min(least, field);
    uint32_t f = static_cast<uint32_t>(max(field, 1)) * 0x04000400u;
    if (clear && (there & 1u) == 0) {
      f = 0;
#pragma unroll
      for (int half = 0; half < D / 64; ++half) x[half] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int half = 0; half < D / 64; ++half) {
      const uint32_t w[4] = {x[half].x, x[half].y, x[half].z, x[half].w};
      uint32_t y[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        e4m3_f16x4(w[k], y[2 * k], y[2 * k + 1]);
        y[2 * k] = mul_f16x2(y[2 * k], f);
        y[2 * k + 1] = mul_f16x2(y[2 * k + 1], f);
      }
      uint8_t* const line = out + half * 128 * 128;
      *reinterpret_cast<uint4*>(line + at0) = make_uint4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<uint4*>(line + at1) = make_uint4(y[4], y[5], y[6], y[7]);
    }
  }
  if (!__any_sync(0xffffffffu, least < 1)) return;  // (by warps: a branch by threads 2% slower)
  out -= 4 * 8 * 128;
#pragma unroll 1
  for (int i = 0; i < 4; ++i, out += 8 * 128) {
    const int e = static_cast<int>(exps[r + 8 * i]) - top + kRise + 14;
    if (e >= 0) continue;
    const float f1 = q8_power(max(e, -126));
    const uint32_t f = pack_f16(f1, f1);
#pragma unroll 1
    for (int n = 0; n < D / 32; ++n) {
      uint4* const at = reinterpret_cast<uint4*>(out + (n >> 1) * 128 * 128 + ((n & 1) ? at1 : at0));
      const uint4 y = *at;
      *at = make_uint4(mul_f16x2(y.x, f), mul_f16x2(y.y, f), mul_f16x2(y.z, f), mul_f16x2(y.w, f));
    }
  }
}

// Largest exponent byte of a tile's rows that are there (0 where none is), by a warp.
__device__ __forceinline__ int top_exponent(const uint8_t* exps, uint32_t groups, int rows, int lane) {
  const uint32_t w = reinterpret_cast<const uint32_t*>(exps)[lane];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (4 * lane + i < rows) top = max(top, (w >> (8 * i)) & 255u);
  if (((groups >> (lane >> 2)) & 1u) == 0) top = 0;
  return static_cast<int>(__reduce_max_sync(0xffffffffu, top));
}

template <int D, bool kSplitP, bool Q8>
__global__ void __launch_bounds__(Q8 ? 512 : 384, 1)
    paged_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const FwdParams p) {
  using C = Cfg<D>;
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  using Sm = Smem<D, Q8>;
  Sm& sm = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
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
      mbar_init(&sm.full[s], Q8 ? 4 : 1);  // (8 bits: the warps that widen the tiles)
      mbar_init(&sm.empty[s], 1);
    }
    if constexpr (Q8) {
      mbar_init(&sm.raw.q_top, 4);
      mbar_init(&sm.raw.q_ready, 4);
      for (int i = 0; i < sm.raw.kRaw; ++i) {
        mbar_init(&sm.raw.k_full[i], 1 + 32);
        mbar_init(&sm.raw.k_empty[i], 4);
        mbar_init(&sm.raw.v_full[i], 1);
        mbar_init(&sm.raw.v_empty[i], 4);
      }
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&sm.item_full[i], 1);
      // MMA thread, 8 softmax warps, warps 2 and 3 (8 bits: 3 and 12 to 15)
      mbar_init(&sm.item_empty[i], Q8 ? 14 : 11);
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
  // 8 bits: 128 * 96 + 256 * 152 + 128 * 112 = 65,536 = 512 * 128
  if (warp < 4) {
    regs_dec<Q8 ? 96 : (D == 64 ? 88 : 104)>();
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
        if constexpr (Q8) {
          // keys through a ring of their own, with the exponents of keys and values
          using Raw = RawTiles<D, true>;
          for (int j = 0; j < nkv; ++j) {
            const int32_t mine = next;
            next = group_page(x, j + 1, nkv);
            const bool exists = mine >= 0 && mine < p.c.n_pages;
            if (lane < 8 && !exists && (x.e.j0 + j) * 128 + lane * 16 < x.e.len)
              atomicCAS(p.status, 0, kStatusPage);
            const uint32_t mask = __ballot_sync(0xffffffffu, exists) & 255u;
            const int page = box_page(mine);
            const int slot = count % Raw::kRaw;
            uint64_t* const bar = &sm.raw.k_full[slot];
            if (count >= Raw::kRaw &&
                !wait_all(&sm.raw.k_empty[slot], ((count / Raw::kRaw) & 1) ^ 1)) {
              ok = false;
              break;
            }
            if (lane == 0) {
              // (the word of 8 tiles ago: the tile kRaw ago has been widened, so the one
              // kRaw + stages + 1 ago has been through both products)
              *const_cast<volatile uint32_t*>(&sm.keys_ok[count % kOkRing]) = mask;
              mbar_arrive_expect_tx(bar, 128 * D);
            }
            __syncwarp();
            if (lane < boxes)
              tma_load_4d(&sm.raw.k[slot][box * rows * D], &tm_k, bar, 0, page_row(x, j), x.hk, page);
            // lanes 0..7 the keys' exponents, 8..15 the values'
            const int32_t group_at = __shfl_sync(0xffffffffu, mine, lane & 7);
            if (lane < 16 && ((mask >> (lane & 7)) & 1u) != 0) {
              const int row = ((x.e.j0 + j) * 128 + (lane & 7) * 16) & ((1 << p.c.shift) - 1);
              cp_async16(&sm.raw.exps[count % Raw::kExps][lane >> 3][(lane & 7) * 16],
                         lane < 8 ? p.ks + group_at * p.ks_sp + x.hk * p.ks_sh + row
                                  : p.vs + group_at * p.vs_sp + x.hk * p.vs_sh + row);
            }
            cp_async_arrive(bar);
            ++count;
          }
        } else {
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
        }
        if (!ok) break;
      }
      if (lane == 0 && *guard.abort != 0) {
        // gave up: the copies in flight land before the block ends
        drain_wait(&sm.q_full, qe_phase ^ 1, p.wait_ns);
        if constexpr (Q8) {
          constexpr uint32_t kRaw = RawTiles<D, true>::kRaw;
          for (uint32_t i = count > kRaw ? count - kRaw : 0; i < count; ++i)
            drain_wait(&sm.raw.k_full[i % kRaw], (i / kRaw) & 1, p.wait_ns);
        } else {
          for (uint32_t i = steps > kStages ? steps - kStages : 0; i < steps; ++i)
            drain_wait(&sm.full[i % kStages], (i / kStages) & 1, p.wait_ns);
        }
      }
    } else if (warp == 3) {
      // ----------------------------------------------------------- values
      // (the step's barrier is armed for both tiles by warp 0; 8 bits: a ring of their own)
      uint32_t stage = 0, phase = 0, raw = 0;
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
            if constexpr (Q8) {
              constexpr int kRaw = RawTiles<D, true>::kRaw;
              const int slot = raw % kRaw;
              uint64_t* const bar = &sm.raw.v_full[slot];
              if (raw >= kRaw && !wait_all(&sm.raw.v_empty[slot], ((raw / kRaw) & 1) ^ 1)) {
                ok = false;
                break;
              }
              if (lane == 0) mbar_arrive_expect_tx(bar, 128 * D);
              __syncwarp();
              if (lane < boxes)
                tma_load_4d(&sm.raw.v[slot][box * rows * D], &tm_v, bar, 0, page_row(x, j - 1), x.hk,
                            page);
              ++raw;
            } else {
              if (!wait_all(&sm.empty[stage], phase ^ 1)) { ok = false; break; }
              if (lane < boxes * C::kSub)
                tma_load_4d(&sm.v[stage][at], &tm_v, &sm.full[stage], sub * 64,
                            page_row(x, j - 1), x.hk, page);
            }
          }
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
      }
      if constexpr (Q8) {  // gave up: the copies in flight land before the block ends
        constexpr uint32_t kRaw = RawTiles<D, true>::kRaw;
        if (lane == 0 && *guard.abort != 0)
          for (uint32_t i = raw > kRaw ? raw - kRaw : 0; i < raw; ++i)
            drain_wait(&sm.raw.v_full[i % kRaw], (i / kRaw) & 1, p.wait_ns);
      }
    } else if (warp == 1 && lane == 0) {
      // ------------------------------------------------------ MMA issuer
      constexpr uint32_t kIdS = Q8 ? idesc_f16_f32(128, 128, 0, 0) : idesc_bf16_f32(128, 128, 0, 0);
      constexpr uint32_t kIdO = Q8 ? idesc_f16_f32(128, D, 0, 1) : idesc_bf16_f32(128, D, 0, 1);
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
        uint32_t q0 = q_lo + t * kTileDesc, k0 = k_lo + stage * kTileDesc, d = tmem + t * 128;
        // (8 bits: with the fewer registers of a warp here, the steps' descriptors are not to
        // be kept across the loop, where they would spill)
        if constexpr (Q8) asm volatile("" : "+r"(q0), "+r"(k0), "+r"(d));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss_lo(d, q0 + static_cast<uint32_t>(kmajor_step(kk, 128)), qk_hi,
                    k0 + static_cast<uint32_t>(kmajor_step(kk, 128)), qk_hi, kIdS,
                    kk > 0 ? 1u : 0u);
        mma_commit(&sm.s_full[t]);
      };
      auto issue_pv = [&](int t, uint32_t stage, uint32_t acc0) {
        uint32_t v0 = v_lo + stage * kTileDesc, d = tmem + t * 128;
        if constexpr (Q8) asm volatile("" : "+r"(v0), "+r"(d));
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts_lo(d + 256, d + kk * 8,
                    v0 + static_cast<uint32_t>(mnmajor_step(kk)), v_hi, kIdO, kk > 0 ? 1u : acc0);
        if constexpr (kSplitP) {  // what P's rounding left out, from the columns behind
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts_lo(d + 256, d + 64 + kk * 8,
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
        const int tail = Q8 ? -1 : tail_tile(p, x.e, nkv);
        mbar_arrive(&sm.item_empty[r % kItems]);
        uint64_t* q_bar = &sm.q_full;
        if constexpr (Q8) q_bar = &sm.raw.q_ready;
        if (!mbar_wait(q_bar, q_phase, guard)) break;
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
#pragma unroll(Q8 ? 1 : 2)
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
    } else if (!Q8 && warp == 2) {
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
  } else if (Q8 && warp >= 12) {
    regs_dec<112>();
    if constexpr (Q8) {
      // --------------------------------------- queries and tiles to f16
      using Raw = RawTiles<D, true>;
      constexpr uint32_t kRaw = Raw::kRaw;
      const int t = threadIdx.x - 384;
      uint32_t stage = 0, phase = 0, count = 0, values = 0, q_phase = 0;
      bool ok = true;
      auto take = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, guard)) != 0;
      };
      for (uint32_t r = 0; ok; ++r) {
        if (!take(&sm.item_full[r % kItems], (r / kItems) & 1)) break;
        const Item& x = sm.item[r % kItems];
        if (x.hk < 0) break;
        const int nkv = x.n[0] > x.n[1] ? x.n[0] : x.n[1];
        const int left = x.e.len - x.e.j0 * 128;  // rows of the item's first tile on
        const int rows0 = tile_tokens(p, x.e, 0) * p.per, rows1 = tile_tokens(p, x.e, 1) * p.per;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.item_empty[r % kItems]);
        if (!take(&sm.q_full, q_phase)) break;
        q_phase ^= 1;
        // Queries, 16 bytes of a row at a time, in place.  (Rows of no token of the item
        // may hold anything; infinities and NaN do not count and stay what they are.)
        constexpr int kPasses = D / 4;  // of 16 lines of 128 bytes
        uint8_t* const q8 = reinterpret_cast<uint8_t*>(sm.q) + t * 16;
        uint32_t top2 = 0;
#pragma unroll 2
        for (int i = 0; i < kPasses; ++i) {
          const int line = i * 16 + (t >> 3);  // [tile][64-column half][row]
          const int row = line & 127, tile = line / (128 * C::kSub);
          if (row < (tile == 0 ? rows0 : rows1)) {
            const uint4 v = *reinterpret_cast<const uint4*>(q8 + i * 2048);
            const uint32_t w[4] = {v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu,
                                   v.w & 0x7fff7fffu};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (__vcmpgeu2(w[k], 0x7f807f80u) == 0u) top2 = __vmaxu2(top2, w[k]);
          }
        }
        const uint32_t top = __reduce_max_sync(0xffffffffu, max(top2 & 0xffffu, top2 >> 16));
        // (a wait with a limit, as all are here: a warp whose wait for the queries ran out has
        // left, and does not come to a barrier)
        if (lane == 0) {
          sm.raw.top[warp - 12] = __uint_as_float(top << 16);
          mbar_arrive(&sm.raw.q_top);
        }
        if (!take(&sm.raw.q_top, q_phase ^ 1)) break;
        const float most = fmaxf(fmaxf(sm.raw.top[0], sm.raw.top[1]),
                                 fmaxf(sm.raw.top[2], sm.raw.top[3]));
        int eq = static_cast<int>(__float_as_uint(most) >> 23) - 127 - 14;
        if (eq < -126) eq = -126;
        const float qf = q8_power(-eq);
#pragma unroll 2
        for (int i = 0; i < kPasses; ++i) {
          uint4* const at = reinterpret_cast<uint4*>(q8 + i * 2048);
          const uint4 v = *at;
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            y[k] = pack_f16(__uint_as_float(w[k] << 16) * qf, __uint_as_float(w[k] & 0xffff0000u) * qf);
          *at = make_uint4(y[0], y[1], y[2], y[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.raw.q_ready);
        const float scale = p.scale_log2 * q8_power(-kRise) * q8_power(eq);
        // of O's unit and of V's tile (weights of a tile without rows are 0 under any exponent)
        int e_ref = 127, e_values = 127;
        bool none = true;
        for (int j = 0; j <= nkv && nkv > 0; ++j) {
          // step j: V of tile j - 1 and K of tile j, as everywhere
          if (!take(&sm.empty[stage], phase ^ 1)) { ok = false; break; }
#pragma unroll 1
          for (int kv = 1; kv >= 0; --kv) {
            if (kv == 0 ? j == nkv : j == 0) continue;
            const uint32_t n = kv == 0 ? count : values;
            const int slot = n % kRaw, rows = left - (j - kv) * 128;
            if (!take(kv == 0 ? &sm.raw.k_full[slot] : &sm.raw.v_full[slot], (n / kRaw) & 1)) {
              ok = false;
              break;
            }
            const uint32_t groups = *const_cast<volatile uint32_t*>(&sm.keys_ok[n % kOkRing]);
            const uint8_t* const exps = sm.raw.exps[n % Raw::kExps][0];
            uint32_t there = 0;  // the thread's rows that are
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = widen_row<D>(t) + 8 * i;
              if (((groups >> (row >> 4)) & 1u) != 0 && row < rows) there |= 1u << i;
            }
            int top = e_values;
            if (kv == 0) {
              const int of_k = top_exponent(exps, groups, rows, lane);
              const int of_v = top_exponent(exps + 128, groups, rows, lane);
              top = of_k > 0 ? of_k : 127;
              float shift = __uint_as_float(0x7fffffffu), grow = 1.f;
              if (of_v > (none ? 0 : e_ref + kSlack)) {
                grow = none ? 1.f : q8_power(e_ref - of_v);
                e_ref = e_values = of_v;
                none = false;
              } else {
                if (of_v > 0) e_values = max(of_v, e_ref - kFar);
                shift = static_cast<float>(e_values - e_ref + kShift);
              }
              if (t == 0)
                // (a factor of 0 or infinity would make masked scores NaN; scores that the
                // bounds change are 0 or infinite all the same)
                sm.raw.info[n % Raw::kInfos] =
                    TileInfo{fminf(fmaxf(scale * q8_scale(top), 1.17549435e-38f), 3.4e38f),
                             shift, q8_power(e_ref - 127 - kShift - kRise), grow};
            }
            widen_tile<D>(kv == 0 ? sm.raw.k[slot] : sm.raw.v[slot], exps + kv * 128, top, there,
                          kv == 1, kv == 0 ? sm.k[stage] : sm.v[stage], t);
            __syncwarp();
            if (lane == 0) mbar_arrive(kv == 0 ? &sm.raw.k_empty[slot] : &sm.raw.v_empty[slot]);
            if (kv == 0) ++count; else ++values;
          }
          if (!ok) break;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.full[stage]);
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
      }
    }
  } else {
    regs_inc<Q8 ? 152 : (D == 64 ? 208 : 200)>();
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
      float m = 0.f, l = 0.f, unit = 1.f;  // (unit: of O, 8 bits)
      bool ok = true, first = true;
      for (; left > 0; --left, ++tile, last -= 128) {
        if (!wait(&sm.s_full[t], s_phase)) { ok = false; break; }
        s_phase ^= 1;
        tc_fence_after();
        const uint32_t okm = *const_cast<volatile uint32_t*>(&sm.keys_ok[tile % kOkRing]);
        // O_t under a new reference, and times `unit_by`; it must hold the finished P_t V of
        // the tile before
        auto rescale = [&](float m_new, float unit_by) {
          if (!wait(&sm.o_full[t], s_phase)) return false;
          tc_fence_after();
          const float alpha = l > 0.f ? ex2(m - m_new) : 0.f;
#pragma unroll
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t u[32];
            tmem_ld32(tO + cc * 32, u);
            tmem_ld_wait32(u);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              u[i] = __float_as_uint(__uint_as_float(u[i]) * (alpha * unit_by));
            tmem_st32(tO + cc * 32, u);
          }
          tmem_st_wait();
          l *= alpha;
          return true;
        };
        if constexpr (Q8) {
          const TileInfo& info = sm.raw.info[tile % RawTiles<D, true>::kInfos];
          const float f = info.factor;
          float shift = info.shift;
          unit = info.unit;
          // The maximum first, 32 scores at a time; masked ones are written back.  (In short
          // loops: see the instruction cache above.)
          float mx = kNegInf;
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            uint32_t u[32];
            tmem_ld32(tS + c, u);
            tmem_ld_wait32(u);
            const uint32_t there = (okm >> (c / 16)) & 3u;
            if (__any_sync(0xffffffffu, last - c < 31) || there != 3u) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i > last - c || ((there >> (i / 16)) & 1u) == 0) u[i] = __float_as_uint(kNegInf);
              tmem_st32(tS + c, u);
            }
            float mx0 = __uint_as_float(u[0]), mx1 = __uint_as_float(u[1]);
#pragma unroll
            for (int i = 2; i < 30; i += 4) {
              mx0 = fmax3(mx0, __uint_as_float(u[i]), __uint_as_float(u[i + 1]));
              mx1 = fmax3(mx1, __uint_as_float(u[i + 2]), __uint_as_float(u[i + 3]));
            }
            mx = fmaxf(mx, fmax3(fmaxf(mx0, mx1), __uint_as_float(u[30]), __uint_as_float(u[31])));
          }
          tmem_st_wait();
          // m moves where a weight that is stored would pass 2^15, and for a row's first keys
          const float top = mx * f;
          if (__any_sync(0xffffffffu, live && !(l > 0.f && top - m + shift <= 15.f))) {
            if (!(shift < 1000.f)) shift = kShift;
            float m_new = fmaxf(top, top + (shift - 8.f));
            m_new = l > 0.f ? fmaxf(m, m_new) : m_new;
            if (!(m_new > kNegInf)) m_new = m;
            if (!first && !rescale(m_new, info.grow)) { ok = false; break; }
            m = m_new;
          }
          const float nm = shift - m;
          const float2 sc2 = make_float2(f, f), nm2 = make_float2(nm, nm);
          float2 la = make_float2(0.f, 0.f), lb = make_float2(0.f, 0.f);
          // weights of 16 pairs of keys and what their roundings left
          auto pairs = [&](const uint32_t (&u)[32], uint32_t (&hi)[16], uint32_t (&lo)[16]) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 arg = __ffma2_rn(
                  make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])), sc2, nm2);
              const float2 e = make_float2(ex2(arg.x), ex2(arg.y));
              if (i & 1) lb = __fadd2_rn(lb, e); else la = __fadd2_rn(la, e);
              hi[i] = pack_f16(e.x, e.y);
              if constexpr (kSplitP) {
                const float2 back = unpack_f16(hi[i]);
                lo[i] = pack_f16(e.x - back.x, e.y - back.y);
              }
            }
          };
          if constexpr (kSplitP) {
            // (the remainders' columns are those of the scores 64 and up: read first)
            uint32_t u0[32], u1[32], hi[16], lo0[16], lo1[16];
            auto load = [&](int c) {
              tmem_ld32(tS + c, u0);
              tmem_ld32(tS + c + 32, u1);
              tmem_ld_wait32(u0);
              reg_fence32(u1);
            };
            load(0);
            pairs(u0, hi, lo0);
            tmem_st16(tS, hi);
            pairs(u1, hi, lo1);
            tmem_st16(tS + 16, hi);
            load(64);
            tmem_st16(tS + 64, lo0);
            tmem_st16(tS + 80, lo1);
            pairs(u0, hi, lo0);
            tmem_st16(tS + 32, hi);
            tmem_st16(tS + 96, lo0);
            pairs(u1, hi, lo1);
            tmem_st16(tS + 48, hi);
            tmem_st16(tS + 112, lo1);
          } else {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t u[32], hi[16], lo[16];
              tmem_ld32(tS + c * 32, u);
              tmem_ld_wait32(u);
              pairs(u, hi, lo);
              tmem_st16(tS + c * 16, hi);
            }
          }
          l += ((la.x + la.y) + (lb.x + lb.y)) * ex2(-shift);
        } else {
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
            const float2 sc2 = make_float2(sl2, sl2), nm2 = make_float2(-m, -m);
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
              if (!rescale(m_new, 1.f)) { ok = false; break; }
            }
            m = m_new;
            part = weights();
          }
          l += part;
        }
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
      const float inv = l == 0.f ? 0.f : (Q8 ? unit / l : 1.f / l);
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

bool encode_pages(CUtensorMap* map, const lsx_tensor& t, bool q8) {
  const uint32_t rows = static_cast<uint32_t>(t.N < 128 ? t.N : 128);
  return q8 ? make_map_u8_4d(map, t.data, t.B, t.H, t.N, t.D, t.stride_b, t.stride_h, t.stride_n,
                             rows, t.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE)
            : encode4(map, t.data, t.D, {t.N, t.H, t.B}, t.stride_n, t.stride_h, t.stride_b, rows,
                      1, 1);
}

template <int D, bool kSplitP, bool Q8>
int launch_tiles(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                 const FwdParams& p, int64_t grid, bool early, int device, cudaStream_t s) {
  auto kern = paged_fwd_kernel<D, kSplitP, Q8>;
  constexpr size_t smem = sizeof(Smem<D, Q8>) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(kern, static_cast<int>(smem), device, done)) return LSX_ERR_LAUNCH;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(Q8 ? 512 : 384);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = early ? 1 : 0;
  timing_begin(kKidPagedFwd, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, p);
  timing_end(kKidPagedFwd, s);
  return e == cudaSuccess ? LSX_OK : LSX_ERR_LAUNCH;
}
int launch_tiles(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                 const FwdParams& p, int64_t d, bool split_p, int64_t grid, bool early, int device,
                 cudaStream_t s) {
  auto pick = [&](auto q8) {
    constexpr bool Q8 = decltype(q8)::value;
    return d == 128 ? (split_p ? launch_tiles<128, true, Q8> : launch_tiles<128, false, Q8>)
                    : (split_p ? launch_tiles<64, true, Q8> : launch_tiles<64, false, Q8>);
  };
  return (p.ks != nullptr ? pick(std::true_type{}) : pick(std::false_type{}))(tq, tk, tv, p, grid,
                                                                            early, device, s);
}
void set_exponents(FwdParams& p, const PagedCache8* c8) {
  p.ks = p.vs = nullptr;
  if (c8 == nullptr) return;
  p.ks = c8->ks; p.ks_sp = c8->ks_sp; p.ks_sh = c8->ks_sh;
  p.vs = c8->vs; p.vs_sp = c8->vs_sp; p.vs_sh = c8->vs_sh;
}

struct FwdLayout {
  int64_t max_entries, max_slots;
  size_t entries, cut, part_l, part_o, dense_table, dense_k, dense_v, total;
  int64_t dense_pages;  // of the bf16 copy, 0: none
};

// Prompts over an 8-bit cache read a bf16 copy of the pages that they see (paged_q8.cu),
// where the copy (with its table) has at most kMostDense bytes and the sequences more than
// dense_rows each for a key head, on the average; otherwise the tiles are widened where they
// are used, which keeps more bits of P.  32 query heads over 8, bf16 results, by a copy and
// in place, us:
//   rows                       1024        1280        1536        2048        4096
//   128, after 8192 keys     71   67     77   79     83   81     98  104    143  169
//   128, after 32768        169  161    194  192    196  205    261  282    435  537
//   128, after 65536        284  274    335  337    348  368    450  495    822 1023
//   128, 8 x after 8192     300  294                409  429    521  568
//   rows                        512        1024        1280        2048        4096
//   64, after 8192           44   42     56   59     63   69     81   91    118  149
//   64, after 32768          86   79    132  138    151  165    212  241    368  482
//   64, after 65536         134  130    218  239    259  290    358  431    690  926
// f32 results cross later, since the copy's second product of P costs more beside less
// else: of 128 at 1500 to 2000 rows (after 32768 keys 1024 rows 261 and 233, 2048 421 and
// 409, 4096 675 and 806), of 64 at 2000 to 4000 (2048 rows 384 and 333, 4096 652 and 689).
// The border is one for both, since workspaces are asked for without the results' type.  One
// long prompt beside 15 single tokens after 4000 keys, whose pages are copied as well:
// 210 both ways, of 64 101.
constexpr double kMostDense = 4294967296.0;
constexpr int64_t dense_rows(int64_t d) { return 8 * d; }
int64_t dense_pages(const lsx_tensor& q, const lsx_tensor& kp, int64_t batch, int64_t max_pages) {
  const int64_t pages = batch * max_pages < kp.B ? batch * max_pages : kp.B;
  const double bytes = 4.0 * (static_cast<double>(pages) * static_cast<double>(kp.N * kp.H * kp.D) +
                              static_cast<double>(batch * max_pages));
  return bytes <= kMostDense && q.N * (q.H / kp.H) > dense_rows(q.D) * batch ? pages : 0;
}
FwdLayout fwd_layout(const lsx_tensor& q, const lsx_tensor& kp, int64_t batch, int64_t max_pages,
                     bool copy, int sm_count) {
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
  x.dense_table = x.part_o + align256(rows * static_cast<size_t>(q.D) * 4);
  x.dense_pages = copy ? dense_pages(q, kp, batch, max_pages) : 0;
  const size_t dense = align256(static_cast<size_t>(x.dense_pages * kp.N * kp.H * kp.D) * 2);
  x.dense_k = x.dense_table +
              (x.dense_pages > 0 ? align256(static_cast<size_t>(batch * max_pages) * 4) : 0);
  x.dense_v = x.dense_k + dense;
  x.total = x.dense_v + dense;
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
                  const PagedCache& prefix, const PagedCache8* c8, int64_t prefix_len,
                  const PrefixPlan& plan,
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
  set_exponents(p, c8);
  CUtensorMap tq, tk, tv;
  if (!encode4(&tq, q.data, q.D, {q.H, q.N, q.B}, q.stride_h, q.stride_n, q.stride_b,
               static_cast<uint32_t>(p.G), static_cast<uint32_t>(q.N),
               static_cast<uint32_t>(p.tpt)) ||
      !encode_pages(&tk, k_pages, c8 != nullptr) || !encode_pages(&tv, v_pages, c8 != nullptr))
    return LSX_ERR_LAUNCH;
  const int64_t items = plan.rows / 256;
  const int64_t grid = items < ctx.sm_count ? items : ctx.sm_count;
  return launch_tiles(tq, tk, tv, p, q.D, split_p, grid, false, ctx.device, s);
}

size_t paged_fwd_workspace(const lsx_tensor& q, const lsx_tensor& k_pages, int64_t batch,
                           int64_t max_pages, bool copy, int sm_count) {
  return fwd_layout(q, k_pages, batch, max_pages, copy, sm_count).total;
}

int launch_paged_fwd(const lsx_tensor& q, const lsx_tensor& pages_k, const lsx_tensor& pages_v,
                     const PagedCache& c, const PagedCache8* c8, const int32_t* kv_lens,
                     const int32_t* cu_q, int64_t batch, float scale, const lsx_tensor& o,
                     const lsx_tensor& lse, void* workspace, size_t workspace_bytes,
                     const DeviceCtx& ctx, cudaStream_t s) {
  const bool split_p = c8 != nullptr && o.dtype == LSX_F32;
  FwdLayout x = fwd_layout(q, pages_k, batch, c.max_pages, c8 != nullptr, ctx.sm_count);
  if (workspace_bytes < x.total)  // no room for the copy: the caller goes without
    x = fwd_layout(q, pages_k, batch, c.max_pages, false, ctx.sm_count);
  char* ws = static_cast<char*>(workspace);
  FwdParams p;
  p.c = c;
  lsx_tensor k_pages = pages_k, v_pages = pages_v;
  const PagedCache8* const source = x.dense_pages > 0 ? c8 : nullptr;
  if (source != nullptr) {  // the copy, a head's rows of a page together, in the place of the cache
    for (lsx_tensor* t : {&k_pages, &v_pages}) {
      t->dtype = LSX_BF16;
      t->B = x.dense_pages;
      t->stride_n = t->D;
      t->stride_h = t->N * t->D;
      t->stride_b = t->H * t->stride_h;
    }
    k_pages.data = ws + x.dense_k;
    v_pages.data = ws + x.dense_v;
    p.c = paged_cache(k_pages, v_pages, reinterpret_cast<const int32_t*>(ws + x.dense_table),
                      c.max_pages, c.max_pages);
    c8 = nullptr;
  }
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
  set_exponents(p, c8);
  CUtensorMap tq, tk, tv;
  if (!encode4(&tq, q.data, q.D, {q.H, q.N, 1}, q.stride_h, q.stride_n, 0,
               static_cast<uint32_t>(p.G), static_cast<uint32_t>(p.tpt), 1) ||
      !encode_pages(&tk, k_pages, c8 != nullptr) || !encode_pages(&tv, v_pages, c8 != nullptr))
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
  if (source != nullptr) {
    const int widened = launch_page_widen(*source, kv_lens, cu_q, batch, q.N, k_pages, v_pages,
                                          reinterpret_cast<int32_t*>(ws + x.dense_table), ctx, s);
    if (widened != LSX_OK) return widened;
  }
  const int64_t most = x.max_entries * p.Hkv;
  const int64_t grid = most < ctx.sm_count ? most : ctx.sm_count;
  const int rc = launch_tiles(tq, tk, tv, p, q.D, split_p, grid, true, ctx.device, s);
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
