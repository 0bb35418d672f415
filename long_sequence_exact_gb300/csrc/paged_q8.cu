// paged_q8.cu -- caches in pages of 8 bits: new rows quantised into their slots,
// and rows of ranges of positions read back.
//
// A row x (a token's key or value of one head) is held as e4m3 values q and one
// exponent e, x ~ q 2^e: e is the smallest integer with max |x| <= 448 2^e, kept
// within [-100, 7], and q = x 2^-e rounded to the nearest e4m3 (ties to even,
// saturating).  e4m3 has the same relative step in every binade, so a scale that
// is not a power of two would gain nothing; with this one x 2^-e is exact, and
// q 2^e has 4 significant bits and an exponent from -109 to 15: a bf16 exactly.
// Reading back rounds nothing, and attention over the cache is attention over
// the bf16 rows that it stands for.
#include <cuda_bf16.h>

#include "paged.h"
#include "ptx.cuh"
#include "q8.cuh"

namespace lsx {
namespace {

constexpr int kAppendCtas = 64;  // per SM, at most

struct AppendQ8Params {
  const void* k;
  const void* v;
  int64_t k_sh, k_sn, v_sh, v_sn;
  uint8_t* kp;
  uint8_t* vp;
  int64_t kp_sp, kp_sh, kp_sn, vp_sp, vp_sh, vp_sn;
  uint8_t* ks;
  uint8_t* vs;
  int64_t ks_sp, ks_sh, vs_sp, vs_sh;
  const int64_t* slots;
  int64_t n_tokens, n_slots;
  int heads, d8, shift;
  int* status;
};

// kWide: rows are 32-byte aligned.
template <bool kF32, bool kWide>
__device__ __forceinline__ void load8(const void* base, int64_t off, float (&x)[8]) {
  if constexpr (kF32 && kWide) {
    uint32_t w[8];
    ld_global32(static_cast<const float*>(base) + off, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  } else if constexpr (kF32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
    const float4 a = __ldcs(p), b = __ldcs(p + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + off));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// Largest |x| of the row whose pieces are in `lanes` neighbouring lanes (NaN
// counts as nothing: it stays a NaN of its own and leaves its row's others alone).
__device__ __forceinline__ float row_max(const float (&x)[8], int lanes) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
  for (int s = lanes >> 1; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
  return m;
}

__device__ __forceinline__ uint2 quantise8(const float (&x)[8], int e) {
  const float f = q8_power(-e);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = pack_e4m3(x[4 * i] * f, x[4 * i + 1] * f) |
           pack_e4m3(x[4 * i + 2] * f, x[4 * i + 3] * f) << 16;
  return make_uint2(w[0], w[1]);
}

// One thread per eight elements of a token's key and value, a row in 8 or 16
// neighbouring lanes, which share its maximum.  Bound: HBM; one pass, 32 bytes of f32 a
// load (16: 82 us instead of 76).  50021 tokens of 8 heads of 128, f32: 73.5 us for 0.40
// GB read and 0.10 written, DRAM at 82% of its peak; one step of 48 tokens 7 us, the
// launch and one trip to memory.
template <bool kF32, bool kWide, typename Index>
__global__ void __launch_bounds__(256) page_append_q8_kernel(const AppendQ8Params p) {
  const Index per = static_cast<Index>(p.heads * p.d8);
  const Index n = static_cast<Index>(p.n_tokens) * per;
  const Index step = static_cast<Index>(gridDim.x) * 256;
  // (whole warps go round together: a row's lanes stay together)
  for (Index i = static_cast<Index>(blockIdx.x) * 256 + threadIdx.x; i - (threadIdx.x & 31) < n;
       i += step) {
    const Index at = i < n ? i : n - 1;
    const Index tok = at / per;
    const int r = static_cast<int>(at - tok * per);
    const int h = r / p.d8, piece = r - h * p.d8, e = piece * 8;
    int64_t slot = i < n ? __ldg(p.slots + tok) : -1;
    if (slot >= p.n_slots) {
      atomicCAS(p.status, 0, kStatusPage);
      slot = -1;
    }
    float k[8] = {}, v[8] = {};
    if (slot >= 0) {
      load8<kF32, kWide>(p.k, h * p.k_sh + tok * p.k_sn + e, k);
      load8<kF32, kWide>(p.v, h * p.v_sh + tok * p.v_sn + e, v);
    }
    const int ek = q8_exponent(row_max(k, p.d8)), ev = q8_exponent(row_max(v, p.d8));
    if (slot < 0) continue;
    const int64_t page = slot >> p.shift, row = slot & ((1 << p.shift) - 1);
    *reinterpret_cast<uint2*>(p.kp + page * p.kp_sp + h * p.kp_sh + row * p.kp_sn + e) =
        quantise8(k, ek);
    *reinterpret_cast<uint2*>(p.vp + page * p.vp_sp + h * p.vp_sh + row * p.vp_sn + e) =
        quantise8(v, ev);
    if (piece == 0) {
      p.ks[page * p.ks_sp + h * p.ks_sh + row] = static_cast<uint8_t>(ek + 127);
      p.vs[page * p.vs_sp + h * p.vs_sh + row] = static_cast<uint8_t>(ev + 127);
    }
  }
}

// ------------------------------------------------------------------- read
constexpr int kReadTokens = 8;  // of a block

struct ReadQ8Params {
  PagedCache8 c;
  const int32_t* first;
  const int32_t* cu;
  int batch;
  int64_t n_tokens;
  int heads, d;
  void* k;
  void* v;
  int64_t k_sh, k_sn, v_sh, v_sn;
  int* status;
};

// Eight values of one word pair as floats times f, or as bf16.
template <bool kF32, bool kWide>
__device__ __forceinline__ void store_values(void* base, int64_t off, const uint32_t* w, float f) {
  constexpr int kWords = kF32 ? 2 : 4;  // 32 bytes of output
  uint32_t out[8];
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    uint32_t lo, hi;
    e4m3_f16x4(w[i], lo, hi);
    const float2 a = unpack_f16(lo), b = unpack_f16(hi);
    if constexpr (kF32) {
      out[4 * i] = __float_as_uint(a.x * f);
      out[4 * i + 1] = __float_as_uint(a.y * f);
      out[4 * i + 2] = __float_as_uint(b.x * f);
      out[4 * i + 3] = __float_as_uint(b.y * f);
    } else {
      out[2 * i] = pack_bf16(a.x * f, a.y * f);
      out[2 * i + 1] = pack_bf16(b.x * f, b.y * f);
    }
  }
  uint4* dst = reinterpret_cast<uint4*>(static_cast<char*>(base) + off * (kF32 ? 4 : 2));
  if constexpr (kWide) {
    st_global32(dst, out);
  } else {
    dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
    dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
  }
}

// A block takes kReadTokens packed tokens: a thread each finds the sequence and the row,
// then the threads stream the rows, 32 bytes of output a piece (16: 205 us instead of
// 165).  Bound: HBM, three quarters of it writes: blocks write neighbouring rows in turn (a
// grid that fits the device and goes round, each block's rows far apart: 167 us).  37
// sequences' ranges of up to 9001 positions, 8 heads of 64, to f32: 146 us for 0.22 GB read
// and 0.71 written, 6.4 TB/s.
template <bool kF32, bool kWide>
__global__ void __launch_bounds__(256) page_read_q8_kernel(const ReadQ8Params p) {
  constexpr int kElems = kF32 ? 8 : 16;
  __shared__ int64_t slot[kReadTokens];  // page << shift | row; -1 zeros, -2 no token
  const int per_row = p.d / kElems, per = p.heads * per_row;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kReadTokens;
  if (threadIdx.x < kReadTokens) {
    const int64_t t = t0 + threadIdx.x;
    int64_t at = -2;
    if (t < p.n_tokens) {
      int lo = 0, hi = p.batch;  // the last sequence that begins at or before t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.cu + mid) <= t) lo = mid; else hi = mid;
      }
      const int64_t c0 = __ldg(p.cu + lo);
      if (t >= c0 && t < __ldg(p.cu + lo + 1)) {
        const int64_t f = __ldg(p.first + lo), pos = (f < 0 ? 0 : f) + (t - c0);
        const int64_t col = pos >> p.c.shift;
        int32_t page = -1;
        if (col < p.c.max_pages) page = __ldg(p.c.table + lo * p.c.table_stride + col);
        if (page < 0 || page >= p.c.n_pages) {
          atomicCAS(p.status, 0, kStatusPage);
          at = -1;
        } else {
          at = (static_cast<int64_t>(page) << p.c.shift) | (pos & ((1 << p.c.shift) - 1));
        }
      }
    }
    slot[threadIdx.x] = at;
  }
  __syncthreads();
#pragma unroll 2
  for (int i = threadIdx.x; i < kReadTokens * per; i += 256) {
    const int tok = i / per, r = i - tok * per, h = r / per_row, e = (r - h * per_row) * kElems;
    const int64_t at = slot[tok];
    if (at == -2) continue;
    uint32_t kw[4] = {}, vw[4] = {};
    float kf = 0.f, vf = 0.f;
    if (at >= 0) {
      const int64_t page = at >> p.c.shift, row = at & ((1 << p.c.shift) - 1);
      const uint8_t* ks = p.c.k + page * p.c.k_sp + h * p.c.k_sh + row * p.c.k_sn + e;
      const uint8_t* vs = p.c.v + page * p.c.v_sp + h * p.c.v_sh + row * p.c.v_sn + e;
      if constexpr (kF32) {
        const uint2 a = __ldcs(reinterpret_cast<const uint2*>(ks));
        const uint2 b = __ldcs(reinterpret_cast<const uint2*>(vs));
        kw[0] = a.x; kw[1] = a.y; vw[0] = b.x; vw[1] = b.y;
      } else {
        const uint4 a = __ldcs(reinterpret_cast<const uint4*>(ks));
        const uint4 b = __ldcs(reinterpret_cast<const uint4*>(vs));
        kw[0] = a.x; kw[1] = a.y; kw[2] = a.z; kw[3] = a.w;
        vw[0] = b.x; vw[1] = b.y; vw[2] = b.z; vw[3] = b.w;
      }
      kf = q8_scale(__ldg(p.c.ks + page * p.c.ks_sp + h * p.c.ks_sh + row));
      vf = q8_scale(__ldg(p.c.vs + page * p.c.vs_sp + h * p.c.vs_sh + row));
    }
    store_values<kF32, kWide>(p.k, h * p.k_sh + (t0 + tok) * p.k_sn + e, kw, kf);
    store_values<kF32, kWide>(p.v, h * p.v_sh + (t0 + tok) * p.v_sn + e, vw, vf);
  }
}

// ------------------------------------------------------------------ widen
// A bf16 copy of the pages that a call's prompts see, for many query rows a key: the
// prompt kernel then reads tiles that its products take as they are.  Every block sums the
// sequences' pages for itself and takes pieces of pages in turn (a whole page: a tenth
// more, 298 us instead of 288 for 256 tokens after 65536 keys, 32 query heads over 8 of
// 128).  Bound: HBM (what it writes is read again at once, from L2 as far as it holds it).
// These 65,792 keys: 65 us for 0.14 GB read and 0.27 written (0.21 of them to DRAM),
// 5.3 TB/s of DRAM.
constexpr int kWidenCtas = 4;      // on an SM at once
constexpr int kWidenPieces = 512;  // 16-byte pieces of keys (and of values) in a block's turn
struct WidenParams {
  PagedCache8 c;
  const int32_t* kv_lens;
  const int32_t* cu_q;
  int batch;
  int64_t n_tokens;
  int heads, log_pieces, page_pieces;  // 16-byte pieces of a row (log2), of a head's page
  bool own;                            // pages numbered by sequence and column
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  int32_t* table;
};

// Pages of sequence b that its tokens see: none without tokens.
__device__ __forceinline__ int32_t seen_pages(const WidenParams& p, int b) {
  int64_t q0 = p.cu_q[b], q1 = p.cu_q[b + 1];
  q0 = q0 < 0 ? 0 : q0;
  q1 = q1 > p.n_tokens ? p.n_tokens : q1;
  const int64_t cap = static_cast<int64_t>(p.c.max_pages) << p.c.shift, n = p.kv_lens[b];
  if (q1 <= q0 || n <= 0) return 0;
  return static_cast<int32_t>(((n < cap ? n : cap) + (1 << p.c.shift) - 1) >> p.c.shift);
}

__global__ void __launch_bounds__(256, kWidenCtas) page_widen_kernel(const WidenParams p) {
  extern __shared__ int64_t first[];  // [batch + 1] pages before each sequence's
  __shared__ int64_t sums[8];
  const int t = threadIdx.x;
  const int per = (p.batch + 255) / 256;
  const int b0 = t * per < p.batch ? t * per : p.batch;
  const int b1 = b0 + per < p.batch ? b0 + per : p.batch;
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += seen_pages(p, b);
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
  for (int w = 0; w < 8; ++w) {
    if (w < (t >> 5)) before += sums[w];
    total += sums[w];
  }
  for (int b = b0; b < b1; ++b) {
    first[b] = before;
    before += seen_pages(p, b);
  }
  __syncthreads();
  // a turn: kWidenPieces pieces of a page; the next one's page is looked up early
  const int pieces = p.heads * p.page_pieces, turns = (pieces + kWidenPieces - 1) / kWidenPieces;
  int64_t i = blockIdx.x, at = 0;
  int32_t page = -1;
  auto find = [&]() {
    if (i >= total * turns) return;
    const int64_t n = i / turns;
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= n) lo = mid; else hi = mid;
    }
    const int64_t col = n - first[lo];
    page = __ldg(p.c.table + lo * p.c.table_stride + col);
    at = static_cast<int64_t>(lo) * p.c.max_pages + col;
  };
  find();
  while (i < total * turns) {
    const bool is = page >= 0 && page < p.c.n_pages;
    const int64_t from = page, to = p.own ? at : from;
    const int x0 = static_cast<int>(i % turns) * kWidenPieces + t;
    if (x0 == 0) p.table[at] = is ? static_cast<int32_t>(to) : -1;
    constexpr int kN = kWidenPieces / 256;
    uint4 a[kN], b[kN];
    float kf[kN], vf[kN];
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int x = x0 + n * 256;
      if (!is || x >= pieces) continue;
      const int h = x / p.page_pieces, y = x - h * p.page_pieces;
      const int row = y >> p.log_pieces, e = (y - (row << p.log_pieces)) * 16;
      a[n] = __ldcs(reinterpret_cast<const uint4*>(
          p.c.k + from * p.c.k_sp + h * p.c.k_sh + row * p.c.k_sn + e));
      b[n] = __ldcs(reinterpret_cast<const uint4*>(
          p.c.v + from * p.c.v_sp + h * p.c.v_sh + row * p.c.v_sn + e));
      kf[n] = q8_scale(__ldg(p.c.ks + from * p.c.ks_sp + h * p.c.ks_sh + row));
      vf[n] = q8_scale(__ldg(p.c.vs + from * p.c.vs_sp + h * p.c.vs_sh + row));
    }
    i += gridDim.x;
    find();
    const int64_t out = to * pieces * 16;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int x = x0 + n * 256;
      if (!is || x >= pieces) continue;
      const uint32_t kw[4] = {a[n].x, a[n].y, a[n].z, a[n].w};
      const uint32_t vw[4] = {b[n].x, b[n].y, b[n].z, b[n].w};
      store_values<false, true>(p.k, out + static_cast<int64_t>(x) * 16, kw, kf[n]);
      store_values<false, true>(p.v, out + static_cast<int64_t>(x) * 16, vw, vf[n]);
    }
  }
  // (the plan before, whose launch this one did not wait for, has ended when this one has)
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace

int launch_page_widen(const PagedCache8& c, const int32_t* kv_lens, const int32_t* cu_q,
                      int64_t batch, int64_t n_tokens, const lsx_tensor& k, const lsx_tensor& v,
                      int32_t* table, const DeviceCtx& ctx, cudaStream_t s) {
  WidenParams p;
  p.c = c;
  p.kv_lens = kv_lens;
  p.cu_q = cu_q;
  p.batch = static_cast<int>(batch);
  p.n_tokens = n_tokens;
  p.heads = static_cast<int>(k.H);
  p.log_pieces = k.D == 128 ? 3 : 2;
  p.page_pieces = static_cast<int>(k.N) << p.log_pieces;
  p.own = batch * c.max_pages <= k.B;
  p.k = static_cast<__nv_bfloat16*>(k.data);
  p.v = static_cast<__nv_bfloat16*>(v.data);
  p.table = table;
  const int64_t most = 4 * kWidenCtas * static_cast<int64_t>(ctx.sm_count);
  const int64_t turns = batch * c.max_pages * ceil_div(p.heads * p.page_pieces, kWidenPieces);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(turns < 1 ? 1 : (turns < most ? turns : most)));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = static_cast<size_t>(batch + 1) * sizeof(int64_t);
  cfg.stream = s;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  timing_begin(kKidPageWiden, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, page_widen_kernel, p);
  timing_end(kKidPageWiden, s);
  return e == cudaSuccess ? LSX_OK : LSX_ERR_LAUNCH;
}

namespace {
// Whether every row starts on a sector of 32 bytes.
bool sectors(const lsx_tensor& t) {
  const int64_t size = t.dtype == LSX_F32 ? 4 : 2;
  return reinterpret_cast<uintptr_t>(t.data) % 32 == 0 && t.stride_h * size % 32 == 0 &&
         t.stride_n * size % 32 == 0;
}
}  // namespace

int launch_page_append_q8(const lsx_tensor& k, const lsx_tensor& v, const int64_t* slot_map,
                          const Pages8& pages, const DeviceCtx& ctx, cudaStream_t s) {
  AppendQ8Params p;
  p.k = k.data; p.v = v.data;
  p.k_sh = k.stride_h; p.k_sn = k.stride_n;
  p.v_sh = v.stride_h; p.v_sn = v.stride_n;
  const lsx_tensor &kp = *pages.k, &vp = *pages.v, &ks = *pages.ks, &vs = *pages.vs;
  p.kp = static_cast<uint8_t*>(kp.data);
  p.vp = static_cast<uint8_t*>(vp.data);
  p.kp_sp = kp.stride_b; p.kp_sh = kp.stride_h; p.kp_sn = kp.stride_n;
  p.vp_sp = vp.stride_b; p.vp_sh = vp.stride_h; p.vp_sn = vp.stride_n;
  p.ks = static_cast<uint8_t*>(ks.data);
  p.vs = static_cast<uint8_t*>(vs.data);
  p.ks_sp = ks.stride_b; p.ks_sh = ks.stride_h;
  p.vs_sp = vs.stride_b; p.vs_sh = vs.stride_h;
  p.slots = slot_map;
  p.n_tokens = k.N;
  p.n_slots = kp.B * kp.N;
  p.heads = static_cast<int>(k.H);
  p.d8 = static_cast<int>(k.D / 8);
  p.shift = 0;
  while ((int64_t{1} << p.shift) < kp.N) ++p.shift;
  p.status = ctx.status;
  const int64_t pieces = k.N * k.H * p.d8;
  int64_t grid = ceil_div(pieces, 256);
  const int64_t most = kAppendCtas * static_cast<int64_t>(ctx.sm_count);
  if (grid > most) grid = most;
  const bool small = pieces < (int64_t{1} << 31);  // (unsigned: a grid more fits too)
  timing_begin(kKidPageAppend, s);
  auto pick = [&](auto index) {
    using Index = decltype(index);
    return k.dtype != LSX_F32              ? page_append_q8_kernel<false, false, Index>
           : sectors(k) && sectors(v) ? page_append_q8_kernel<true, true, Index>
                                      : page_append_q8_kernel<true, false, Index>;
  };
  auto kern = small ? pick(uint32_t{}) : pick(int64_t{});
  kern<<<static_cast<unsigned>(grid), 256, 0, s>>>(p);
  timing_end(kKidPageAppend, s);
  return cudaGetLastError() == cudaSuccess ? LSX_OK : LSX_ERR_LAUNCH;
}

int launch_page_read_q8(const PagedCache8& c, const int32_t* first, const int32_t* cu,
                        int64_t batch, const lsx_tensor& k, const lsx_tensor& v,
                        const DeviceCtx& ctx, cudaStream_t s) {
  const ReadQ8Params p{c, first, cu, static_cast<int>(batch), k.N, static_cast<int>(k.H),
                       static_cast<int>(k.D), k.data, v.data, k.stride_h, k.stride_n, v.stride_h,
                       v.stride_n, ctx.status};
  const int64_t grid = ceil_div(k.N, kReadTokens);
  timing_begin(kKidPageRead, s);
  const bool wide = sectors(k) && sectors(v);
  auto kern = k.dtype == LSX_F32
                  ? (wide ? page_read_q8_kernel<true, true> : page_read_q8_kernel<true, false>)
                  : (wide ? page_read_q8_kernel<false, true> : page_read_q8_kernel<false, false>);
  kern<<<static_cast<unsigned>(grid), 256, 0, s>>>(p);
  timing_end(kKidPageRead, s);
  return cudaGetLastError() == cudaSuccess ? LSX_OK : LSX_ERR_LAUNCH;
}

}  // namespace lsx
