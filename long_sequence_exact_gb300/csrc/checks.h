// checks.h -- argument checks shared by the entry points (host code).  Each
// returns LSX_OK or the LSX_ERR_* code of the first rule that is broken.
#pragma once

#include <math.h>
#include <stdint.h>

#include "internal.h"

namespace lsx {
namespace {

// ---------------------------------------------------------- validation
int check_view(const lsx_tensor* t) {
  if (t == nullptr) return LSX_ERR_NULL;
  if (t->data == nullptr && t->N != 0) return LSX_ERR_NULL;  // empty views may be NULL
  if (t->dtype != LSX_BF16 && t->dtype != LSX_F32) return LSX_ERR_DTYPE;
  if (t->B <= 0 || t->H <= 0 || t->N < 0 || t->D <= 0) return LSX_ERR_SHAPE;
  if (t->stride_b < 0 || t->stride_h < 0 || t->stride_n < 0) return LSX_ERR_SHAPE;
  if (reinterpret_cast<uintptr_t>(t->data) % 16 != 0) return LSX_ERR_ALIGN;
  return LSX_OK;
}

int elem_size(int dtype) { return dtype == LSX_F32 ? 4 : 2; }

// A row of D elements is read/written with 16-byte vectors (or 8-byte for
// bf16 rows of 64/128 in the merge kernels): rows must start 16-B aligned.
int check_row_aligned(const lsx_tensor* t) {
  const int64_t vec = 16 / elem_size(t->dtype);
  if (t->stride_n % vec || t->stride_h % vec || t->stride_b % vec) return LSX_ERR_ALIGN;
  return LSX_OK;
}

int check_lse(const lsx_tensor* l, const lsx_tensor* like) {
  if (l == nullptr || l->data == nullptr) return LSX_ERR_NULL;
  if (l->dtype != LSX_F32) return LSX_ERR_DTYPE;
  if (l->D != 1 || l->B != like->B || l->H != like->H || l->N != like->N) return LSX_ERR_SHAPE;
  if (reinterpret_cast<uintptr_t>(l->data) % 4 != 0) return LSX_ERR_ALIGN;
  if (l->stride_b < 0 || l->stride_h < 0 || l->stride_n < 0) return LSX_ERR_SHAPE;
  return LSX_OK;
}

bool same_bhn_d(const lsx_tensor* a, const lsx_tensor* b) {
  return a->B == b->B && a->H == b->H && a->N == b->N && a->D == b->D;
}

#define LSX_TRY(expr)          \
  do {                         \
    const int _rc = (expr);    \
    if (_rc != LSX_OK) return _rc; \
  } while (0)

// q [B,Hq,Lq,D], k/v [B,Hkv,Lk,D], same dtype, D in {64,128}, Hq % Hkv == 0.
int check_qkv(const lsx_tensor* q, const lsx_tensor* k, const lsx_tensor* v) {
  LSX_TRY(check_view(q));
  LSX_TRY(check_view(k));
  LSX_TRY(check_view(v));
  if (k->dtype != q->dtype || v->dtype != q->dtype) return LSX_ERR_DTYPE;
  if (k->B != q->B || v->B != q->B || k->D != q->D || v->D != q->D ||
      v->H != k->H || v->N != k->N)
    return LSX_ERR_SHAPE;
  if (q->H % k->H != 0) return LSX_ERR_SHAPE;
  if (q->D != 64 && q->D != 128) return LSX_ERR_UNSUPPORTED;
  LSX_TRY(check_row_aligned(q));
  LSX_TRY(check_row_aligned(k));
  LSX_TRY(check_row_aligned(v));
  // TMA: every coordinate must fit a 32-bit signed integer
  const int64_t lim = int64_t(1) << 31;
  if (q->N >= lim || k->N >= lim || q->H >= lim || q->B >= lim) return LSX_ERR_UNSUPPORTED;
  return LSX_OK;
}

float resolve_scale(float scale, int64_t d) {
  return scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(d));
}

cudaStream_t as_stream(lsx_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace
}  // namespace lsx
