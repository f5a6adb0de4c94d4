// Checks of the 8-bit cache's arguments, shared by its entry points.
#pragma once

#include <stdint.h>

#include "../../include/gemv.h"
#include "gemv_internal.h"
#include "gemv_kv8.cuh"

namespace gemv {

inline bool mul_ok(int64_t a, int64_t b, int64_t *out) { return !__builtin_mul_overflow(a, b, out); }
inline bool aligned(const void *p, int bytes) { return ((uintptr_t)p % (uintptr_t)bytes) == 0; }

constexpr int kKvMaxWidth = 1 << 24;  // blocks of a sequence: positions stay below 2^30

// The cache's own checks: sizes, pointers, alignment (a block is copied in 16-byte
// pieces).  On success *bytes is the size of the keys (and of the values).
inline gemv_status_t check_cache(const gemv_kv8_cache_t *c, int64_t *bytes) {
  if (c == nullptr || c->blocks < 0 || c->heads < 0 || c->dim < 0 || c->width < 0) return GEMV_ERR_INVALID_VALUE;
  if (c->dim != 64 && c->dim != 128 && c->dim != 192 && c->dim != 256) return GEMV_ERR_UNSUPPORTED;
  // grid dimensions and block numbers
  if (c->heads > 65535 || c->blocks > 0x7fffffff || c->width > kKvMaxWidth) return GEMV_ERR_INVALID_VALUE;
  if (!mul_ok(c->blocks * (int64_t)c->heads, kKvBlock * c->dim, bytes)) return GEMV_ERR_INVALID_VALUE;
  return GEMV_SUCCESS;
}
inline bool cache_pointers(const gemv_kv8_cache_t *c) {
  return c->blocks > 0 && c->k != nullptr && c->v != nullptr && c->k_scale != nullptr && c->v_scale != nullptr &&
         aligned(c->k, 16) && aligned(c->v, 16) && aligned(c->k_scale, 4) && aligned(c->v_scale, 4) && aligned(c->table, 4) &&
         (c->table != nullptr || c->width == 0);
}
// Bytes from the first to the last of `rows` rows of `row` elements, `stride` apart.
inline bool span(int64_t rows, int64_t row, int64_t stride, int size, int64_t *out) {
  int64_t n;
  return mul_ok(rows - 1, stride, &n) && !__builtin_add_overflow(n, row, &n) && mul_ok(n, size, out);
}

// Two sets of rows of `row` elements are different columns of the same matrix.
inline bool columns(const void *p, int64_t p_stride, const void *q, int64_t q_stride, int64_t row, int size) {
  if (p == nullptr || q == nullptr || p_stride != q_stride) return false;
  const int64_t stride = p_stride * size, bytes = row * size;
  int64_t d = (int64_t)((uintptr_t)q - (uintptr_t)p) % stride;
  if (d < 0) d += stride;
  return d >= bytes && stride - d >= bytes;
}

inline KvArgs cache_args(const gemv_kv8_cache_t *c) {
  KvArgs a;
  a.k = c->k;
  a.v = c->v;
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.table = c->table;
  a.blocks = c->blocks;
  a.heads = c->heads;
  a.width = (int)c->width;
  return a;
}

}  // namespace gemv
