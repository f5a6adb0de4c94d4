// gemv_kv8_append, gemv_kv8_read and gemv_kv8_attention: argument checks, the choice of the form,
// launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gemv.h"
#include "gemv_internal.h"
#include "gemv_kv8.cuh"
#include "gemv_kv8_host.h"
#include "gemv_launch.cuh"

namespace gemv {
namespace {

// Blocks that the rows can reach, at most: CTAs along x.
int64_t reached(const KvArgs &a) {
  return a.starts == nullptr ? (int64_t)a.S * ((a.T + kKvBlock - 2) / kKvBlock + 1) : a.N / kKvBlock + 2 * (int64_t)a.S;
}

template <int D>
cudaError_t append(KvArgs a, int sms, cudaStream_t s) {
  const int64_t x = reached(a);
  if (x > 0x7fffffff) return cudaErrorInvalidConfiguration;
  // one unit for each CTA while the SMs hold all of them (four CTAs each), else two, so that
  // finding the block is paid once for both (us with one / two / four, 5 ragged prompts of
  // 10 k tokens in all 22.6 / 21.1 / 23.4, one of 8192 14.7 / 14.4 / 16.7)
  const int64_t units = 2 * (int64_t)a.heads;
  a.per_cta = x * units > (int64_t)sms * 4 ? 2 : 1;
  auto kern = a.dtype == GEMV_DTYPE_F32 ? k_kv8_append<D, GEMV_DTYPE_F32> : a.dtype == GEMV_DTYPE_F16 ? k_kv8_append<D, GEMV_DTYPE_F16>
                                                                         : k_kv8_append<D, GEMV_DTYPE_BF16>;
  return launch_k(kern, dim3((unsigned)x, (unsigned)((units + a.per_cta - 1) / a.per_cta)), dim3(kKvAppendThreads), 0, s,
                  launch_overlap(), a);
}

template <int D>
cudaError_t read_back(const KvArgs &a, cudaStream_t s) {
  const int64_t x = reached(a), parts = (int64_t)a.sides * a.heads * (D / 64), y = (parts + kKvReadThreads / 32 - 1) / (kKvReadThreads / 32);
  if (x > 0x7fffffff) return cudaErrorInvalidConfiguration;
  auto kern = a.dtype == GEMV_DTYPE_F32 ? k_kv8_read<D, GEMV_DTYPE_F32> : a.dtype == GEMV_DTYPE_F16 ? k_kv8_read<D, GEMV_DTYPE_F16>
                                                                         : k_kv8_read<D, GEMV_DTYPE_BF16>;
  return launch_k(kern, dim3((unsigned)x, (unsigned)(y < 65535 ? y : 65535)), dim3(kKvReadThreads), 0, s, launch_overlap(), a);
}

// Tables of at most so many blocks per sequence: every item is one warp's, whole, in one
// launch that needs no scratch buffer.  (us a call on the GPU, whole / shared and joined,
// 8 heads of 128 channels: 128 tokens 6.7 / 8.2 for one sequence, 7.3 / 11.4 for 64; 256
// tokens 9.8 / 8.3 and 10.8 / 11.9, where the host's time, 11 / 14, decides; 512 tokens
// 16 / 8.7.)
constexpr int kKvWhole = 4;

template <int D, int NT>
gemv_status_t attend(KvArgs a, int sms, cudaStream_t s) {
  using F = KvForm<D, NT>;
  a.row_tiles = (a.T * a.group + NT * 8 - 1) / (NT * 8);
  if ((int64_t)a.heads * a.row_tiles > 65535) return GEMV_ERR_UNSUPPORTED;
  const int items = a.heads * a.row_tiles;
  const int pdl = launch_overlap();
  if (a.width <= kKvWhole) {
    cudaError_t e = allow_smem_once<k_kv8_attention<D, NT, true>>(F::kSmem);
    if (e == cudaSuccess)
      e = launch_k(k_kv8_attention<D, NT, true>, dim3((unsigned)sms), dim3(F::kThreads), (size_t)F::kSmem, s, pdl, a);
    if (e != cudaSuccess) return fail((int)e);
    count_launches(1);
    return GEMV_SUCCESS;
  }
  a.workers = sms * F::kWarps;  // one CTA per SM
  const int64_t parts = (int64_t)a.workers * 2 * kv_part<D, NT>() * 4;
  void *ws = nullptr;
  cudaError_t e = workspace(&ws, (size_t)(parts + (int64_t)a.S * items * 16), s);
  if (e != cudaSuccess) return fail((int)e);
  a.ws = static_cast<float *>(ws);
  a.parts = reinterpret_cast<int4 *>(static_cast<char *>(ws) + parts);
  e = allow_smem_once<k_kv8_attention<D, NT, false>>(F::kSmem);
  if (e == cudaSuccess)
    e = launch_k(k_kv8_attention<D, NT, false>, dim3((unsigned)sms), dim3(F::kThreads), (size_t)F::kSmem, s, pdl, a);
  if (e == cudaSuccess) {
    const int rows = a.T * a.group < NT * 8 ? a.T * a.group : NT * 8;
    auto join = [&](auto kern, int along) {
      return launch_k(kern, dim3((unsigned)a.S, (unsigned)items, (unsigned)((rows * D / 4 + along - 1) / along)),
                      dim3(kKvJoinThreads), 0, s, pdl, a);
    };
    // Threads for the parts of the same channels: as many as two CTAs for each SM allow (us,
    // 16 sequences of 1000 tokens, eight / four, 512 / 256 CTAs: 12.2 / 10.9; 32 of 2000,
    // four / one, 512 / 128 CTAs: 21.4 / 20.0; 12 of a window of 4096, 24 rows, four / one,
    // 288 / 72 CTAs: 20.2 / 22.8; 8 of 2000, eight / one 10.5 / 12.2), and 32 where an item can be
    // in so many parts that eight would take two turns at them (32 / eight: one key head, 16
    // queries of 192 channels, 30000 tokens 18.5 / 22.9; 8 key heads, 8000 tokens 9.9 /
    // 10.9, 1000 tokens, 16 parts, 9.6 / 9.3).
    const int64_t threads = (int64_t)a.S * items * rows * (D / 4), most = (int64_t)sms * 2 * kKvJoinThreads / threads;
    const int64_t spread = (int64_t)sms * F::kWarps / ((int64_t)a.S * items), in_parts = a.width < spread ? a.width : spread;
    if (most >= 32 && in_parts > 64)
      e = join(k_kv8_join<D, NT, 32>, kKvJoinThreads / 32);
    else if (most >= 8)
      e = join(k_kv8_join<D, NT, 8>, kKvJoinThreads / 8);
    else if (most >= 4)
      e = join(k_kv8_join<D, NT, 4>, kKvJoinThreads / 4);
    else
      e = join(k_kv8_join<D, NT, 1>, kKvJoinThreads);
  }
  const cudaError_t e2 = cudaFreeAsync(ws, s);
  if (e == cudaSuccess) e = e2;
  if (e != cudaSuccess) return fail((int)e);
  count_launches(2);
  return GEMV_SUCCESS;
}

}  // namespace
}  // namespace gemv

using namespace gemv;

extern "C" {

gemv_status_t gemv_kv8_append(gemv_dtype_t dtype, const gemv_kv8_cache_t *cache, const void *k, int64_t k_stride, const void *v,
                              int64_t v_stride, const int32_t *lens, const int32_t *starts, int S, int64_t N,
                              gemv_stream_t stream) {
  if (dtype < GEMV_DTYPE_F32 || dtype > GEMV_DTYPE_BF16 || S < 0 || N < 0) return GEMV_ERR_INVALID_VALUE;
  int64_t kv_bytes;
  gemv_status_t st = check_cache(cache, &kv_bytes);
  if (st != GEMV_SUCCESS) return st;
  if (S == 0 || N == 0 || cache->heads == 0) return GEMV_SUCCESS;
  if (N > 0x7fffffff || (starts == nullptr && N % S != 0)) return GEMV_ERR_INVALID_VALUE;
  const int size = dtype == GEMV_DTYPE_F32 ? 4 : 2;
  const int64_t row = (int64_t)cache->heads * cache->dim;
  if (k_stride < row || v_stride < row) return GEMV_ERR_INVALID_VALUE;
  int64_t kb, vb;
  if (!span(N, row, k_stride, size, &kb) || !span(N, row, v_stride, size, &vb)) return GEMV_ERR_INVALID_VALUE;
  if (!cache_pointers(cache) || k == nullptr || v == nullptr || lens == nullptr || !aligned(k, size) || !aligned(v, size) ||
      !aligned(lens, 4) || !aligned(starts, 4))
    return GEMV_ERR_INVALID_VALUE;
  // nothing that is written may overlap anything else
  const int64_t sb = cache->blocks * cache->heads * 4;
  const struct { const void *p; int64_t n; } part[] = {
      {cache->k, kv_bytes}, {cache->v, kv_bytes}, {cache->k_scale, sb}, {cache->v_scale, sb},
      {cache->table, (int64_t)S * cache->width * 4}, {k, kb}, {v, vb}, {lens, (int64_t)S * 4}, {starts, ((int64_t)S + 1) * 4}};
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 9; ++j)
      if (overlaps(part[i].p, part[i].n, part[j].p, part[j].n)) return GEMV_ERR_INVALID_VALUE;
  KvArgs a = cache_args(cache);
  if ((st = device_status_word(&a.status)) != GEMV_SUCCESS) return st;
  a.new_k = k;
  a.new_v = v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.lens = lens;
  a.starts = starts;
  a.S = S;
  a.N = N;
  a.T = (int)(N / S);
  a.dtype = (int)dtype;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int sms = 0;
  if ((st = device_sms(&sms)) != GEMV_SUCCESS) return st;
  const cudaError_t e = cache->dim == 64 ? append<64>(a, sms, s) : cache->dim == 128 ? append<128>(a, sms, s)
                        : cache->dim == 192 ? append<192>(a, sms, s) : append<256>(a, sms, s);
  if (e != cudaSuccess) return fail((int)e);
  count_launches(1);
  return GEMV_SUCCESS;
}

gemv_status_t gemv_kv8_read(gemv_dtype_t dtype, const gemv_kv8_cache_t *cache, void *k, int64_t k_stride, void *v,
                            int64_t v_stride, const int32_t *lens, const int32_t *starts, int S, int64_t N,
                            gemv_stream_t stream) {
  if (dtype < GEMV_DTYPE_F32 || dtype > GEMV_DTYPE_BF16 || S < 0 || N < 0) return GEMV_ERR_INVALID_VALUE;
  int64_t kv_bytes;
  gemv_status_t st = check_cache(cache, &kv_bytes);
  if (st != GEMV_SUCCESS) return st;
  if (S == 0 || N == 0 || cache->heads == 0 || (k == nullptr && v == nullptr)) return GEMV_SUCCESS;
  if (N > 0x7fffffff || (starts == nullptr && N % S != 0)) return GEMV_ERR_INVALID_VALUE;
  const int size = dtype == GEMV_DTYPE_F32 ? 4 : 2;
  const int64_t row = (int64_t)cache->heads * cache->dim;
  int64_t kb = 0, vb = 0;
  if (k != nullptr && (k_stride < row || !aligned(k, size) || !span(N, row, k_stride, size, &kb))) return GEMV_ERR_INVALID_VALUE;
  if (v != nullptr && (v_stride < row || !aligned(v, size) || !span(N, row, v_stride, size, &vb))) return GEMV_ERR_INVALID_VALUE;
  if (!cache_pointers(cache) || lens == nullptr || !aligned(lens, 4) || !aligned(starts, 4)) return GEMV_ERR_INVALID_VALUE;
  // nothing that is written may overlap anything else
  const int64_t sb = cache->blocks * cache->heads * 4;
  const struct { const void *p; int64_t n; } part[] = {
      {k, kb}, {v, vb}, {cache->k, kv_bytes}, {cache->v, kv_bytes}, {cache->k_scale, sb}, {cache->v_scale, sb},
      {cache->table, (int64_t)S * cache->width * 4}, {lens, (int64_t)S * 4}, {starts, ((int64_t)S + 1) * 4}};
  for (int i = 0; i < 2; ++i)
    for (int j = i + 1; j < 9; ++j) {
      if (i == 0 && j == 1 && columns(k, k_stride, v, v_stride, row, size)) continue;
      if (overlaps(part[i].p, part[i].n, part[j].p, part[j].n)) return GEMV_ERR_INVALID_VALUE;
    }
  KvArgs a = cache_args(cache);
  if ((st = device_status_word(&a.status)) != GEMV_SUCCESS) return st;
  a.out_k = k;
  a.out_v = v;
  a.sides = (k != nullptr) + (v != nullptr);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.lens = lens;
  a.starts = starts;
  a.S = S;
  a.N = N;
  a.T = (int)(N / S);
  a.dtype = (int)dtype;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->dim == 64 ? read_back<64>(a, s) : cache->dim == 128 ? read_back<128>(a, s)
                        : cache->dim == 192 ? read_back<192>(a, s) : read_back<256>(a, s);
  if (e != cudaSuccess) return fail((int)e);
  count_launches(1);
  return GEMV_SUCCESS;
}

gemv_status_t gemv_kv8_attention(gemv_dtype_t dtype, const gemv_kv8_cache_t *cache, const void *q, int64_t q_stride,
                                 const int32_t *lens, void *out, float *lse, int S, int T, int q_heads, float scale,
                                 int64_t window, int64_t sinks, gemv_stream_t stream) {
  if ((dtype != GEMV_DTYPE_F16 && dtype != GEMV_DTYPE_BF16) || S < 0 || T < 0 || q_heads < 0 || window < 0 || sinks < 0)
    return GEMV_ERR_INVALID_VALUE;
  int64_t kv_bytes;
  gemv_status_t st = check_cache(cache, &kv_bytes);
  if (st != GEMV_SUCCESS) return st;
  if (T > GEMV_KV8_MAX_TOKENS) return GEMV_ERR_UNSUPPORTED;
  if (S == 0 || T == 0 || q_heads == 0) return GEMV_SUCCESS;
  if (cache->heads == 0 || q_heads % cache->heads != 0 || q_heads > 65535) return GEMV_ERR_INVALID_VALUE;
  const int64_t row = (int64_t)q_heads * cache->dim, tokens = (int64_t)S * T;
  if (q_stride < row) return GEMV_ERR_INVALID_VALUE;
  int64_t qb, ob;
  if (!span(tokens, row, q_stride, 2, &qb) || !mul_ok(tokens, row * 2, &ob)) return GEMV_ERR_INVALID_VALUE;
  if (!cache_pointers(cache) || q == nullptr || out == nullptr || lens == nullptr || !aligned(q, 2) || !aligned(out, 2) ||
      !aligned(lens, 4) || !aligned(lse, 4))
    return GEMV_ERR_INVALID_VALUE;
  const int64_t sb = cache->blocks * cache->heads * 4;
  const struct { const void *p; int64_t n; } part[] = {
      {out, ob}, {lse, tokens * q_heads * 4}, {q, qb}, {lens, (int64_t)S * 4}, {cache->k, kv_bytes}, {cache->v, kv_bytes},
      {cache->k_scale, sb}, {cache->v_scale, sb}, {cache->table, (int64_t)S * cache->width * 4}};
  for (int i = 0; i < 2; ++i)
    for (int j = i + 1; j < 9; ++j)
      if (overlaps(part[i].p, part[i].n, part[j].p, part[j].n)) return GEMV_ERR_INVALID_VALUE;
  int sms = 0;
  if ((st = device_sms(&sms)) != GEMV_SUCCESS) return st;
  KvArgs a = cache_args(cache);
  if ((st = device_status_word(&a.status)) != GEMV_SUCCESS) return st;
  a.timeout_ns = wait_limit(&a.test_stall);
  a.q = q;
  a.q_stride = q_stride;
  a.lens = lens;
  a.out = out;
  a.lse = lse;
  a.S = S;
  a.T = T;
  a.group = q_heads / cache->heads;
  a.dtype = (int)dtype;
  // (positions are below it, by the limit on the table's width)
  const int64_t most = (int64_t)kKvMaxWidth * kKvBlock;
  a.window = (int)(window < most ? window : most);
  a.sinks = (int)(sinks < most ? sinks : most);
  a.scale_log2 = scale * 1.44269504088896f;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // rows of queries that meet a block at once: a tile of eight, or two (the registers of
  // more than two tiles' sums are there for 64 channels only)
  const int rows = T * a.group;
  switch (cache->dim) {
    case 64:
      return rows <= 8 ? attend<64, 1>(a, sms, s) : rows <= 16 ? attend<64, 2>(a, sms, s)
             : rows <= 24 ? attend<64, 3>(a, sms, s) : attend<64, 4>(a, sms, s);
    case 128:
      return rows <= 8 ? attend<128, 1>(a, sms, s) : attend<128, 2>(a, sms, s);
    case 192:
      return rows <= 8 ? attend<192, 1>(a, sms, s) : attend<192, 2>(a, sms, s);
    default:
      return rows <= 8 ? attend<256, 1>(a, sms, s) : attend<256, 2>(a, sms, s);
  }
}

}  // extern "C"
