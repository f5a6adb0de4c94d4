// gemv_kv8_prefix_attention: argument checks, the choice of the form, launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gemv.h"
#include "gemv_internal.h"
#include "gemv_kv8_host.h"
#include "gemv_launch.cuh"
#include "gemv_prefix.cuh"

namespace gemv {
namespace {

// Where sharing pays: three launches and the time to fill the tensor cores against reading
// every sequence's tokens apart, which takes some 9 us and 0.1 us for each MB of them and
// eight query rows that meet them (the tables' width is what the host knows of the lengths).
// us, apart / shared, 8 heads of 128 channels, 4 query heads each: 32 sequences behind 2048
// tokens (142 MB) 24 / 37, 64 behind 2048 (285) 40 / 33, 8 behind 8192 (136) 23 / 39, 8 behind
// 32768 (538) 65 / 54; 16 queries each (eight times eight rows), 2 behind 2048 (9 x 8) 20 / 39, 8
// behind 2048 (36 x 8) 36 / 37, 32 behind 512 (42 x 8) 57 / 44; 256 channels: 8 behind 8192
// (272) 46 / 43, 32 behind 2048 (285) 50 / 48.
// A group's blocks take the shared kernel what two or three times eight rows take apart: 32 groups of
// one, two, three and four sequences behind 8192 tokens 95 / 174, 123 / 175, 255 / 179, 306 / 183; 4
// groups of four 38 / 50, of six 52 / 49.  A group may be a single sequence, whose queries share its
// blocks: one of 64 behind 65536 tokens, 4 heads of 256, 8 query heads each 891 / 176.  (Over 3858
// batches of up to 64 groups the choice costs 0.7 % against the better form each time, 3.7 % by the
// rows alone; the worst 1.5 times as long and 2.6.)
bool px_pays(int64_t S, int64_t groups, int64_t width, int64_t heads, int64_t dim, int64_t rows) {
  const double mb = (double)width * kKvBlock * (double)heads * (double)dim * 2e-6;  // of a sequence
  const double eights = (double)S * (double)((rows + 7) / 8);
  if (groups == 0 || eights < 3.0 * (double)groups) return false;
  return mb * (eights - 2.5 * (double)(groups == S ? groups : groups - 1)) > (dim <= 128 ? 230.0 : 300.0);
}

// Scratch memory that a call takes at most, by the size of its output; `otherwise` is the call
// passed on.  Full tiles take some 4 times the output, one row to a tile of eight up to 20 times;
// hundreds of groups of a few rows, each with whole tiles for every head (66 to 133 KB), any number
// of times (512 groups of three sequences with 32 heads of 128: 620 MB for 13).
bool px_fits(int64_t bytes, int64_t out) { return bytes <= (64 << 20) + 24 * out; }

template <int D, int NT, class Else>
gemv_status_t attend(KvArgs a, int sms, cudaStream_t s, Else otherwise) {
  using F = KvForm<D, NT>;
  using P = PxForm<D>;
  a.row_tiles = (a.T * a.group + NT * 8 - 1) / (NT * 8);
  if ((int64_t)a.heads * a.row_tiles > 65535) return GEMV_ERR_UNSUPPORTED;
  const int items = a.heads * a.row_tiles;
  const int64_t px_items = ((int64_t)a.S * a.T * a.group / P::kRows + a.groups + 1) * a.heads;
  if (px_items + sms > 0x7fffffff) return otherwise();
  const int pdl = launch_overlap();
  a.workers = sms * F::kWarps;
  // partial results of the sequences' own blocks, where they are, those of the shared ones, where
  // they are (pieces of 16 bytes all)
  int64_t own, px, bytes;
  const int64_t own_items = (int64_t)a.S * items;
  if (!mul_ok(a.workers + own_items, kv_part<D, NT>() * 4, &own) || !mul_ok(sms + px_items, P::kSets * P::kPart * 4, &px) ||
      __builtin_add_overflow(own, px, &bytes) || __builtin_add_overflow(bytes, (own_items + px_items) * 16, &bytes) ||
      !px_fits(bytes, (int64_t)a.S * a.T * a.heads * a.group * D * 2))
    return otherwise();
  void *ws = nullptr;
  cudaError_t e = workspace(&ws, (size_t)bytes, s);
  if (e != cudaSuccess) return fail((int)e);
  char *p = static_cast<char *>(ws);
  a.ws = reinterpret_cast<float *>(p);
  a.px_ws = reinterpret_cast<float *>(p + own);
  a.parts = reinterpret_cast<int4 *>(p + own + px);
  a.px_parts = a.parts + own_items;
  const bool half = a.dtype == GEMV_DTYPE_F16;
  e = half ? allow_smem_once<k_kv8_prefix<D, GEMV_DTYPE_F16>>(P::kSmem) : allow_smem_once<k_kv8_prefix<D, GEMV_DTYPE_BF16>>(P::kSmem);
  if (e == cudaSuccess)
    e = launch_k(half ? k_kv8_prefix<D, GEMV_DTYPE_F16> : k_kv8_prefix<D, GEMV_DTYPE_BF16>, dim3((unsigned)sms), dim3(P::kThreads),
                 (size_t)P::kSmem, s, pdl, a);
  if (e == cudaSuccess) e = allow_smem_once<k_kv8_attention<D, NT, false, true>>(F::kSmem);
  if (e == cudaSuccess)
    e = launch_k(k_kv8_attention<D, NT, false, true>, dim3((unsigned)sms), dim3(F::kThreads), (size_t)F::kSmem, s, pdl, a);
  if (e == cudaSuccess) {
    const int rows = a.T * a.group < NT * 8 ? a.T * a.group : NT * 8;
    auto join = [&](auto kern, int along) {
      return launch_k(kern, dim3((unsigned)a.S, (unsigned)items, (unsigned)((rows * (D / 16) + along - 1) / along)),
                      dim3(kPxJoinThreads), 0, s, pdl, a, sms);
    };
    // threads for the parts of the same channels: four where an item of the shared blocks is in many
    if (px_items * 4 <= sms)
      e = join(k_kv8_prefix_join<D, NT, 4>, kPxJoinThreads / 4);
    else
      e = join(k_kv8_prefix_join<D, NT, 1>, kPxJoinThreads);
  }
  const cudaError_t e2 = cudaFreeAsync(ws, s);
  if (e == cudaSuccess) e = e2;
  if (e != cudaSuccess) return fail((int)e);
  count_launches(3);
  return GEMV_SUCCESS;
}

}  // namespace
}  // namespace gemv

using namespace gemv;

extern "C" {

gemv_status_t gemv_kv8_prefix_attention(gemv_dtype_t dtype, const gemv_kv8_cache_t *cache, const void *q, int64_t q_stride,
                                        const int32_t *lens, const int32_t *firsts, const int32_t *prefix, int groups, void *out,
                                        float *lse, int S, int T, int q_heads, float scale, gemv_stream_t stream) {
  if ((dtype != GEMV_DTYPE_F16 && dtype != GEMV_DTYPE_BF16) || S < 0 || T < 0 || q_heads < 0 || groups < 0)
    return GEMV_ERR_INVALID_VALUE;
  int64_t kv_bytes;
  gemv_status_t st = check_cache(cache, &kv_bytes);
  if (st != GEMV_SUCCESS) return st;
  if (T > GEMV_KV8_MAX_TOKENS) return GEMV_ERR_UNSUPPORTED;
  if (S == 0 || T == 0 || q_heads == 0) return GEMV_SUCCESS;
  if (cache->heads == 0 || q_heads % cache->heads != 0 || q_heads > 65535) return GEMV_ERR_INVALID_VALUE;
  if (groups > S || (firsts == nullptr && groups > 1) || (groups > 0 && prefix == nullptr)) return GEMV_ERR_INVALID_VALUE;
  const int64_t row = (int64_t)q_heads * cache->dim, tokens = (int64_t)S * T;
  // (places of the work list and rows of a group are counted in 31 bits)
  const int64_t rows = (int64_t)T * (q_heads / cache->heads);
  const int64_t most = (S * rows / 128 + groups) * cache->heads * kPxCost2;
  const bool pass_on = !px_pays(S, groups, cache->width, cache->heads, cache->dim, rows) ||
                       most > 0x7fffffff / cache->width || S * rows > (1 << 30);
  if (q_stride < row) return GEMV_ERR_INVALID_VALUE;
  int64_t qb, ob;
  if (!span(tokens, row, q_stride, 2, &qb) || !mul_ok(tokens, row * 2, &ob)) return GEMV_ERR_INVALID_VALUE;
  if (!cache_pointers(cache) || q == nullptr || out == nullptr || lens == nullptr || !aligned(q, 2) || !aligned(out, 2) ||
      !aligned(lens, 4) || !aligned(lse, 4) || !aligned(firsts, 4) || !aligned(prefix, 4))
    return GEMV_ERR_INVALID_VALUE;
  const int64_t sb = cache->blocks * cache->heads * 4;
  const struct { const void *p; int64_t n; } part[] = {
      {out, ob}, {lse, tokens * q_heads * 4}, {q, qb}, {lens, (int64_t)S * 4}, {cache->k, kv_bytes}, {cache->v, kv_bytes},
      {cache->k_scale, sb}, {cache->v_scale, sb}, {cache->table, (int64_t)S * cache->width * 4},
      {firsts, ((int64_t)groups + 1) * 4}, {prefix, (int64_t)groups * 4}};
  for (int i = 0; i < 2; ++i)
    for (int j = i + 1; j < 11; ++j)
      if (overlaps(part[i].p, part[i].n, part[j].p, part[j].n)) return GEMV_ERR_INVALID_VALUE;
  auto otherwise = [&]() { return gemv_kv8_attention(dtype, cache, q, q_stride, lens, out, lse, S, T, q_heads, scale, 0, 0, stream); };
  if (pass_on) return otherwise();
  int sms = 0;
  if ((st = device_sms(&sms)) != GEMV_SUCCESS) return st;
  KvArgs a = cache_args(cache);
  if ((st = device_status_word(&a.status)) != GEMV_SUCCESS) return st;
  a.timeout_ns = wait_limit(&a.test_stall);
  a.q = q;
  a.q_stride = q_stride;
  a.lens = lens;
  a.firsts = firsts;
  a.prefix = prefix;
  a.groups = groups;
  a.out = out;
  a.lse = lse;
  a.S = S;
  a.T = T;
  a.group = q_heads / cache->heads;
  a.dtype = (int)dtype;
  a.scale_log2 = scale * 1.44269504088896f;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // rows of queries of one sequence that meet a block of its own at once, as in gemv_kv8_attention
  switch (cache->dim) {
    case 64:
      return rows <= 8 ? attend<64, 1>(a, sms, s, otherwise) : rows <= 16 ? attend<64, 2>(a, sms, s, otherwise)
             : rows <= 24 ? attend<64, 3>(a, sms, s, otherwise) : attend<64, 4>(a, sms, s, otherwise);
    case 128:
      return rows <= 8 ? attend<128, 1>(a, sms, s, otherwise) : attend<128, 2>(a, sms, s, otherwise);
    case 192:
      return rows <= 8 ? attend<192, 1>(a, sms, s, otherwise) : attend<192, 2>(a, sms, s, otherwise);
    default:
      return rows <= 8 ? attend<256, 1>(a, sms, s, otherwise) : attend<256, 2>(a, sms, s, otherwise);
  }
}

}  // extern "C"
