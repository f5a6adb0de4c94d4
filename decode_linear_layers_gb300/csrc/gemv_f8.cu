// gemv_f8 and gemv_f8_quantize: argument checks, the choice of the form, launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/gemv.h"
#include "gemv_f8.cuh"
#include "gemv_internal.h"
#include "gemv_launch.cuh"

namespace gemv {
namespace {

// Clusters of n CTAs that the device holds at a time (asked once; the devices of a process
// are taken to be alike).  A cluster's CTAs share a part of the GPU, so that clusters of
// three, say, do not fill it: a second round of them would cost more than smaller ones.
template <int N, bool kPrompt>
int64_t f8_clusters(int n) {
  using F = F8Form<N, kPrompt>;
  static std::atomic<int> known[kTcMaxSlices + 1];
  int v = known[n].load(std::memory_order_relaxed);
  if (v == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n);
    cfg.blockDim = dim3(F::kThreads);
    cfg.dynamicSmemBytes = F::kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)n;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&v, k_f8<N, kPrompt>, &cfg) != cudaSuccess || v < 1) {
      (void)cudaGetLastError();
      v = 1;
    }
    known[n].store(v, std::memory_order_relaxed);
  }
  return v;
}

template <int N, bool kPrompt>
gemv_status_t f8_launch(F8Args a, const void *A, const void *x, int64_t K, int sms, cudaStream_t s) {
  using F = F8Form<N, kPrompt>;
  a.tm = (int)((a.M + (kPrompt ? N : kF8Rows) - 1) / (kPrompt ? N : kF8Rows));
  a.tn = kPrompt ? (a.B + kF8Rows - 1) / kF8Rows : 1;
  a.tiles = (int64_t)a.tm * a.tn;
  cudaError_t e = allow_smem_once<k_f8<N, kPrompt>>(F::kSmem);
  if (e != cudaSuccess) return fail((int)e);
  // The tiles that fill no whole round of the CTAs.  Each form's cost, in k-blocks of a CTA:
  //   - a round of their own, as many as a tile has;
  //   - shared among all CTAs, their share of it and the join, kJoin (us, shared / a round:
  //     14336x3584 B=4 16.3 / 14.5, 10000x3584 B=100 20.1 / 22.1, 24000x3584 B=100 33.4 /
  //     41.1; prompts, whose parts are 128 KB each, 11593x3584 B=1430 98.7 / 85.2,
  //     11592x7168 130 / 115); not for few tiles, where its second launch shows;
  //   - a cluster for each, their slice and its sum.  That weighs more against a round that
  //     leaves SMs free, whose k-blocks are quick, than against the join (us, clusters / a
  //     round: 4096x1024 B=1 5.2 / 4.5, 4096x2048 B=64 7.0 / 7.7, 28672x1024 B=16 8.3 / 7.1,
  //     14336x4096 B=300 31.4 / 42.5, 7168x2048 B=1024 25.0 / 22.3; clusters / shared:
  //     28672x4096 B=16 22.7 / 25.1, 20480x4096 B=1 18.2 / 20.6, 10000x8192 B=500 46.5 / 57.4).
  constexpr int64_t kJoin = kPrompt ? 28 : 12;
  const int64_t rest = a.tiles % sms;
  int64_t W = a.tiles < sms ? a.tiles : sms;  // one CTA per SM
  int64_t least = (a.tiles + sms - 1) / sms * a.groups, sum = kPrompt ? 14 : 12;
  if (a.tiles * 2 > sms && a.tiles * a.groups / sms + kJoin < least) {
    least = a.tiles * a.groups / sms + kJoin;
    a.shared = rest;
    W = sms;
    sum = kPrompt ? 6 : 2;
  }
  for (int64_t n = 2; n <= kTcMaxSlices && n <= a.groups; ++n) {
    const int64_t c = f8_clusters<N, kPrompt>((int)n), q = a.tiles / (c * n), r = a.tiles - q * c * n;
    const int64_t cost = q * a.groups + (a.groups + n - 1) / n + sum;
    if (r > 0 && r <= c && cost < least) {
      least = cost;
      a.slices = (int)n;
      a.shared = r;
      W = (q > 0 ? c : r) * n;
    }
  }
  a.sharers = (int)(a.shared * a.groups < W ? a.shared * a.groups : W);
  CUtensorMap map_a, map_x;
  if (!map_bytes(&map_a, A, a.M, K, kPrompt ? N : kF8Rows, kF8Group) ||
      !map_bytes(&map_x, x, a.B, K, kPrompt ? kF8Rows : N, kF8Group))
    return fail((int)cudaErrorInvalidValue);
  const bool join = a.slices == 1 && a.shared > 0;
  void *ws = nullptr;
  if (join) {
    e = workspace(&ws, (size_t)(W * 2 * F::kPartial * 4), s);
    if (e != cudaSuccess) return fail((int)e);
    a.ws = static_cast<float *>(ws);
  }
  const int pdl = launch_overlap();
  if (e == cudaSuccess)
    e = launch_k_cluster_x(k_f8<N, kPrompt>, dim3((unsigned)W), dim3(F::kThreads), (size_t)F::kSmem, s, pdl, a.slices,
                           kPrompt ? map_x : map_a, kPrompt ? map_a : map_x, a);
  int n = 1;
  if (e == cudaSuccess && join) {
    e = launch_k(k_f8_join<N, kPrompt>, dim3((unsigned)a.shared, (unsigned)(F::kPartial / kF8JoinPiece)),
                 dim3(kF8JoinThreads), 0, s, pdl, a);
    n = 2;
  }
  if (ws != nullptr) {
    const cudaError_t e2 = cudaFreeAsync(ws, s);
    if (e == cudaSuccess) e = e2;
  }
  if (e != cudaSuccess) return fail((int)e);
  count_launches(n);
  return GEMV_SUCCESS;
}

gemv_status_t f8_launch_pair(F8Args a, const void *A, const void *x, int64_t K, int sms, cudaStream_t s) {
  using F = F8Pair;
  a.tm = (int)((a.M + F::kN - 1) / F::kN);
  a.tn = (a.B + 255) / 256;
  a.tiles = (int64_t)a.tm * a.tn;
  const int64_t pairs = a.tiles < sms / 2 ? a.tiles : sms / 2;
  cudaError_t e = allow_smem_once<k_f8_pair>(F::kSmem);
  if (e != cudaSuccess) return fail((int)e);
  CUtensorMap map_a, map_x;
  if (!map_bytes(&map_a, A, a.M, K, 128, kF8Group) || !map_bytes(&map_x, x, a.B, K, 128, kF8Group))
    return fail((int)cudaErrorInvalidValue);
  e = launch_k_cluster_x(k_f8_pair, dim3((unsigned)(2 * pairs)), dim3(F::kThreads), (size_t)F::kSmem, s, launch_overlap(), 2,
                         map_x, map_a, a);
  if (e != cudaSuccess) return fail((int)e);
  count_launches(1);
  return GEMV_SUCCESS;
}

bool mul_ok(int64_t a, int64_t b, int64_t *out) { return !__builtin_mul_overflow(a, b, out); }
bool aligned(const void *p, int bytes) { return ((uintptr_t)p % (uintptr_t)bytes) == 0; }

template <int DT>
cudaError_t quantize(const void *x, uint8_t *q, float *scale, int64_t K, int64_t G, int64_t groups, int sms, cudaStream_t s) {
  const bool eight = K % 8 == 0 && aligned(x, 16) && aligned(q, 8);
  const bool two = K % 2 == 0 && aligned(x, DT == GEMV_DTYPE_F32 ? 8 : 4) && aligned(q, 2);
  constexpr int kTeams = kF8QThreads / kF8QTeam;
  // two groups of a team in flight once every SM's threads have one
  const bool many = groups > (int64_t)sms * (2048 / kF8QTeam) * 2;
  auto go = [&](auto kern, int u) {
    const int64_t grid = (groups + kTeams * u - 1) / (kTeams * u);
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return launch_k(kern, dim3((unsigned)grid), dim3(kF8QThreads), 0, s, launch_overlap(), x, q, scale, K, (int)G, groups);
  };
  if (eight) return many ? go(k_f8_quantize<DT, 8, 2>, 2) : go(k_f8_quantize<DT, 8, 1>, 1);
  if (two) return many ? go(k_f8_quantize<DT, 2, 2>, 2) : go(k_f8_quantize<DT, 2, 1>, 1);
  return many ? go(k_f8_quantize<DT, 1, 2>, 2) : go(k_f8_quantize<DT, 1, 1>, 1);
}

}  // namespace
}  // namespace gemv

using namespace gemv;

extern "C" {

gemv_status_t gemv_f8_quantize(gemv_dtype_t dtype, const void *x, uint8_t *q, float *scale, int64_t K, int B,
                               gemv_stream_t stream) {
  if (K < 0 || B < 0 || dtype < GEMV_DTYPE_F32 || dtype > GEMV_DTYPE_BF16) return GEMV_ERR_INVALID_VALUE;
  if (K == 0 || B == 0) return GEMV_SUCCESS;
  const int sx = dtype == GEMV_DTYPE_F32 ? 4 : 2;
  const int64_t G = (K + GEMV_F8_GROUP - 1) / GEMV_F8_GROUP;
  int64_t bk, xb, groups, sb;
  if (K > 0x7fffffff || !mul_ok(B, K, &bk) || !mul_ok(bk, sx, &xb) || !mul_ok(B, G, &groups) || !mul_ok(groups, 4, &sb))
    return GEMV_ERR_INVALID_VALUE;
  if (x == nullptr || q == nullptr || scale == nullptr || !aligned(x, sx) || !aligned(scale, 4)) return GEMV_ERR_INVALID_VALUE;
  if (overlaps(q, bk, x, xb) || overlaps(scale, sb, x, xb) || overlaps(scale, sb, q, bk)) return GEMV_ERR_INVALID_VALUE;
  int sms = 0;
  gemv_status_t st = device_sms(&sms);
  if (st != GEMV_SUCCESS) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == GEMV_DTYPE_F32   ? quantize<GEMV_DTYPE_F32>(x, q, scale, K, G, groups, sms, s)
                        : dtype == GEMV_DTYPE_F16 ? quantize<GEMV_DTYPE_F16>(x, q, scale, K, G, groups, sms, s)
                                                  : quantize<GEMV_DTYPE_BF16>(x, q, scale, K, G, groups, sms, s);
  if (e != cudaSuccess) return fail((int)e);
  count_launches(1);
  return GEMV_SUCCESS;
}

gemv_status_t gemv_f8(const uint8_t *A, const float *a_scale, const uint8_t *x, const float *x_scale, const void *bias,
                      void *y, gemv_dtype_t y_dtype, int64_t M, int64_t K, int B, gemv_stream_t stream) {
  if (M < 0 || K < 0 || B < 0 || y_dtype < GEMV_DTYPE_F32 || y_dtype > GEMV_DTYPE_BF16) return GEMV_ERR_INVALID_VALUE;
  if (K % GEMV_F8_ALIGN != 0) return GEMV_ERR_INVALID_VALUE;
  if (M == 0 || B == 0) return GEMV_SUCCESS;
  const int sy = y_dtype == GEMV_DTYPE_F32 ? 4 : 2;
  const int64_t G = (K + GEMV_F8_GROUP - 1) / GEMV_F8_GROUP;
  int64_t mk, bk, bm, yb, bg;
  // row and column numbers are 32-bit coordinates of the copies; tiles, and the k-blocks of
  // one CTA, are counted in 32 bits
  if (M > 0x7fffff00 || B > 0x7fffff00 || K > ((int64_t)1 << 29)) return GEMV_ERR_INVALID_VALUE;
  const int64_t tiles = (M / 128 + 1) * ((int64_t)B / 128 + 1);
  if (tiles > ((int64_t)1 << 30) || tiles * G > ((int64_t)1 << 37) || !mul_ok(M, K, &mk) || !mul_ok(B, K, &bk) ||
      !mul_ok(B, M, &bm) || !mul_ok(bm, sy, &yb) || !mul_ok(B, G * 4, &bg))
    return GEMV_ERR_INVALID_VALUE;
  const int64_t ag = (M + GEMV_F8_GROUP - 1) / GEMV_F8_GROUP * G * 4;
  if (y == nullptr || (K > 0 && (A == nullptr || a_scale == nullptr || x == nullptr || x_scale == nullptr)))
    return GEMV_ERR_INVALID_VALUE;
  if (!aligned(A, GEMV_F8_ALIGN) || !aligned(x, GEMV_F8_ALIGN) || !aligned(a_scale, 4) || !aligned(x_scale, 4) ||
      !aligned(y, sy) || !aligned(bias, sy))
    return GEMV_ERR_INVALID_VALUE;
  if (overlaps(y, yb, A, mk) || overlaps(y, yb, x, bk) || overlaps(y, yb, a_scale, ag) || overlaps(y, yb, x_scale, bg) ||
      overlaps(y, yb, bias, M * sy))
    return GEMV_ERR_INVALID_VALUE;
  int sms = 0;
  gemv_status_t st = device_sms(&sms);
  if (st != GEMV_SUCCESS) return st;
  F8Args a;
  a.a_scale = a_scale;
  a.x_scale = x_scale;
  a.bias = bias;
  a.y = y;
  a.y_dtype = (int)y_dtype;
  a.M = M;
  a.B = B;
  a.groups = (int)G;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) {
    const int64_t grid = (bm + 255) / 256;
    const cudaError_t e = launch_k(k_f8_empty, dim3((unsigned)(grid < sms * 8 ? grid : sms * 8)), dim3(256), 0, s, launch_overlap(), a);
    if (e != cudaSuccess) return fail((int)e);
    count_launches(1);
    return GEMV_SUCCESS;
  }
  st = device_status_word(&a.status);
  if (st != GEMV_SUCCESS) return st;
  a.timeout_ns = wait_limit(&a.test_stall);
  if (B <= 16) return f8_launch<16, false>(a, A, x, K, sms, s);
  if (B <= 32) return f8_launch<32, false>(a, A, x, K, sms, s);
  if (B <= 64) return f8_launch<64, false>(a, A, x, K, sms, s);
  // More vectors: they are the tile's rows, a thread's factor then one number per k-block
  // (us, 128 vectors as rows / as columns: 14336x4096 16.7 / 20.9, 4096x14336 21.4 / 23.9).
  // Tiles of 256 weight rows where those occupy half the SMs, of 128 else (us, 256 / 128:
  // 4096x4096 B=256 20.6 / 17.4, B=1000 21.6 / 26.1, 1000x2048 B=500 17.3 / 11.9).
  if (B <= 128 || (M + 255) / 256 * (((int64_t)B + 127) / 128) * 2 < sms) return f8_launch<128, true>(a, A, x, K, sms, s);
  // From two rounds of 256 x 256 tiles on, pairs of SMs: they move less through shared memory
  // and so draw less power (us, pairs / single, thirty calls in a row: 4096x14336 B=8192 391 /
  // 425, B=4864 228 / 240, B=3584 160 / 171; 128256x4096 B=256 132 / 141; 28672x4096 B=4096
  // 429 / 430; 4096x4096 B=2048, one round, 40.7 / 40.4).  They know whole rounds only, and
  // lose where the last one is nearly empty: 4096x14336 B=2432 and 2560, 160 tiles for 152
  // pairs' places, 155 / 109 and 156 / 135; B=2816 157 / 143.
  if ((M + 255) / 256 * (((int64_t)B + 255) / 256) >= sms) return f8_launch_pair(a, A, x, K, sms, s);
  return f8_launch<256, true>(a, A, x, K, sms, s);
}

}  // extern "C"
