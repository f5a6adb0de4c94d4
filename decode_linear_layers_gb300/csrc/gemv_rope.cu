// gemv_qk_norm_rope and gemv_rope_frequencies: the norm of each head of the queries and
// keys and the rotation by their positions, in one pass.
//
//     n_c = x_c w_c / sqrt(mean_c x_c^2 + eps)
//     (y_a, y_b) = factor (n_a cos t - n_b sin t, n_b cos t + n_a sin t),  t = position x inv_freq[i]
//
// for the pair i of channels (a, b): (i, i + rot / 2), or (2 i, 2 i + 1).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/gemv.h"
#include "gemv_f8.cuh"
#include "gemv_internal.h"
#include "gemv_launch.cuh"

namespace gemv {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxDim = 512;

struct RopeArgs {
  const void *x[2] = {nullptr, nullptr}, *w[2] = {nullptr, nullptr};  // queries, keys
  void *y[2] = {nullptr, nullptr};
  int64_t xs[2] = {0, 0}, ys[2] = {0, 0};
  const float *inv_freq = nullptr;
  const int32_t *lens = nullptr, *starts = nullptr;
  int64_t N = 0;
  int heads[2] = {0, 0};
  int S = 0, T = 0, dim = 0, rot = 0, per = 1, chunks = 1;
  bool inter = false;
  float eps = 0.f, factor = 1.f;
};

// The position of a row; false for a row that no sequence has (one warp, converged).
__device__ __forceinline__ bool rope_position(const RopeArgs &a, int64_t row, int lane, int32_t &pos) {
  int s;
  int64_t b, n;
  if (a.starts == nullptr) {
    s = (int)(row / a.T);
    b = (int64_t)s * a.T;
    n = a.T;
  } else {  // the last sequence that starts at the row or before, in steps of 32
    int lo = 0, hi = a.S;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, i = lo + lane * step;
      const int below = __popc(__ballot_sync(0xffffffffu, i < hi && (int64_t)__ldg(a.starts + i) <= row));
      if (below == 0) break;
      lo += (below - 1) * step;
      hi = lo + step < hi ? lo + step : hi;
    }
    s = lo;
    b = __ldg(a.starts + s);
    n = (int64_t)__ldg(a.starts + s + 1) - b;
    if (row < b || row >= b + n) return false;
  }
  const int64_t before = (int64_t)__ldg(a.lens + s) - n;
  pos = (int32_t)(before + row - b);
  return before >= 0;
}

// cos and sin of pos x f.  The product is formed in turns, as a whole number of 2^-64
// turns, whose overflow drops whole turns; its top 32 bits, as fp32, are good to 2^-23
// radians at any position (a product in fp32 would be off by 2^-24 of the angle itself,
// 0.008 at 131072).  Turns a radian to 96 bits: 64 are off by 2^-65 of a turn for each
// radian, of which there may be 2^55 (3.8e-4 radians for f = 2^20 at the last position).
__device__ __forceinline__ void rope_turn(float f, int32_t pos, float &c, float &s) {
  constexpr uint64_t kPerRadian = 0x28BE60DB9391054Aull;  // 2^64 / (2 pi), and 32 bits more
  constexpr uint32_t kRest = 0x7F09D5F4u;
  const uint32_t bits = __float_as_uint(f), e = (bits >> 23) & 0xff;
  const uint64_t m = (bits & 0x7fffff) | (e != 0 ? 0x800000u : 0u);  // |f| = m 2^-sh
  const int sh = 150 - (int)(e != 0 ? e : 1);
  const uint64_t rest = __umulhi((uint32_t)m, kRest), lo = m * kPerRadian + rest, hi = __umul64hi(m, kPerRadian) + (lo < rest ? 1 : 0);
  uint64_t t = sh >= 128 ? 0 : sh >= 64 ? hi >> (sh - 64) : sh > 0 ? (lo >> sh) | (hi << (64 - sh)) : sh > -64 ? lo << -sh : 0;
  t *= (uint64_t)(int64_t)pos;
  if ((bits >> 31) != 0) t = 0 - t;
  const int32_t x = (int32_t)((t + 0x80000000ull) >> 32);
  sincospif((float)x * 4.656612873077393e-10f /* 2^-31 */, &s, &c);
}

// Two fp32 values as one operand, and packed arithmetic on them.
__device__ __forceinline__ uint64_t rope_two(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 rope_apart(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t rope_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t rope_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Eight values: loads that may be of what the kernel writes later (in place), stores.
template <int DT>
struct RopeRaw : F8Raw<DT> {
  __device__ __forceinline__ void fetch(const void *p, int64_t i) {
    const uint4 *q = reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(p) + i * (DT == GEMV_DTYPE_F32 ? 4 : 2));
#pragma unroll
    for (int h = 0; h < F8Raw<DT>::kWords / 4; ++h) {
      uint4 v;
      asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(q + h));
      this->w[4 * h] = v.x;
      this->w[4 * h + 1] = v.y;
      this->w[4 * h + 2] = v.z;
      this->w[4 * h + 3] = v.w;
    }
  }
};
template <int DT>
__device__ __forceinline__ void rope_store8(void *p, int64_t i, const uint64_t (&o)[4]) {
  const float2 a = rope_apart(o[0]), b = rope_apart(o[1]), c = rope_apart(o[2]), d = rope_apart(o[3]);
  if constexpr (DT == GEMV_DTYPE_F32) {
    float4 *q = reinterpret_cast<float4 *>(reinterpret_cast<float *>(p) + i);
    q[0] = make_float4(a.x, a.y, b.x, b.y);
    q[1] = make_float4(c.x, c.y, d.x, d.y);
  } else {
    *reinterpret_cast<uint4 *>(reinterpret_cast<unsigned short *>(p) + i) =
        make_uint4(f8_pack16(a.x, a.y, DT), f8_pack16(b.x, b.y, DT), f8_pack16(c.x, c.y, DT), f8_pack16(d.x, d.y, DT));
  }
}

// P lanes have a head, 16 channels each: two pieces of eight, in which both channels of
// its eight pairs lie (the eight channels of the first half and those rot / 2 further on;
// or sixteen neighbours; behind the rotated channels sixteen others).  A warp takes
// 32 / P heads of a row at a time, `per` times; its lanes work out the row's cosines
// once, a few pairs each, and keep those of their own pairs, times the weights, in registers
// over the heads: an output is 1 / rms times a sum of two products, packed two by two.
// Bound by the bytes, in and out once each, and by instructions (15 k tokens of 40 heads of
// 128, us with weights and cosines apart / multiplied ahead and packed: 62 / 47, three CTAs an SM; with two
// and two or three turns' reads on their way 49, 47); a single
// token by its chain of dependent reads (starts, lens, frequencies beside the heads).
// kFull: every channel turns.
template <int DT, int P, bool kInter, bool kFull>
__global__ void __launch_bounds__(kRopeThreads, 3) k_qk_norm_rope(const RopeArgs a) {
  constexpr int kHeads = 32 / P;                        // of a turn
  constexpr int kMine = kHeads >= 8 ? 1 : 8 / kHeads;   // cosines that a lane works out
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, u = lane % P, grp = lane / P;
  const int64_t warp = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = warp / a.chunks;
  if (row >= a.N) return;
  const int all = a.heads[0] + a.heads[1], turns = (all + kHeads - 1) / kHeads;
  int turn = (int)(warp - row * a.chunks) * a.per;
  const int end = turn + a.per < turns ? turn + a.per : turns;

  const int half = a.rot / 2;
  const bool turned = 8 * u < half;  // this lane has rotated pairs
  const int c0 = kInter ? 16 * u : turned ? 8 * u : a.rot + (8 * u - half) * 2;
  const int c1 = kInter || !turned ? c0 + 8 : c0 + half;
  const bool has0 = c0 < a.dim, has1 = c1 < a.dim;

  RopeRaw<DT> next[2];  // the next turn's values, on their way
  auto side = [&](int t) { return t * kHeads + grp < a.heads[0] ? 0 : 1; };  // queries, keys
  auto start = [&](int t) { return (int64_t)(t * kHeads + grp - (side(t) ? a.heads[0] : 0)) * a.dim; };
  auto begin = [&](int t, RopeRaw<DT> (&x)[2]) {  // the reads of a turn
    x[0].zero();
    x[1].zero();
    if (t < end && t * kHeads + grp < all) {
      const int64_t from = row * a.xs[side(t)] + start(t);
      if (has0) x[0].fetch(a.x[side(t)], from + c0);
      if (has1) x[1].fetch(a.x[side(t)], from + c1);
    }
  };
  begin(turn, next);

  int32_t pos = 0;
  if (!rope_position(a, row, lane, pos)) return;
  float cs[8], sn[8];
  {
    float c[kMine], s[kMine];
#pragma unroll
    for (int p = 0; p < kMine; ++p) {
      const int i = 8 * u + (kHeads >= 8 ? grp & 7 : grp * kMine) + p;
      c[p] = 1.f;
      s[p] = 0.f;
      if (i < half) {
        rope_turn(__ldg(a.inv_freq + i), pos, c[p], s[p]);
        c[p] *= a.factor;
        s[p] *= a.factor;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      cs[j] = __shfl_sync(0xffffffffu, c[j % kMine], j / kMine * P + u);
      sn[j] = __shfl_sync(0xffffffffu, s[j % kMine], j / kMine * P + u);
    }
  }

  // Of two channels at a time (x, y): their own factors, and those of their partners.  Half: the
  // neighbours j, j + 1 of the first piece and of the second; else a pair.
  uint64_t own[8], other[8];
  int have = -1;  // whose weights are in them
  for (; turn < end; ++turn) {
    const int k = side(turn);
    const int64_t at = row * a.ys[k] + start(turn);
    const bool on = turn * kHeads + grp < all;
    if (have != k) {
      have = k;
      F8Raw<DT> w[2];
      const bool weighs = a.w[k] != nullptr;
      w[0].zero();
      w[1].zero();
      if (weighs && has0) w[0].load(a.w[k], c0);
      if (weighs && has1) w[1].load(a.w[k], c1);
      auto weight = [&](int c) { return weighs ? w[c / 8].get(c % 8) : 1.f; };
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (kInter) {
          const float wa = weight(2 * j), wb = weight(2 * j + 1);
          own[j] = rope_two(wa * cs[j], wb * cs[j]);
          other[j] = rope_two(-wb * sn[j], wa * sn[j]);
        } else {
          const int i = 2 * j % 8;  // j < 4: channels i, i + 1 of the first piece, else of the second
          const float x = weight(2 * j), y = weight(2 * j + 1), px = weight((2 * j + 8) % 16), py = weight((2 * j + 9) % 16);
          own[j] = rope_two(x * cs[i], y * cs[i + 1]);
          other[j] = j < 4 ? rope_two(-px * sn[i], -py * sn[i + 1]) : rope_two(px * sn[i], py * sn[i + 1]);
        }
      }
    }
    uint64_t v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = rope_two(next[0].get(2 * j), next[0].get(2 * j + 1));
      v[4 + j] = rope_two(next[1].get(2 * j), next[1].get(2 * j + 1));
    }
    begin(turn + 1, next);
    if (a.w[0] != nullptr || a.w[1] != nullptr) {  // (the same for all lanes)
      uint64_t two = rope_mul(v[0], v[0]), more = rope_mul(v[1], v[1]);
#pragma unroll
      for (int j = 2; j < 8; j += 2) {
        two = rope_fma(v[j], v[j], two);
        more = rope_fma(v[j + 1], v[j + 1], more);
      }
      const float2 s0 = rope_apart(two), s1 = rope_apart(more);
      float sum = (s0.x + s0.y) + (s1.x + s1.y);
#pragma unroll
      for (int d = 1; d < P; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (a.w[k] != nullptr) {
        const float inv = rsqrtf(sum / (float)a.dim + a.eps);
        const uint64_t inv2 = rope_two(inv, inv);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = rope_mul(v[j], inv2);
      }
    }
    uint64_t o[2][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint64_t kept = rope_mul(v[j], own[j]);
      uint64_t partner = v[j ^ 4];
      if constexpr (kInter) {
        const float2 p = rope_apart(v[j]);
        partner = rope_two(p.y, p.x);
      }
      uint64_t r = rope_fma(partner, other[j], kept);
      // (chosen, not multiplied by 0: a channel beyond the rotated ones may be anything)
      if constexpr (!kFull) r = (kInter ? 8 * u + j < half : turned) ? r : kept;
      o[j / 4][j % 4] = r;
    }
    if (on) {
      if (has0) rope_store8<DT>(a.y[k], at + c0, o[0]);
      if (has1) rope_store8<DT>(a.y[k], at + c1, o[1]);
    }
  }
}

// Any number of channels, any alignment: a warp has a head at a time, a lane every
// 32nd pair (behind the rotated channels, of two neighbours), up to kPairs of them, value by
// value; it keeps its pairs' cosines over the heads, as above (bf16, 41 k heads of 128 channels,
// 36 of them rotated: 26 us, bound by instructions; with the cosines worked out for each
// head 71).
template <int DT, int kPairs>
__global__ void __launch_bounds__(kRopeThreads) k_qk_norm_rope_any(const RopeArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, all = a.heads[0] + a.heads[1], half = a.rot / 2;
  const int64_t warp = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = warp / a.chunks;
  if (row >= a.N) return;
  int32_t pos = 0;
  if (!rope_position(a, row, lane, pos)) return;
  // (reads that the kernel's own writes may follow, in place)
  auto get = [](const void *p, int64_t i) {
    if constexpr (DT == GEMV_DTYPE_F32) return reinterpret_cast<const volatile float *>(p)[i];
    const unsigned short b = reinterpret_cast<const volatile unsigned short *>(p)[i];
    return DT == GEMV_DTYPE_F16 ? __half2float(__ushort_as_half(b)) : __uint_as_float((uint32_t)b << 16);
  };
  auto put = [](void *p, int64_t i, float v) {
    if constexpr (DT == GEMV_DTYPE_F32)
      reinterpret_cast<float *>(p)[i] = v;
    else
      reinterpret_cast<unsigned short *>(p)[i] = f8_round16(v, DT);
  };
  float cs[kPairs], sn[kPairs], w0[kPairs], w1[kPairs];
  auto pair = [&](int j) { return lane + 32 * j; };
  auto c0 = [&](int j) { return pair(j) < half ? (a.inter ? 2 * pair(j) : pair(j)) : a.rot + 2 * (pair(j) - half); };
  auto c1 = [&](int j) { return pair(j) < half && !a.inter ? pair(j) + half : c0(j) + 1; };
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    cs[j] = sn[j] = 0.f;
    if (pair(j) < half) {
      rope_turn(__ldg(a.inv_freq + pair(j)), pos, cs[j], sn[j]);
      cs[j] *= a.factor;
      sn[j] *= a.factor;
    }
  }
  int have = -1;
  int h = (int)(warp - row * a.chunks) * a.per;
  const int end = h + a.per < all ? h + a.per : all;
  for (; h < end; ++h) {
    const int k = h < a.heads[0] ? 0 : 1;
    const int64_t head = (int64_t)(h - (k ? a.heads[0] : 0)) * a.dim;
    const int64_t from = row * a.xs[k] + head, to = row * a.ys[k] + head;
    const bool norm = a.w[k] != nullptr;
    if (have != k) {
      have = k;
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        w0[j] = norm && c0(j) < a.dim ? get(a.w[k], c0(j)) : 1.f;
        w1[j] = norm && c1(j) < a.dim ? get(a.w[k], c1(j)) : 1.f;
      }
    }
    float x0[kPairs], x1[kPairs], sum = 0.f;
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      x0[j] = c0(j) < a.dim ? get(a.x[k], from + c0(j)) : 0.f;
      x1[j] = c1(j) < a.dim ? get(a.x[k], from + c1(j)) : 0.f;
    }
    if (norm) {
#pragma unroll
      for (int j = 0; j < kPairs; ++j) sum = fmaf(x0[j], x0[j], fmaf(x1[j], x1[j], sum));
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      const float inv = rsqrtf(sum / (float)a.dim + a.eps);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        x0[j] *= inv * w0[j];
        x1[j] *= inv * w1[j];
      }
    }
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const bool turned = pair(j) < half;
      if (c0(j) < a.dim) put(a.y[k], to + c0(j), turned ? x0[j] * cs[j] - x1[j] * sn[j] : x0[j]);
      if (c1(j) < a.dim) put(a.y[k], to + c1(j), turned ? x1[j] * cs[j] + x0[j] * sn[j] : x1[j]);
    }
  }
}

bool mul_ok(int64_t a, int64_t b, int64_t *out) { return !__builtin_mul_overflow(a, b, out); }
bool aligned(const void *p, int bytes) { return ((uintptr_t)p % (uintptr_t)bytes) == 0; }

// N rows of `row` bytes, `stride` bytes apart.
struct Rows {
  const void *p;
  int64_t row, stride, span;
};
bool make_rows(Rows *r, const void *p, int64_t N, int64_t row, int64_t stride, int size) {
  int64_t n;
  r->p = p;
  return mul_ok(row, size, &r->row) && mul_ok(stride, size, &r->stride) && mul_ok(N - 1, r->stride, &n) &&
         !__builtin_add_overflow(n, r->row, &r->span);
}
// They share a byte, or may: columns of one matrix do not, whatever their rows.
bool meet(const Rows &a, const Rows &b) {
  if (a.row == 0 || b.row == 0 || !overlaps(a.p, a.span, b.p, b.span)) return false;
  if (a.stride != b.stride) return true;
  int64_t d = (int64_t)((uintptr_t)b.p - (uintptr_t)a.p) % a.stride;
  if (d < 0) d += a.stride;
  return d < a.row || a.stride - d < b.row;
}

// Turns (of a row's `most`) that a warp takes one after the other: one while the SMs hold all
// warps at once, 24 each, else as many as keep those busy, up to sixteen, over which the row's
// cosines are kept.
int share(int64_t turns, int most, int sms) {
  const int64_t n = turns / ((int64_t)sms * 24), cap = most < 16 ? most : 16;
  return (int)(n < 1 ? 1 : n < cap ? n : cap);
}

template <int DT, int P>
cudaError_t rope_launch(RopeArgs a, int sms, cudaStream_t s) {
  const int turns = (a.heads[0] + a.heads[1] + 32 / P - 1) / (32 / P);
  a.per = share(a.N * turns, turns, sms);
  a.chunks = (turns + a.per - 1) / a.per;
  const int64_t ctas = (a.N * a.chunks + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const bool full = a.rot == a.dim && a.dim % 16 == 0;
  auto kern = a.inter ? (full ? k_qk_norm_rope<DT, P, true, true> : k_qk_norm_rope<DT, P, true, false>)
                      : (full ? k_qk_norm_rope<DT, P, false, true> : k_qk_norm_rope<DT, P, false, false>);
  return launch_k(kern, dim3((unsigned)ctas), dim3(kRopeThreads), 0, s, launch_overlap(), a);
}
template <int DT, int kPairs>
cudaError_t rope_any(RopeArgs a, int sms, cudaStream_t s) {
  const int all = a.heads[0] + a.heads[1];
  a.per = share(a.N * all, all, sms);
  a.chunks = (all + a.per - 1) / a.per;
  const int64_t ctas = (a.N * a.chunks + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  return launch_k(k_qk_norm_rope_any<DT, kPairs>, dim3((unsigned)ctas), dim3(kRopeThreads), 0, s, launch_overlap(), a);
}
template <int DT>
cudaError_t rope(const RopeArgs &a, bool vec, int sms, cudaStream_t s) {
  if (vec)
    return a.dim <= 64    ? rope_launch<DT, 4>(a, sms, s)
           : a.dim <= 128 ? rope_launch<DT, 8>(a, sms, s)
           : a.dim <= 256 ? rope_launch<DT, 16>(a, sms, s)
                          : rope_launch<DT, 32>(a, sms, s);
  // pairs of a lane: the rotated ones, and two by two the other channels
  const int pairs = (a.rot / 2 + (a.dim - a.rot + 1) / 2 + 31) / 32;
  return pairs <= 1   ? rope_any<DT, 1>(a, sms, s)
         : pairs == 2 ? rope_any<DT, 2>(a, sms, s)
         : pairs <= 4 ? rope_any<DT, 4>(a, sms, s)
                      : rope_any<DT, 8>(a, sms, s);
}

}  // namespace
}  // namespace gemv

using namespace gemv;

extern "C" {

gemv_status_t gemv_qk_norm_rope(gemv_dtype_t dtype, const void *q, int64_t q_stride, void *q_out, int64_t q_out_stride,
                                const void *q_weight, int q_heads, const void *k, int64_t k_stride, void *k_out,
                                int64_t k_out_stride, const void *k_weight, int k_heads, int dim, float eps,
                                const float *inv_freq, int rot, gemv_rope_layout_t layout, float factor, const int32_t *lens,
                                const int32_t *starts, int S, int64_t N, gemv_stream_t stream) {
  if (dtype < GEMV_DTYPE_F32 || dtype > GEMV_DTYPE_BF16 || q_heads < 0 || k_heads < 0 || dim < 0 || S < 0 || N < 0 ||
      rot < 0 || rot > dim || rot % 2 != 0 || !(eps >= 0.f) ||
      (layout != GEMV_ROPE_HALF && layout != GEMV_ROPE_INTERLEAVED))
    return GEMV_ERR_INVALID_VALUE;
  if (dim > kRopeMaxDim) return GEMV_ERR_UNSUPPORTED;
  if (q_heads > 65535 || k_heads > 65535) return GEMV_ERR_INVALID_VALUE;
  if (S == 0 || N == 0 || dim == 0 || q_heads + k_heads == 0) return GEMV_SUCCESS;
  if (N > 0x7fffffff || (starts == nullptr && N % S != 0)) return GEMV_ERR_INVALID_VALUE;
  const int size = dtype == GEMV_DTYPE_F32 ? 4 : 2;
  const int heads[2] = {q_heads, k_heads};
  const void *const x[2] = {q, k}, *const w[2] = {q_weight, k_weight};
  void *const y[2] = {q_out, k_out};
  const int64_t xs[2] = {q_stride, k_stride}, ys[2] = {q_out_stride, k_out_stride};
  RopeArgs a;
  Rows in[2] = {}, out[2] = {};
  // pieces of eight channels, whole pairs of pieces
  bool vec = dim % 8 == 0 && (layout == GEMV_ROPE_INTERLEAVED || rot % 16 == 0);
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0) continue;
    const int64_t row = (int64_t)heads[i] * dim;
    if (x[i] == nullptr || y[i] == nullptr || xs[i] < row || ys[i] < row || !aligned(x[i], size) || !aligned(y[i], size) ||
        !aligned(w[i], size) || !make_rows(&in[i], x[i], N, row, xs[i], size) || !make_rows(&out[i], y[i], N, row, ys[i], size))
      return GEMV_ERR_INVALID_VALUE;
    vec = vec && aligned(x[i], 16) && aligned(y[i], 16) && aligned(w[i], 16) && xs[i] * size % 16 == 0 && ys[i] * size % 16 == 0;
    a.x[i] = x[i];
    a.y[i] = y[i];
    a.w[i] = w[i];
    a.xs[i] = xs[i];
    a.ys[i] = ys[i];
    a.heads[i] = heads[i];
  }
  if (lens == nullptr || (rot > 0 && inv_freq == nullptr) || !aligned(lens, 4) || !aligned(starts, 4) || !aligned(inv_freq, 4))
    return GEMV_ERR_INVALID_VALUE;
  // what is written overlaps nothing but, in place, its own input
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0) continue;
    if (!(x[i] == y[i] && xs[i] == ys[i]) && meet(out[i], in[i])) return GEMV_ERR_INVALID_VALUE;
    if (meet(out[i], in[1 - i]) || (i == 0 && meet(out[0], out[1]))) return GEMV_ERR_INVALID_VALUE;
    const struct { const void *p; int64_t n; } rest[] = {{q_weight, (int64_t)dim * size}, {k_weight, (int64_t)dim * size},
                                                         {inv_freq, (int64_t)rot * 2}, {lens, (int64_t)S * 4},
                                                         {starts, ((int64_t)S + 1) * 4}};
    for (const auto &r : rest)
      if (overlaps(out[i].p, out[i].span, r.p, r.n)) return GEMV_ERR_INVALID_VALUE;
  }
  a.inv_freq = inv_freq;
  a.lens = lens;
  a.starts = starts;
  a.N = N;
  a.S = S;
  a.T = (int)(N / S);
  a.dim = dim;
  a.rot = rot;
  a.inter = layout == GEMV_ROPE_INTERLEAVED;
  a.eps = eps;
  a.factor = factor;
  int sms = 0;
  const gemv_status_t st = device_sms(&sms);
  if (st != GEMV_SUCCESS) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == GEMV_DTYPE_F32   ? rope<GEMV_DTYPE_F32>(a, vec, sms, s)
                        : dtype == GEMV_DTYPE_F16 ? rope<GEMV_DTYPE_F16>(a, vec, sms, s)
                                                  : rope<GEMV_DTYPE_BF16>(a, vec, sms, s);
  if (e != cudaSuccess) return fail((int)e);
  count_launches(1);
  return GEMV_SUCCESS;
}

gemv_status_t gemv_rope_frequencies(float *inv_freq, int rot, double base, gemv_rope_scaling_t scaling, double factor,
                                    double original, double low, double high, float *attention) {
  if (rot < 0 || rot % 2 != 0 || !(base > 1.0) || !isfinite(base) || scaling < GEMV_ROPE_SCALE_NONE ||
      scaling > GEMV_ROPE_SCALE_INDEX || (rot > 0 && inv_freq == nullptr))
    return GEMV_ERR_INVALID_VALUE;
  if (scaling != GEMV_ROPE_SCALE_NONE && (!(factor > 0.0) || !isfinite(factor))) return GEMV_ERR_INVALID_VALUE;
  if (scaling >= GEMV_ROPE_SCALE_TURNS && (!(original > 0.0) || !(low > 0.0) || !(high > low) || !isfinite(original) || !isfinite(high)))
    return GEMV_ERR_INVALID_VALUE;
  constexpr double kTurn = 6.283185307179586;
  if (scaling == GEMV_ROPE_SCALE_BASE && rot > 2) base *= pow(factor, (double)rot / (rot - 2));
  // the pair that turns `turns` times in the original context
  auto pair_of = [&](double turns) { return rot * log(original / (turns * kTurn)) / (2.0 * log(base)); };
  double first = 0.0, last = 0.0;
  if (scaling == GEMV_ROPE_SCALE_INDEX) {
    first = fmax(floor(pair_of(high)), 0.0);
    last = fmin(ceil(pair_of(low)), rot - 1.0);
    if (last <= first) last = first + 0.001;  // (no ramp: a step)
  }
  for (int i = 0; i < rot / 2; ++i) {
    const double f = pow(base, -2.0 * i / rot);
    double keep = 1.0;  // share of the unscaled frequency
    if (scaling == GEMV_ROPE_SCALE_LINEAR)
      keep = 0.0;
    else if (scaling == GEMV_ROPE_SCALE_TURNS)
      keep = fmin(fmax((original * f / kTurn - low) / (high - low), 0.0), 1.0);
    else if (scaling == GEMV_ROPE_SCALE_INDEX)
      keep = 1.0 - fmin(fmax((i - first) / (last - first), 0.0), 1.0);
    const bool scaled = scaling != GEMV_ROPE_SCALE_NONE && scaling != GEMV_ROPE_SCALE_BASE;
    inv_freq[i] = (float)(scaled ? keep * f + (1.0 - keep) * f / factor : f);
  }
  if (attention != nullptr) *attention = scaling == GEMV_ROPE_SCALE_INDEX && factor > 1.0 ? (float)(0.1 * log(factor) + 1.0) : 1.f;
  return GEMV_SUCCESS;
}

}  // extern "C"
