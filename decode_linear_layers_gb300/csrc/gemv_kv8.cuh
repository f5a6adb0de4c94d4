// Kernels of the 8-bit cache of keys and values: the append of new tokens
// (gemv_kv8_append), cached tokens read back (gemv_kv8_read) and the attention over it
// (gemv_kv8_attention).
//
// A block holds kKvBlock = 64 tokens of one head: the keys as 64 rows of D e4m3 values,
// the values as D rows of 64 (token index innermost, so that the second product finds
// consecutive tokens, its summation index, in consecutive bytes), and one scale for
// each, a power of two.
#pragma once

#include "gemv_f8.cuh"

namespace gemv {

constexpr int kKvBlock = 64;
constexpr int kKvStatusTable = 64;  // a block needed lies outside the pool, or past the table

struct KvArgs {
  uint8_t *k = nullptr, *v = nullptr;
  float *k_scale = nullptr, *v_scale = nullptr;
  const int32_t *table = nullptr, *lens = nullptr;
  int64_t blocks = 0;
  int heads = 0, width = 0;
  int S = 0, T = 0;
  int *status = nullptr;
  // append
  const void *new_k = nullptr, *new_v = nullptr;
  int64_t k_stride = 0, v_stride = 0;
  const int32_t *starts = nullptr;
  int64_t N = 0;
  int dtype = 0, per_cta = 1;
  // read
  void *out_k = nullptr, *out_v = nullptr;
  int sides = 0;  // keys, values: how many of them
  // attention
  const void *q = nullptr;
  void *out = nullptr;
  float *lse = nullptr;
  float *ws = nullptr;    // partial results: two for each warp
  int4 *parts = nullptr;  // of each item: the first warp with a part, parts, which of that warp's
  int workers = 0;        // warps of the attention kernel: ws has two partial results of each
  int64_t q_stride = 0;
  int64_t timeout_ns = 0;
  int group = 0, window = 0, sinks = 0, row_tiles = 0, test_stall = 0;
  float scale_log2 = 0.f;  // softmax scale x log2 e
  // attention of groups that share a prefix
  const int32_t *firsts = nullptr, *prefix = nullptr;  // first sequence of each group (and S); its tokens in common
  int groups = 0;
  float *px_ws = nullptr;    // partial results of the shared blocks
  int4 *px_parts = nullptr;  // of each item of theirs: the first CTA with a part, parts
};

// ------------------------------------------------------------------ values
// Two e4m3 values (the low, the high half of a word) as fp16, exact.
__device__ __forceinline__ uint32_t kv_half2_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t kv_half2_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
// The smallest power of two s >= 2^-126 with m <= 448 s: 448 = 1.75 x 2^8, so s = 2^(e - 8)
// for m = f x 2^e with f <= 1.75, and twice that above.
__device__ __forceinline__ float kv_power(float m) {
  const int bits = __float_as_int(m);
  int e = ((bits >> 23) & 0xff) - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
  return __int_as_float((e < 1 ? 1 : e) << 23);
}
// Four e4m3 values times a power of two, rounded to e4m3 again (exact but for
// subnormal results).
__device__ __forceinline__ uint32_t kv_rescale4(uint32_t w, float r) {
  const float2 a = f16x2_to_f2(kv_half2_lo(w)), b = f16x2_to_f2(kv_half2_hi(w));
  return f8_pack2(a.x * r, a.y * r) | (f8_pack2(b.x * r, b.y * r) << 16);
}

// ------------------------------------------------------------------ rows and blocks
// The rows of gemv_kv8_append and gemv_kv8_read: n of each sequence, its last n positions.
// A CTA (blockIdx.x) has one block that they reach.
struct KvReach {
  int64_t first, before, len, p0;  // the sequence's first row, its tokens before that, all, the block's first token
  int32_t block;                   // of the pool
};
// One warp, converged; false where there is nothing to do.  `tell` (one thread of the CTA):
// reports a block that is missing, and (`once`: one CTA of those with the same blockIdx.x)
// a sequence with fewer tokens than rows.
__device__ __forceinline__ bool kv_reach(const KvArgs &a, int lane, bool tell, bool once, KvReach &r) {
  // the sequence, and which of its blocks
  int s;
  int64_t first, n, nth;  // its first new token, how many, and the block's number among those they reach
  if (a.starts == nullptr) {
    const int per = (a.T + kKvBlock - 2) / kKvBlock + 1;
    s = blockIdx.x / per;
    nth = blockIdx.x - s * per;
    first = (int64_t)s * a.T;
    n = a.T;
  } else {
    // n tokens reach at most n / 64 + 2 blocks: sequence s has the CTAs from
    // starts[s] / 64 + 2 s on
    // (each warp looks for the last such sequence in steps of 32)
    int lo = 0, hi = a.S;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, i = lo + lane * step;
      const bool from = i < hi && (int64_t)(__ldg(a.starts + i) / kKvBlock) + 2 * (int64_t)i <= (int64_t)blockIdx.x;
      const int below = __popc(__ballot_sync(0xffffffffu, from));
      lo += below > 0 ? (below - 1) * step : 0;
      hi = lo + step < hi ? lo + step : hi;
      if (below == 0) break;
    }
    s = lo;
    const int64_t b = __ldg(a.starts + s), e = __ldg(a.starts + s + 1);
    first = b < 0 ? 0 : b > a.N ? a.N : b;
    n = (e > a.N ? a.N : e) - first;
    nth = (int64_t)blockIdx.x - (b / kKvBlock + 2 * (int64_t)s);
  }
  r.first = first;
  r.len = __ldg(a.lens + s);
  r.before = r.len - n;
  if (n <= 0 || nth < 0) return false;
  if (r.before < 0) {  // fewer tokens than the new ones: nothing says where they go
    if (tell && nth == 0 && once && a.status != nullptr) atomicOr(a.status, kKvStatusTable);
    return false;
  }
  const int64_t blk = r.before / kKvBlock + nth;
  r.p0 = blk * kKvBlock;
  if (r.p0 >= r.len) return false;
  r.block = blk < a.width ? __ldg(a.table + (int64_t)s * a.width + blk) : -1;
  if (r.block < 0 || r.block >= a.blocks) {
    if (tell && a.status != nullptr) atomicOr(a.status, kKvStatusTable);
    return false;
  }
  return true;
}

// ------------------------------------------------------------------ append
// A CTA has a block that new tokens reach, and of it one or more units (a head's keys, or
// its values): it reads a unit's new tokens once (eight values of a token per load), finds
// their largest, and so the unit's scale; where that grows it moves the tokens the block
// held to the new scale; and it writes the new ones.  No other CTA touches the unit, so
// nothing is atomic.  Values pass through shared memory to lie token-innermost.  Bound by
// latency (lengths, table, tokens, one after the other) and instructions: 64 sequences of
// one new token 6 us, 5 prompts of 10 k tokens in all 17 us (67 MB: 9.8 at the copy rate).
constexpr int kKvAppendThreads = 256;
template <int D, int DT>
__global__ void __launch_bounds__(kKvAppendThreads) k_kv8_append(const KvArgs a) {
  constexpr int kPieces = D / 8;                          // of a token
  constexpr int kLoads = (kKvBlock * kPieces / kKvAppendThreads + 3) / 4 * 4;
  constexpr int kStride = kKvBlock / kLoads;              // threads along the tokens
  constexpr int kActive = kStride * kPieces;              // threads with channels
  static_assert(kActive <= kKvAppendThreads && kKvBlock % kLoads == 0);
  __shared__ float part[kKvAppendThreads / 32];
  __shared__ __align__(16) uint32_t tile[D * (kKvBlock / 4)];  // values: words of four tokens
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  KvReach b;
  if (!kv_reach(a, lane, tid == 0, blockIdx.y == 0, b)) return;
  const int64_t p0 = b.p0, len = b.len, before = b.before, first = b.first;
  const int32_t pb = b.block;
  const int held = before > p0 ? (int)(before - p0) : 0;             // tokens the block has
  const int end = len - p0 < kKvBlock ? (int)(len - p0) : kKvBlock;  // and will have
  const int64_t t0 = first + (p0 + held - before);                   // the first of its new tokens
  const int units = 2 * a.heads;
  for (int unit = blockIdx.y * a.per_cta; unit < units && unit < (int)(blockIdx.y + 1) * a.per_cta; ++unit) {
    const bool values = (unit & 1) != 0;
    const int h = unit >> 1;
    if (unit > (int)blockIdx.y * a.per_cta) __syncthreads();  // the unit before is done with shared memory
    const void *src = values ? a.new_v : a.new_k;
    const int64_t stride = values ? a.v_stride : a.k_stride;
    uint8_t *dst = (values ? a.v : a.k) + ((int64_t)pb * a.heads + h) * (kKvBlock * D);
    float *sc = (values ? a.v_scale : a.k_scale) + (int64_t)pb * a.heads + h;
    const float old = held > 0 ? *sc : 0.f;

    // this thread's eight channels of kLoads tokens: of every kStride-th token, or (values)
    // of four neighbouring ones, which share the words of the block's rows
    const bool vec = (reinterpret_cast<uintptr_t>(src) & 15) == 0 && (stride * (DT == GEMV_DTYPE_F32 ? 4 : 2)) % 16 == 0;
    const int ch = (tid % kPieces) * 8;
    auto token = [&](int i) {
      const int j = tid / kPieces;
      return values ? j * 4 + (i & 3) + (i >> 2) * 4 * kStride : j + i * kStride;
    };
    F8Raw<DT> x[kLoads];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int tok = token(i);
      x[i].zero();
      if (tid < kActive && tok >= held && tok < end) {
        const int64_t at = (t0 + tok - held) * stride + (int64_t)h * D + ch;
        if (vec) {
          x[i].load(src, at);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[i].set(j, src, at + j);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) m = fmaxf(m, x[i].top());
    if (m == __int_as_float(0x7f800000)) {  // an infinity: the finite values' largest
      m = 0.f;
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, f8_finite_abs(x[i].get(j)));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((tid & 31) == 0) part[tid >> 5] = m;
    __syncthreads();  // every thread has read the old scale, too
#pragma unroll
    for (int w = 0; w < kKvAppendThreads / 32; ++w) m = fmaxf(m, part[w]);
    const float scale = fmaxf(kv_power(m), old), r = 1.f / scale;  // powers of two: exact
    if (tid == 0) *sc = scale;
    const bool move = held > 0 && scale != old;
    const float ratio = old * r;

    if (!values) {
      if (move)
        for (int i = tid; i < held * (D / 16); i += kKvAppendThreads) {
          uint4 w = reinterpret_cast<const uint4 *>(dst)[i];
          w.x = kv_rescale4(w.x, ratio);
          w.y = kv_rescale4(w.y, ratio);
          w.z = kv_rescale4(w.z, ratio);
          w.w = kv_rescale4(w.w, ratio);
          reinterpret_cast<uint4 *>(dst)[i] = w;
        }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int tok = token(i);
        if (tid < kActive && tok >= held && tok < end)
          *reinterpret_cast<uint2 *>(dst + tok * D + ch) =
              make_uint2(f8_pack2(x[i].get(0) * r, x[i].get(1) * r) | (f8_pack2(x[i].get(2) * r, x[i].get(3) * r) << 16),
                         f8_pack2(x[i].get(4) * r, x[i].get(5) * r) | (f8_pack2(x[i].get(6) * r, x[i].get(7) * r) << 16));
      }
      continue;
    }
    // word `w` (four tokens) of channel c lies at tile[c][w ^ 4 (c / 8 mod 4)]: the lanes of
    // a warp, which write eight channels apart, spread over the banks, and four words of
    // a channel stay together
#pragma unroll
    for (int i = 0; i < kLoads; i += 4) {
      const int w = token(i) / 4;
      if (tid < kActive) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          tile[(ch + j) * (kKvBlock / 4) + (w ^ (((ch >> 3) & 3) * 4))] =
              f8_pack2(x[i].get(j) * r, x[i + 1].get(j) * r) | (f8_pack2(x[i + 2].get(j) * r, x[i + 3].get(j) * r) << 16);
      }
    }
    __syncthreads();
    // sixteen tokens of a channel at a time: with new ones, and with held ones to move;
    // bytes of no token stay
    const int q_lo = move ? 0 : held / 16, q_n = (end + 15) / 16 - q_lo;
    for (int i = tid; i < D * q_n; i += kKvAppendThreads) {
      const int c = q_n == 4 ? i / 4 : q_n == 1 ? i : i / q_n, at_q = q_lo + i - c * q_n, tok0 = at_q * 16;
      const uint32_t *from = tile + c * (kKvBlock / 4) + (at_q ^ ((c >> 3) & 3)) * 4;
      uint32_t *at = reinterpret_cast<uint32_t *>(dst) + c * (kKvBlock / 4) + at_q * 4;
      if (tok0 >= held && tok0 + 16 <= end) {
        *reinterpret_cast<uint4 *>(at) = *reinterpret_cast<const uint4 *>(from);
        continue;
      }
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const int lo = held - (tok0 + 4 * k), hi = end - (tok0 + 4 * k);  // bytes [lo, hi) of the word are new
        if (hi <= 0 || (!move && lo >= 4)) continue;
        uint32_t w = from[k];
        if (lo > 0 || hi < 4) {
          const uint32_t was = at[k];
          const uint32_t below = lo >= 4 ? 0xffffffffu : lo > 0 ? (1u << (8 * lo)) - 1 : 0u;  // held bytes
          const uint32_t above = hi >= 4 ? 0u : ~((1u << (8 * hi)) - 1);                       // bytes of no token
          w = (w & ~(below | above)) | ((move ? kv_rescale4(was, ratio) : was) & below) | (was & above);
        }
        at[k] = w;
      }
    }
  }
}

// ------------------------------------------------------------------ read
// The mirror of the append: cached tokens back as rows.  A warp has 64 x 64 values of a
// block and head at a time, keys or values, and no other does; there is nothing to share.
//   keys    a lane reads eight channels of a token (eight bytes), sixteen times
//   values  a lane reads sixteen tokens of eight channels (eight words of 16 bytes; four
//           lanes read a channel's 64 tokens) and turns 4 x 4 bytes at a time, so that it
//           has eight channels of a token to store, and eight neighbours 128 bytes (16 bits)
// Either way 64 or 128 bytes a lane are on their way at once.  Bound by the bytes.
constexpr int kKvReadThreads = 128;

__device__ __forceinline__ uint32_t kv_prmt(uint32_t a, uint32_t b, uint32_t how) { return __byte_perm(a, b, how); }
// Eight e4m3 values (channels, as two words) times the scale, as a row's elements.
template <int DT>
__device__ __forceinline__ void kv_row8(void *out, int64_t i, uint32_t lo, uint32_t hi, float scale, bool vec) {
  const float2 a = f16x2_to_f2(kv_half2_lo(lo)), b = f16x2_to_f2(kv_half2_hi(lo));
  const float2 c = f16x2_to_f2(kv_half2_lo(hi)), d = f16x2_to_f2(kv_half2_hi(hi));
  const float v[8] = {a.x * scale, a.y * scale, b.x * scale, b.y * scale, c.x * scale, c.y * scale, d.x * scale, d.y * scale};
  if constexpr (DT == GEMV_DTYPE_F32) {
    float *p = reinterpret_cast<float *>(out) + i;
    if (vec) {
      *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = v[j];
    }
  } else {
    unsigned short *p = reinterpret_cast<unsigned short *>(out) + i;
    const uint4 w = make_uint4(f8_pack16(v[0], v[1], DT), f8_pack16(v[2], v[3], DT), f8_pack16(v[4], v[5], DT), f8_pack16(v[6], v[7], DT));
    if (vec) {
      *reinterpret_cast<uint4 *>(p) = w;
    } else {
      const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = (unsigned short)(h[j / 2] >> (16 * (j & 1)));
    }
  }
}

template <int D, int DT>
__global__ void __launch_bounds__(kKvReadThreads) k_kv8_read(const KvArgs a) {
  constexpr int kParts = D / 64;  // 64 x 64 values: of a head's keys, and of its values
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  KvReach b;
  if (!kv_reach(a, lane, tid == 0, blockIdx.y == 0, b)) return;
  const int lo = b.before > b.p0 ? (int)(b.before - b.p0) : 0;                // the block's tokens that are asked for
  const int hi = b.len - b.p0 < kKvBlock ? (int)(b.len - b.p0) : kKvBlock;
  const int64_t row0 = b.first + b.p0 - b.before;                            // row of the block's token 0
  constexpr int kSize = DT == GEMV_DTYPE_F32 ? 4 : 2;
  const int of_side = a.heads * kParts;
  for (int part = blockIdx.y * (kKvReadThreads / 32) + (tid >> 5); part < a.sides * of_side; part += gridDim.y * (kKvReadThreads / 32)) {
    // keys first, then values, of those that are asked for
    const int side = part / of_side, at = part - side * of_side, h = at / kParts, q = at - h * kParts;
    const bool values = side == 1 || a.out_k == nullptr;
    void *const out = values ? a.out_v : a.out_k;
    const int64_t stride = values ? a.v_stride : a.k_stride;
    const bool vec = (reinterpret_cast<uintptr_t>(out) & 15) == 0 && (stride * kSize) % 16 == 0;
    const int64_t unit = (int64_t)b.block * a.heads + h;
    const float scale = __ldg((values ? a.v_scale : a.k_scale) + unit);
    const uint8_t *src = (values ? a.v : a.k) + unit * (kKvBlock * D) + q * (kKvBlock * 64);
    if (!values) {
      // bytes 4096 q .. of the block's keys, 16 pieces of 8 for each lane
      const uint2 *p = reinterpret_cast<const uint2 *>(src) + lane;
      uint2 x[16];
  #pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __ldg(p + i * 32);
  #pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int byte = q * (kKvBlock * 64) + (i * 32 + lane) * 8, tok = byte / D, ch = byte - tok * D;
        if (tok >= lo && tok < hi) kv_row8<DT>(out, (row0 + tok) * stride + (int64_t)h * D + ch, x[i].x, x[i].y, scale, vec);
      }
      continue;
    }
    const int ch = (lane >> 2) * 8, t0 = (lane & 3) * 16;  // channels 64 q + ch .., tokens t0 ..
    uint4 x[8];
  #pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __ldg(reinterpret_cast<const uint4 *>(src + (ch + j) * kKvBlock + t0));
  #pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t r[8];
  #pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = w == 0 ? x[j].x : w == 1 ? x[j].y : w == 2 ? x[j].z : x[j].w;
  #pragma unroll
      for (int g = 0; g < 2; ++g) {  // four channels of four tokens to four tokens of four channels
        const uint32_t e0 = kv_prmt(r[4 * g], r[4 * g + 1], 0x5140), e1 = kv_prmt(r[4 * g + 2], r[4 * g + 3], 0x5140);
        const uint32_t f0 = kv_prmt(r[4 * g], r[4 * g + 1], 0x7362), f1 = kv_prmt(r[4 * g + 2], r[4 * g + 3], 0x7362);
        r[4 * g] = kv_prmt(e0, e1, 0x5410);
        r[4 * g + 1] = kv_prmt(e0, e1, 0x7632);
        r[4 * g + 2] = kv_prmt(f0, f1, 0x5410);
        r[4 * g + 3] = kv_prmt(f0, f1, 0x7632);
      }
  #pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int tok = t0 + 4 * w + t;
        if (tok >= lo && tok < hi)
          kv_row8<DT>(out, (row0 + tok) * stride + (int64_t)h * D + q * 64 + ch, r[t], r[4 + t], scale, vec);
      }
    }
  }
}

// ------------------------------------------------------------------ attention: work
// What the T queries of a sequence see of it, in blocks: the `sink` first ones, then
// those from `from` on.
struct KvSeen {
  int len, sink, from, count;
};
// A group of sequences: [first, end), and the blocks that they have in common.
struct KvGroup {
  int first, end, blocks;
};
__device__ __forceinline__ KvGroup kv_group(const KvArgs &a, int g) {
  KvGroup k = {0, a.S, 0};
  if (a.firsts != nullptr) {
    k.first = __ldg(a.firsts + g);
    k.end = __ldg(a.firsts + g + 1);
    k.first = k.first < 0 ? 0 : k.first > a.S ? a.S : k.first;
    k.end = k.end < k.first ? k.first : k.end > a.S ? a.S : k.end;
  }
  const int n = __ldg(a.prefix + g) / kKvBlock;
  k.blocks = n < 0 || k.first == k.end ? 0 : n < a.width ? n : a.width;
  return k;
}
// The group that sequence s is in, or -1.
__device__ __forceinline__ int kv_group_of(const KvArgs &a, int s) {
  if (a.firsts == nullptr) return 0;
  int lo = 0, hi = a.groups;  // the last one that starts at s or before
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (__ldg(a.firsts + mid) <= s)
      lo = mid;
    else
      hi = mid;
  }
  return s >= __ldg(a.firsts + lo) && s < __ldg(a.firsts + lo + 1) ? lo : -1;
}
// Blocks of sequence s that are attended to for its whole group at once: those in common,
// if every query of it sees all of them, else none.
__device__ __forceinline__ int kv_shared(const KvArgs &a, int s, int len) {
  const int g = kv_group_of(a, s);
  if (g < 0) return 0;
  const int n = kv_group(a, g).blocks;
  return (int64_t)len - a.T >= (int64_t)n * kKvBlock ? n : 0;
}
template <bool kOwn = false>
__device__ __forceinline__ KvSeen kv_seen(const KvArgs &a, int s) {
  KvSeen v;
  v.len = __ldg(a.lens + s);
  v.len = v.len < 0 ? 0 : v.len;
  if ((int64_t)v.len > (int64_t)a.width * kKvBlock) v.len = a.width * kKvBlock;
  if constexpr (kOwn) {
    v.from = kv_shared(a, s, v.len);
    v.sink = 0;
    v.count = (v.len + kKvBlock - 1) / kKvBlock - v.from;
    return v;
  }
  const int64_t lo = a.window > 0 ? (int64_t)v.len - a.T - a.window + 1 : 0;
  v.from = lo > 0 ? (int)(lo / kKvBlock) : 0;
  const int need = a.window > 0 ? (a.sinks + kKvBlock - 1) / kKvBlock : 0;
  v.sink = need < v.from ? need : v.from;
  v.count = v.sink + (v.len + kKvBlock - 1) / kKvBlock - v.from;
  return v;
}

// The work list: the items (a sequence's heads and row tiles) one after the other, each
// with kKvItemCost places for its queries and its output and one for each block.  It is
// cut into equal ranges, one for each warp of the grid: a batch of very different lengths
// and a single long sequence both keep every SM busy, and no warp waits for another.
// A range holds the end of an item, whole items, and the start of one.
constexpr int kKvItemCost = 1;

__device__ __forceinline__ int kv_places(const KvSeen &v) { return v.count > 0 ? v.count + kKvItemCost : 0; }
// Places of one item of each of the sequences [from, to).  (A sequence has at most 2^24
// blocks: those of 32 fit 32 bits.)
template <bool kOwn>
__device__ __forceinline__ int64_t kv_between(const KvArgs &a, int from, int to, int lane) {
  int64_t n = 0;
  for (int i = from; i < to; i += 32)
    n += __reduce_add_sync(0xffffffffu, i + lane < to ? (unsigned)kv_places(kv_seen<kOwn>(a, i + lane)) : 0u);
  return n;
}
__device__ __forceinline__ int64_t kv_div(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// `total` places in ranges for W warps, the first `more` of them one longer.
struct KvShares {
  int64_t each, more;
  __device__ void cut(int64_t total, int64_t W) {
    each = kv_div(total, W);
    more = total - each * W;
  }
  __device__ int64_t first(int64_t w) const { return w * each + (w < more ? w : more); }
  __device__ int64_t owner(int64_t u) const {
    const int64_t longer = more * (each + 1);
    return u < longer ? kv_div(u, each + 1) : more + kv_div(u - longer, each);
  }
};

// An item, and the places [lo, hi) of its blocks.
template <bool kOwn>
struct KvItem {
  int64_t lo, hi;
  int s, item;
  KvSeen seen;
  __device__ void load(const KvArgs &a, int s_, int64_t at) {
    s = s_;
    item = 0;
    seen = kv_seen<kOwn>(a, s);
    lo = at + (seen.count > 0 ? kKvItemCost : 0);
    hi = lo + seen.count;
  }
  __device__ void next(const KvArgs &a) {
    if (seen.count > 0 && item + 1 < a.heads * a.row_tiles) {
      ++item;
      lo = hi + kKvItemCost;
      hi = lo + seen.count;
    } else {
      load(a, s + 1, hi);
    }
  }
  __device__ void skip(int64_t n) {  // n items of the same sequence
    item += (int)n;
    lo += n * (seen.count + kKvItemCost);
    hi = lo + seen.count;
  }
  // the item that ends past place u (u below the total)
  __device__ void seek(const KvArgs &a, int64_t u) {
    while (u >= hi) next(a);
  }
};

// ------------------------------------------------------------------ attention
__device__ __forceinline__ void kv_bulk(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(tc_smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(tc_smem_u32(bar))
               : "memory");
}
// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), fp16
__device__ __forceinline__ void kv_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The n lowest bits; none below 0, all from 64 on.
__device__ __forceinline__ uint64_t kv_low_bits(int64_t n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}
// Four 16-bit values from anywhere (a call: such rows are rare, and their loads many).
static __device__ __noinline__ uint2 kv_load4(const unsigned short *p) {
  const uint32_t a = __ldg(p), b = __ldg(p + 1), c = __ldg(p + 2), d = __ldg(p + 3);
  return make_uint2(a | (b << 16), c | (d << 16));
}
// Two 16-bit values: wider, and the larger ones of two pairs (none negative, NaN passed over).
__device__ __forceinline__ float kv_wide_lo(uint32_t w, int dt) {
  return dt == GEMV_DTYPE_F16 ? __half2float(__ushort_as_half((unsigned short)w)) : bf16_lo(w);
}
__device__ __forceinline__ float kv_wide_hi(uint32_t w, int dt) {
  return dt == GEMV_DTYPE_F16 ? __half2float(__ushort_as_half((unsigned short)(w >> 16))) : bf16_hi(w);
}
__device__ __forceinline__ uint32_t kv_max2(uint32_t a, uint32_t b, int dt) {
  uint32_t r;
  if (dt == GEMV_DTYPE_F16)
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Bytes of ones for the ones among the four lowest bits.
__device__ __forceinline__ uint32_t kv_bytes(uint32_t b) { return (((b & 15u) * 0x00204081u) & 0x01010101u) * 255u; }
__device__ __forceinline__ uint32_t kv_transpose(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float kv_exp2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ uint32_t kv_pack_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int D, int NT>
struct KvForm {
  // warps x slots x slot bytes of copies in flight or in use: 144 to 216 KB; an odd number
  // of slots, so that each freed one takes the other half of a block.  Twelve warps where
  // 168 registers do (us, 12 / 8 warps, 64 channels, 30 sequences of up to 8000 tokens:
  // one tile 32.5 / 33.3, two 36.1 / 39.2; three tiles would spill).
  static constexpr int kWarps = D == 64 && NT <= 2 ? 12 : D <= 128 ? 8 : D == 192 ? 6 : 4;
  static constexpr int kSlots = D == 64 && NT > 2 ? 5 : 3;
  static constexpr int kSlot = kKvBlock * D;  // the keys or the values of a block
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kSmem = 128 + kWarps * kSlots * kSlot;
};
// floats of a partial result: rows x (D sums, then largest logits, then sums of weights;
// a whole number of 16 bytes)
template <int D, int NT>
__host__ __device__ constexpr int64_t kv_part() { return (int64_t)NT * 8 * (D + 4); }

// The weights leave exp2 times 2^14, so that fp16 holds those down to 2^-28 of the
// largest in full.  The sums of weights keep that factor, the values' scales take it
// back: weighted values then overflow fp32 only where their sum, relative to the largest
// weight, does.
constexpr float kKvLift = 14.f, kKvLifted = 16384.f;
__device__ __forceinline__ float kv_lse(float m, float den) {
  return den == 0.f ? -INFINITY : (m - kKvLift + log2f(den)) * 0.693147180559945f;
}
// Row of out (and of lse) of an item's query row.
__device__ __forceinline__ int64_t kv_out_row(const KvArgs &a, int s, int h, int row) {
  const int t = row / a.group;
  return ((int64_t)s * a.T + t) * ((int64_t)a.heads * a.group) + (int64_t)h * a.group + (row - t * a.group);
}

// Each warp works through its own range of blocks.  It has a ring of slots in shared
// memory: lane 0 has the copy engine bring each block's keys, then its values (one
// contiguous piece each), as soon as a slot is free, and a slot's mbarrier says that the
// piece is there.  For a block of 64 tokens and NT tiles of eight query rows (the rows of
// all queries of the item's head):
//   logits^T (tokens x rows) = K Q^T, four m16n8k16 tiles of 16 tokens.  A lane's 16-byte
//     piece of a key row is four instructions' worth of its columns: k is a summation
//     index, so any order will do that Q's registers follow.
//   weights in fp32 with the running maximum and sum of each row, rounded to fp16 (11
//     bits, against the 4 of the values they meet), transposed in registers (movmatrix)
//     to the operand of
//   O^T (channels x rows) += V^T weights, the tokens again in the order of a lane's
//     16-byte piece of a value row.  Which tokens a logit tile holds is chosen so that
//     the transposed weights come out in that order.
// The scales join outside: the keys' in the logits' factor, the values' when a block's
// product is added to the running sums.
// At the end of an item (or of the range) the warp writes the output, or a partial
// result that k_kv8_join adds up.
// Decode is bound by the cache's bytes: 64 sequences of up to 8192 tokens (537 MB) 94 us,
// 5.7 TB/s with the join; one of 131072 tokens 51.5 us.  mma.sync at a sixth of its rate is
// enough for that, and takes eight rows where tcgen05 would take 128.  More rows a block
// (16 with 128 channels: 38 us where the bytes take 18) are bound by the latency of eight
// warps' dependent instructions; their registers allow no more.
// kOwn: only the blocks that a sequence does not share with its group (gemv_kv8_prefix_attention);
// every result is a part then, in the place of its warp's number plus its item's, both of which
// only rise along the work list.
template <int D, int NT, bool kWhole, bool kOwn = false>
__global__ void __launch_bounds__(KvForm<D, NT>::kThreads, 1) k_kv8_attention(const KvArgs a) {
  static_assert(!(kWhole && kOwn));
  using F = KvForm<D, NT>;
  constexpr int W = F::kWarps, R = F::kSlots, Q = D / 64, DT = D / 16;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[W * R];
  __shared__ float meta[W * R][2];  // of the slot's block: the keys' and the values' scale
  __shared__ int meta_bad[W * R];
  __shared__ int abort_flag;
  // (kOwn: the kernel before is k_kv8_prefix, which writes nothing that this one reads and lets it
  // start after its own wait: an SM that is done there begins here.  The wait at the end is for
  // the join, which needs both.)
  if constexpr (!kOwn) pdl_wait();
  pdl_trigger();  // after the wait: the join reads lens before its own
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  unsigned char *smem = smem_raw + ((128u - (tc_smem_u32(smem_raw) & 127u)) & 127u);
  unsigned char *ring = smem + (size_t)warp * R * F::kSlot;
  uint64_t *bar = bars + warp * R;
  if (lane == 0)
    for (int i = 0; i < R; ++i) tc_mbar_init(&bar[i], 2);  // the piece, and with keys the block's scales
  if (tid == 0) abort_flag = 0;
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncthreads();

  const int items = a.heads * a.row_tiles;
  const int64_t worker = (int64_t)warp * gridDim.x + blockIdx.x, workers = (int64_t)gridDim.x * W;  // (few blocks: one for each SM)
  KvShares shares;
  KvItem<kOwn> at;
  int64_t u_lo, u_hi;
  // (kOwn: with the search for its group a sequence takes several reads one after the other, so each
  // warp has a part of them: 8192 sequences in 1024 groups 670 -> 116 us)
  __shared__ int64_t sums[kOwn ? W : 1];
  const int part_s = kOwn ? (a.S - 1) / (32 * W) * 32 + 32 : 0;
  if constexpr (kOwn) {
    const int64_t from = (int64_t)warp * part_s, to = from + part_s;
    const int64_t n = kv_between<true>(a, (int)(from < a.S ? from : a.S), (int)(to < a.S ? to : a.S), lane);
    if (lane == 0) sums[warp] = n;
    __syncthreads();
  }
  int slot = 0, issued = 0, taken = 0;  // the ring: slot in use, pieces begun, pieces used
  uint32_t phase = 0;
  bool dead = false;
  // by shares: one round; else (kWhole, short sequences) an item, whole, each round
  for (int64_t round = worker; !dead && (kWhole ? round < (int64_t)a.S * items : round == worker); round += workers) {
    if constexpr (kWhole) {
      const int s = (int)kv_div(round, items);
      at.load(a, s, 0);
      at.item = (int)(round - (int64_t)s * items);
      u_lo = at.lo;
      u_hi = at.hi;
      if (u_lo >= u_hi) {  // no tokens
        const int h = at.item / a.row_tiles, row0 = (at.item - h * a.row_tiles) * NT * 8;
        for (int r = 0; r < NT * 8 && row0 + r < a.T * a.group; ++r) {
          const int64_t at_row = kv_out_row(a, s, h, row0 + r);
          for (int d = lane; d < D; d += 32) reinterpret_cast<unsigned short *>(a.out)[at_row * D + d] = 0;
          if (lane == 0 && a.lse != nullptr) a.lse[at_row] = -INFINITY;
        }
        continue;
      }
    } else {
      int64_t total = 0;
      if constexpr (kOwn) {
        for (int w = 0; w < W; ++w) total += sums[w];
      } else {
        total = kv_between<false>(a, 0, a.S, lane);
      }
      shares.cut(total * items, workers);
      u_lo = shares.first(worker);
      u_hi = shares.first(worker + 1);
      if (u_lo >= u_hi) break;

      // the item of place u_lo
      int64_t base = 0;
      int s0 = 0;
      if constexpr (kOwn) {
        for (int w = 0; base + sums[w] * items <= u_lo; ++w) {
          base += sums[w] * items;
          s0 += part_s;
        }
      }
      for (;; s0 += 32) {  // 32 sequences at a time
        const int s = s0 + lane;
        unsigned n = s < a.S ? (unsigned)kv_places(kv_seen<kOwn>(a, s)) : 0u;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const unsigned o = __shfl_up_sync(0xffffffffu, n, d);
          if (lane >= d) n += o;
        }
        const unsigned past = __ballot_sync(0xffffffffu, base + (int64_t)n * items > u_lo);
        if (past != 0) {
          const int f = __ffs(past) - 1;
          const unsigned before = __shfl_sync(0xffffffffu, n, f > 0 ? f - 1 : 0);
          at.load(a, s0 + f, base + (f > 0 ? (int64_t)before * items : 0));
          at.skip(kv_div(u_lo - (at.lo - kKvItemCost), kv_places(at.seen)));
          break;
        }
        base += (int64_t)__shfl_sync(0xffffffffu, n, 31) * items;
      }
    }

    // An item's queries as stored: rows g of its tiles, 16 channels 16 c .. of each 64.  The
    // first item's are on their way before the blocks are: behind those they would wait.
    const bool q_vec = (reinterpret_cast<uintptr_t>(a.q) & 15) == 0 && a.q_stride % 8 == 0;
    constexpr bool kEarly = NT * DT <= 16;  // (more would not stay in registers)
    uint32_t raw[NT][DT][2];
    auto load_q = [&](const KvItem<kOwn> &it) {
      const int h = it.item / a.row_tiles, row0 = (it.item - h * a.row_tiles) * NT * 8;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int row = row0 + n * 8 + g, t = row / a.group;
        const unsigned short *qp = reinterpret_cast<const unsigned short *>(a.q) + ((int64_t)it.s * a.T + t) * a.q_stride +
                                   ((int64_t)h * a.group + row - t * a.group) * D + 16 * c;
#pragma unroll
        for (int i = 0; i < DT; ++i) raw[n][i][0] = raw[n][i][1] = 0;
        if (row < a.T * a.group) {
          if (q_vec) {
#pragma unroll
            for (int i = 0; i < DT; i += 2) {
              const uint4 v = __ldg(reinterpret_cast<const uint4 *>(qp + (i >> 2) * 64 + (i & 3) * 4));
              raw[n][i][0] = v.x;
              raw[n][i][1] = v.y;
              raw[n][i + 1][0] = v.z;
              raw[n][i + 1][1] = v.w;
            }
          } else {
#pragma unroll
            for (int i = 0; i < DT; ++i) {
              const uint2 v = kv_load4(qp + (i >> 2) * 64 + (i & 3) * 4);
              raw[n][i][0] = v.x;
              raw[n][i][1] = v.y;
            }
          }
        }
      }
    };

    // ---- copies: the pieces of this warp's blocks
    KvItem<kOwn> is = at;                          // the item of place `iu`
    int64_t iu = u_lo > at.lo ? u_lo : at.lo;
    int batch = -1;                          // first of the item's blocks whose table entries the lanes hold
    int32_t entries = 0;
    auto look = [&](int j) {
      batch = j;
      const int i = j + lane;
      entries = -1;
      if (i < is.seen.count)
        entries = __ldg(a.table + (int64_t)is.s * a.width + (i < is.seen.sink ? i : is.seen.from + i - is.seen.sink));
    };
    // the next block: its number in the pool x heads + head; -1: none is left, -2 - head:
    // the table's entry is none of the pool
    auto advance = [&]() -> int64_t {
      if (iu >= u_hi) return -1;
      const int j = (int)(iu - is.lo), h = is.item / a.row_tiles;
      if (batch < 0 || j >= batch + 32) look(j);
      const int32_t entry = __shfl_sync(0xffffffffu, entries, j - batch);
      if (++iu == is.hi) {
        if (iu + kKvItemCost < u_hi) {
          is.seek(a, iu);
          iu = is.lo;
          batch = -1;
        } else {
          iu = u_hi;
        }
      }
      return entry >= 0 && entry < a.blocks ? (int64_t)entry * a.heads + h : -2 - (int64_t)h;
    };
    auto issue = [&](int64_t block, bool keys, int to) {
      if (block == -1) return;
      if (lane == 0) {
        const bool good = block >= 0;
        const int64_t at_block = good ? block : -2 - block;  // (of an entry that is no block: any, unseen)
        uint64_t *b = &bar[to];
        if (keys) {
          meta_bad[warp * R + to] = !good;
          if (!good && a.status != nullptr) atomicOr(a.status, kKvStatusTable);
          f8_copy4(&meta[warp * R + to][0], a.k_scale + at_block, true);
          f8_copy4(&meta[warp * R + to][1], a.v_scale + at_block, true);
          f8_copy4_arrive(b);
        } else {
          tc_mbar_arrive(b);
        }
        if (!a.test_stall || keys) {  // test: no values ever come
          tc_mbar_arrive_expect_tx(b, F::kSlot);
          kv_bulk(ring + (size_t)to * F::kSlot, (keys ? a.k : a.v) + at_block * F::kSlot, F::kSlot, b);
        }
      }
      ++issued;
    };
    if (iu < u_hi) {
      look((int)(iu - is.lo));
      if constexpr (kEarly) load_q(at);
    }
    // While block n's keys are used, the ring holds its values and the R - 2 pieces after
    // them; the slot of the keys takes the values of block n + R / 2 (`ahead`), that of its
    // values the keys of the block after that.
    static_assert(R % 2 == 1);
    int64_t ahead;
    {
      ahead = advance();
      int to = slot;
      auto next = [&]() { return to = to + 1 == R ? 0 : to + 1; };
#pragma unroll 1
      for (int i = 0; i + 1 < R; i += 2) {
        issue(ahead, true, to);
        issue(ahead, false, next());
        next();
        if (ahead != -1) ahead = advance();
      }
      issue(ahead, true, to);
    }

    auto arrived = [&]() {
      const bool ok = f8_wait(&bar[slot], phase, a.timeout_ns, &abort_flag);
      dead = !__all_sync(0xffffffffu, ok);
      return !dead;
    };
    auto release = [&](bool keys) {
      __syncwarp();  // every lane has read the slot
      if (!keys && ahead != -1) ahead = advance();
      issue(ahead, !keys, slot);
      ++taken;
      if (++slot == R) {
        slot = 0;
        phase ^= 1;
      }
    };

    bool first_item = true;
    int64_t u = u_lo > at.lo ? u_lo : at.lo;
    while (u < u_hi) {
      const int64_t seg = u, seg_end = at.hi < u_hi ? at.hi : u_hi;
      const int h = at.item / a.row_tiles, row0 = (at.item - h * a.row_tiles) * NT * 8;
      const int rows = a.T * a.group - row0;  // of this tile, at most NT * 8
      const int len = at.seen.len;

      // Q's registers: row g of each tile, in the order of the key pieces.  Each row is
      // scaled by a power of two so that its largest value lies in [2^14, 2^15): fp16
      // then holds what is within 2^-28 of it as the input does.
      uint32_t qf[NT][DT][2];
      float qs[NT][2];  // factor of the logits of rows 2 c, 2 c + 1: softmax scale x log2 e / that power
      if (!kEarly || !first_item) load_q(at);
      {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          // (an infinity takes the largest exponent: the row's result is NaN, or 0, with it)
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) top = kv_max2(top, raw[n][i][e] & 0x7fff7fffu, a.dtype);
          float mx = fmaxf(kv_wide_lo(top, a.dtype), kv_wide_hi(top, a.dtype));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          int e = (__float_as_int(mx) >> 23) & 0xff;  // exponent field, 127 for [1, 2)
          e = e < 16 ? 16 : e;
          const float up = __int_as_float((127 + 14 + 127 - e) << 23);
#pragma unroll
          for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              qf[n][i][k] = kv_pack_half(kv_wide_lo(raw[n][i][k], a.dtype) * up, kv_wide_hi(raw[n][i][k], a.dtype) * up);
          const float f = a.scale_log2 / up;
          qs[n][0] = __shfl_sync(0xffffffffu, f, 8 * c);
          qs[n][1] = __shfl_sync(0xffffffffu, f, 8 * c + 4);
        }
      }

      float o[NT][DT][4], m[NT][2], l[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
      }

      for (; u < seg_end; ++u) {
        const int j = (int)(u - at.lo);
        const int64_t pos0 = (int64_t)(j < at.seen.sink ? j : at.seen.from + j - at.seen.sink) * kKvBlock;
        if (!arrived()) break;
        const float ks = meta[warp * R + slot][0];
        const bool bad = meta_bad[warp * R + slot] != 0;  // no such block: nothing of it is seen
        const float vs = bad ? 0.f : meta[warp * R + slot][1] * (1.f / kKvLifted);
        // does every query see every token of the block?
        const bool edge = bad || pos0 + kKvBlock - 1 > (int64_t)len - a.T ||
                          (a.window > 0 && len - 1 - pos0 >= a.window && pos0 + kKvBlock > a.sinks);
        // bit `tok`: query t sees that token of the block
        auto mask = [&](int t) {
          const int64_t i = (int64_t)len - a.T + t - pos0;  // the query's position, from the block's start
          uint64_t w = kv_low_bits(i + 1);
          if (a.window > 0) w &= ~kv_low_bits(i + 1 - a.window) | kv_low_bits(a.sinks - pos0);
          return bad ? 0ull : w;
        };

        // ---- logits: tile j holds tokens 16 (r / 2) + 4 j + r % 2 (rows r = 0..7 of the
        // tile) and those + 2 (rows 8..15)
        float s[NT][4][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][t][e] = 0.f;
        const unsigned char *kp = ring + (size_t)slot * F::kSlot + (16 * (g >> 1) + (g & 1)) * D + 16 * c;
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint4 x = *reinterpret_cast<const uint4 *>(kp + (4 * t) * D + 64 * q);
            const uint4 y = *reinterpret_cast<const uint4 *>(kp + (4 * t + 2) * D + 64 * q);
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t f[4] = {kv_half2_lo(xw[i]), kv_half2_lo(yw[i]), kv_half2_hi(xw[i]), kv_half2_hi(yw[i])};
#pragma unroll
              for (int n = 0; n < NT; ++n) kv_mma(s[n][t], f, qf[n][q * 4 + i][0], qf[n][q * 4 + i][1]);
            }
          }
        release(true);

        // ---- weights
        uint32_t p[NT][4][2];
        float keep[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float f0 = qs[n][0] * ks, f1 = qs[n][1] * ks;
          float m0 = m[n][0], m1 = m[n][1];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            s[n][t][0] *= f0;
            s[n][t][1] *= f1;
            s[n][t][2] *= f0;
            s[n][t][3] *= f1;
          }
          if (edge) {
            // the tokens that the queries of rows 2 c, 2 c + 1 see, from this lane's first on
            const int r0 = row0 + n * 8 + 2 * c, first = 16 * (g >> 1) + (g & 1);
            const uint32_t wa = (uint32_t)(mask(r0 / a.group) >> first), wb = (uint32_t)(mask((r0 + 1) / a.group) >> first);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              if (!(wa >> (4 * t) & 1)) s[n][t][0] = -INFINITY;
              if (!(wb >> (4 * t) & 1)) s[n][t][1] = -INFINITY;
              if (!(wa >> (4 * t + 2) & 1)) s[n][t][2] = -INFINITY;
              if (!(wb >> (4 * t + 2) & 1)) s[n][t][3] = -INFINITY;
            }
          }
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            m0 = fmaxf(m0, fmaxf(s[n][t][0], s[n][t][2]));
            m1 = fmaxf(m1, fmaxf(s[n][t][1], s[n][t][3]));
          }
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, d));
            m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, d));
          }
          // a row that has seen nothing yet: any finite reference leaves its weights 0
          const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
          keep[n][0] = kv_exp2(m[n][0] - z0);
          keep[n][1] = kv_exp2(m[n][1] - z1);
          m[n][0] = m0;
          m[n][1] = m1;
          float l0 = 0.f, l1 = 0.f;
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const float w0 = kv_exp2(s[n][t][0] - z0 + kKvLift), w1 = kv_exp2(s[n][t][1] - z1 + kKvLift);
            const float w2 = kv_exp2(s[n][t][2] - z0 + kKvLift), w3 = kv_exp2(s[n][t][3] - z1 + kKvLift);
            l0 += w0 + w2;
            l1 += w1 + w3;
            p[n][t][0] = kv_transpose(kv_pack_half(w0, w1));
            p[n][t][1] = kv_transpose(kv_pack_half(w2, w3));
          }
          // (this lane's tokens; the lanes' sums meet at the end)
          l[n][0] = l[n][0] * keep[n][0] + l0;
          l[n][1] = l[n][1] * keep[n][1] + l1;
        }

        // ---- sums
        // Values that no query of the tile sees may be anything, NaN among it: they count as
        // 0.  So do, to a query, those that only others see: their weights are 0; unless
        // they are NaN, then its product leaves them out.
        uint32_t keep4[4] = {~0u, ~0u, ~0u, ~0u};  // the bytes that count, tile t of tokens
        bool mixed = false;                        // some queries see what others do not
        if (edge) {
          const int t_lo = row0 / a.group, t_hi = (row0 + (rows < NT * 8 ? rows : NT * 8) - 1) / a.group;
          uint64_t some = 0, all = ~0ull;
          for (int q = t_lo; q <= t_hi; ++q) {
            some |= mask(q);
            all &= mask(q);
          }
#pragma unroll
          for (int t = 0; t < 4; ++t) keep4[t] = kv_bytes((uint32_t)(some >> (16 * c + 4 * t)));
          mixed = some != all;
        }
        if (!arrived()) break;
        const unsigned char *vp = ring + (size_t)slot * F::kSlot + g * kKvBlock + 16 * c;
        // channels 16 k ..: V^T's registers, tile t of tokens
        auto load_v = [&](int k, uint32_t (&f)[4][4]) {
          const uint4 x = *reinterpret_cast<const uint4 *>(vp + k * 16 * kKvBlock);
          const uint4 y = *reinterpret_cast<const uint4 *>(vp + (k * 16 + 8) * kKvBlock);
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint32_t xm = xw[t] & keep4[t], ym = yw[t] & keep4[t];
            f[t][0] = kv_half2_lo(xm);
            f[t][1] = kv_half2_lo(ym);
            f[t][2] = kv_half2_hi(xm);
            f[t][3] = kv_half2_hi(ym);
          }
        };
        bool nan = false;
        if (mixed) {
#pragma unroll 1
          for (int k = 0; k < 2 * DT; ++k) {
            const uint4 x = *reinterpret_cast<const uint4 *>(vp + k * 8 * kKvBlock);
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int t = 0; t < 4; ++t) nan |= __vcmpeq4(xw[t] & keep4[t] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
          }
          nan = __any_sync(0xffffffffu, nan);
        }
        if (!nan) {
#pragma unroll
          for (int k = 0; k < DT; ++k) {
            uint32_t f[4][4];
            load_v(k, f);
            // two row tiles' products by turns, each a chain of four (us, by turns / one after the
            // other: 16 rows of 192 channels 40.1 / 42.4, of 128 42.7 / 43.3, of 64 27.2 / 27.7;
            // three tiles, short of registers, 30.2 / 29.9)
            constexpr int kTurns = NT == 2 ? 2 : 1;
#pragma unroll
            for (int n0 = 0; n0 < NT; n0 += kTurns) {
              float d[kTurns][4] = {};
#pragma unroll
              for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int n = 0; n < kTurns; ++n) kv_mma(d[n], f[t], p[n0 + n][t][0], p[n0 + n][t][1]);
#pragma unroll
              for (int n = 0; n < kTurns; ++n) {
                float(&acc)[4] = o[n0 + n][k];
                const float(&by)[2] = keep[n0 + n];
                acc[0] = fmaf(vs, d[n][0], acc[0] * by[0]);
                acc[1] = fmaf(vs, d[n][1], acc[1] * by[1]);
                acc[2] = fmaf(vs, d[n][2], acc[2] * by[0]);
                acc[3] = fmaf(vs, d[n][3], acc[3] * by[1]);
              }
            }
          }
        } else {
          // for each query of a tile of rows the product with the values that it sees,
          // for its rows only
          const uint32_t any4[4] = {keep4[0], keep4[1], keep4[2], keep4[3]};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int r_lo = row0 + n * 8, r_hi = r_lo + 7 < a.T * a.group - 1 ? r_lo + 7 : a.T * a.group - 1;
            const int ta = (r_lo + 2 * c) / a.group, tb = (r_lo + 2 * c + 1) / a.group;
#pragma unroll
            for (int k = 0; k < DT; ++k)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[n][k][e] *= keep[n][e & 1];
#pragma unroll 1
            for (int t1 = r_lo / a.group; t1 <= r_hi / a.group; ++t1) {
              const uint64_t w = mask(t1);
#pragma unroll
              for (int t = 0; t < 4; ++t) keep4[t] = kv_bytes((uint32_t)(w >> (16 * c + 4 * t)));
#pragma unroll
              for (int k = 0; k < DT; ++k) {
                uint32_t f[4][4];
                load_v(k, f);
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                float(&acc)[4] = o[n][k];
#pragma unroll
                for (int t = 0; t < 4; ++t) kv_mma(d, f[t], p[n][t][0], p[n][t][1]);
                if (ta == t1) {
                  acc[0] = fmaf(vs, d[0], acc[0]);
                  acc[2] = fmaf(vs, d[2], acc[2]);
                }
                if (tb == t1) {
                  acc[1] = fmaf(vs, d[1], acc[1]);
                  acc[3] = fmaf(vs, d[3], acc[3]);
                }
              }
            }
          }
#pragma unroll
          for (int t = 0; t < 4; ++t) keep4[t] = any4[t];
        }
        release(false);
      }

      if (dead) break;

      // ---- the item's output, or this range's part of it
      const bool whole = !kOwn && (kWhole || (seg == at.lo && seg_end == at.hi));
      if (!kWhole && seg == at.lo && lane == 0)  // the item's first blocks: where its parts are
        a.parts[(int64_t)at.s * items + at.item] =
            make_int4((int)worker, (int)(shares.owner(at.hi - 1) - worker) + 1, first_item ? 0 : 1, 0);
      const int64_t place = kOwn ? worker + (int64_t)at.s * items + at.item : worker * 2 + (first_item ? 0 : 1);
      float *part = a.ws + place * kv_part<D, NT>();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float den = l[n][e];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) den += __shfl_xor_sync(0xffffffffu, den, d);
          const int r = n * 8 + 2 * c + e;
          if (r >= rows) continue;
          if (whole) {
            const int64_t at_row = kv_out_row(a, at.s, h, row0 + r);
            unsigned short *out = reinterpret_cast<unsigned short *>(a.out) + at_row * D + g;
            const float inv = den == 0.f ? 0.f : kKvLifted * (1.f / den);
#pragma unroll
            for (int i = 0; i < DT; ++i) {
              out[16 * i] = f8_round16(o[n][i][e] * inv, a.dtype);
              out[16 * i + 8] = f8_round16(o[n][i][e + 2] * inv, a.dtype);
            }
            if (g == 0 && a.lse != nullptr) a.lse[at_row] = kv_lse(m[n][e], den);
          } else {
#pragma unroll
            for (int i = 0; i < DT; ++i) {
              part[r * D + 16 * i + g] = o[n][i][e];
              part[r * D + 16 * i + 8 + g] = o[n][i][e + 2];
            }
            if (g == 0) {
              part[NT * 8 * D + r] = m[n][e];
              part[NT * 8 * (D + 1) + r] = den;
            }
          }
        }
      }
      first_item = false;
      if (u >= u_hi) break;
      at.seek(a, u);
      u = at.lo;
    }
  }  // rounds
  if (dead) {
    // no copy may be in flight when the CTA exits
    if (lane == 0) {
      if (a.status != nullptr) atomicOr(a.status, kTcStatusMma);
      bool drained = true;
      for (; taken < issued; ++taken) {
        if (!tc_mbar_wait(&bar[slot], phase, a.timeout_ns)) drained = false;
        if (++slot == R) {
          slot = 0;
          phase ^= 1;
        }
      }
      if (!drained && a.status != nullptr) atomicOr(a.status, kTcStatusDrain);
    }
  }
  if constexpr (kOwn) pdl_wait();
}

// Items that several warps of k_kv8_attention share: their partial results, merged in the
// order of the blocks; and the outputs of sequences without tokens: zeros.  A thread adds
// up four channels of a row, eight parts on their way at a time; kGroups threads share the
// parts of the same channels, where there are few items, each perhaps in a hundred parts.
// grid (S, items, pieces of a tile's rows).  Three dependent reads: 2 to 6 us after the
// attention kernel.  Three CTAs an SM (us, with registers for three / two: 64 sequences of up
// to 4000 tokens, 8 heads of 64, 512 CTAs 33.0 / 34.4).
constexpr int kKvJoinThreads = 256;
struct KvSum {  // a row's (part of a) softmax: largest logit, sum of weights, weighted values
  float m = -INFINITY, den = 0.f;
  float4 v = {0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ void add(float fm, float fden, const float4 &f) {
    const float big = fmaxf(m, fm), z = big == -INFINITY ? 0.f : big;
    const float x = kv_exp2(m - z), y = kv_exp2(fm - z);
    m = big;
    den = den * x + fden * y;
    v.x = v.x * x + f.x * y;
    v.y = v.y * x + f.y * y;
    v.z = v.z * x + f.z * y;
    v.w = v.w * x + f.w * y;
  }
};
template <int D, int NT, int kGroups>
__global__ void __launch_bounds__(kKvJoinThreads, 3) k_kv8_join(const KvArgs a) {
  constexpr int kAlong = kKvJoinThreads / kGroups;  // threads along the channels
  constexpr int64_t kPart = kv_part<D, NT>();
  __shared__ KvSum sums[kGroups > 1 ? kGroups : 1][kGroups > 1 ? kAlong : 1];
  pdl_trigger();
  const int s = blockIdx.x, item = blockIdx.y, items = a.heads * a.row_tiles;
  // (lens is older than the attention kernel, which let this one start after its own wait)
  const int count = kv_seen(a, s).count;
  pdl_wait();  // by every CTA: the next kernel counts on it
  const int4 of = count > 0 ? __ldcg(&a.parts[(int64_t)s * items + item]) : make_int4(0, 0, 0, 0);
  // A warp whose wait ran out leaves its items' entries as the scratch memory had them: any
  // bits.  The call's outputs are undefined then; what is read stays within the partial results.
  if (of.x < 0 || of.y < 0 || (int64_t)of.x + of.y > a.workers || (of.z & ~1) != 0) return;
  if (of.y == 1) return;  // one warp had the whole item and wrote it
  const int h = item / a.row_tiles, row0 = (item - h * a.row_tiles) * NT * 8;
  const int rows = a.T * a.group - row0 < NT * 8 ? a.T * a.group - row0 : NT * 8;
  const int along = threadIdx.x % kAlong, grp = threadIdx.x / kAlong;
  const int e = (blockIdx.z * kAlong + along) * 4, r = e / D, d = e - r * D;
  KvSum sum;
  if (r < rows) {
    const float *const p = a.ws + (int64_t)of.x * 2 * kPart;
    for (int i0 = grp; i0 < of.y; i0 += 8 * kGroups) {
      float m[8], den[8];
      float4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = i0 + k * kGroups;
        if (i < of.y) {
          const float *q = p + (i == 0 ? of.z * kPart : i * 2 * kPart);
          m[k] = __ldcg(q + NT * 8 * D + r);
          den[k] = __ldcg(q + NT * 8 * (D + 1) + r);
          v[k] = __ldcg(reinterpret_cast<const float4 *>(q + e));
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (i0 + k * kGroups < of.y) sum.add(m[k], den[k], v[k]);
    }
  }
  if constexpr (kGroups > 1) {
    sums[grp][along] = sum;
    __syncthreads();
    constexpr int kLast = kGroups < 8 ? kGroups : 8;
    auto add = [&](int k) { sum.add(sums[k][along].m, sums[k][along].den, sums[k][along].v); };
    if constexpr (kGroups > kLast) {  // to eight sums first
      if (grp < kLast) {
#pragma unroll
        for (int k = kLast; k < kGroups; k += kLast) add(grp + k);
        sums[grp][along] = sum;
      }
      __syncthreads();
    }
    if (grp > 0) return;
#pragma unroll
    for (int k = 1; k < kLast; ++k) add(k);
  }
  if (r >= rows) return;
  const int64_t at_row = kv_out_row(a, s, h, row0 + r);
  unsigned short *out = reinterpret_cast<unsigned short *>(a.out) + at_row * D + d;
  const float inv = sum.den == 0.f ? 0.f : kKvLifted * (1.f / sum.den), v[4] = {sum.v.x, sum.v.y, sum.v.z, sum.v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) out[j] = f8_round16(v[j] * inv, a.dtype);
  if (d == 0 && a.lse != nullptr) a.lse[at_row] = kv_lse(sum.m, sum.den);
}

}  // namespace gemv
