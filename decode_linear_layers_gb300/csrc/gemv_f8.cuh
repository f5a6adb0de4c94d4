// Kernels of the block-scaled 8-bit floating point product (gemv_f8) and of the
// quantiser of its vectors (gemv_f8_quantize).
//
//     y[b][m] = sum_g sa[m / 128][g] sx[b][g] P_g[b][m] + bias[m],
//     P_g[b][m] = sum_{k in group g} A[m][k] x[b][k]
//
// A and x hold e4m3 values; g runs over the groups of 128 columns.  The tensor cores
// (tcgen05 kind::f8f6f4) compute P_g, a tile of 128 x N values for each k-block of 128
// columns, into one of a few accumulators in tensor memory.  The scales are fp32 numbers,
// not powers of two alone, so P_g cannot stay there: the scaling warps read it
// (tcgen05.ld), and add (sa sx) P_g to the tile's fp32 sums in their registers, while the
// next k-blocks' products fill the other accumulators.  sa sx is formed first and has to
// be 0 or a normal number: a test of it for each k-block, with P_g taking one scale after
// the other where it is not, costs 2 to 5 % (us, tested / not: 6144x4096 B=1 8.2 / 7.8,
// 28672x4096 B=16 23.4 / 22.9, 4096x14336 B=8192 388 / 381), for sums of 1e-31 or 1e38.
#pragma once

#include "../../include/gemv.h"
#include "gemv_tc.cuh"

namespace gemv {

constexpr int kF8Group = 128;    // columns per scale, and per k-block: one 128-byte swizzle atom
constexpr int kF8Rows = 128;     // rows of a tile: the MMA's M
constexpr int kF8RoleThreads = 128;  // warps 0 (copies), 1 (MMAs) and 2 (scales), one idle
constexpr int kF8MaxStages = 12;

struct F8Args {
  const float *a_scale = nullptr, *x_scale = nullptr;
  const void *bias = nullptr;
  void *y = nullptr;
  float *ws = nullptr;   // partial sums of tiles that several CTAs share
  int *status = nullptr;
  int64_t timeout_ns = 0, M = 0;
  int64_t tiles = 0;     // row tiles x column tiles
  int64_t shared = 0;    // tiles 0 .. shared - 1 are split, the rest go whole
  int B = 0, groups = 0; // groups = k-blocks
  int sharers = 0;       // CTAs that the shared tiles are split over
  int slices = 1;        // or: CTAs of the cluster that each of them is split over
  int tm = 0, tn = 0;    // tiles along the weight rows and along the vectors
  int y_dtype = 0, test_stall = 0;
};

// A bounded wait of one of several cooperating threads: false after timeout_ns, or once
// another has set *abort.  The timer and the flag are looked at after every 256 failed
// tries only.
__device__ __forceinline__ bool f8_wait(uint64_t *b, uint32_t parity, int64_t timeout_ns, volatile int *abort) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (tc_mbar_try_wait(b, parity)) return true;
    if ((i & 255) == 0) {
      if (*abort) return false;
      const uint64_t t = tc_global_ns();
      if (t0 == 0) t0 = t;
      if ((int64_t)(t - t0) > timeout_ns) {
        *abort = 1;
        return false;
      }
    }
  }
}

// ------------------------------------------------------------------ output types
__device__ __forceinline__ unsigned short f8_round16(float v, int dt) {
  return dt == GEMV_DTYPE_F16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
__device__ __forceinline__ float f8_bias(const F8Args &a, int64_t m) {
  if (a.y_dtype == GEMV_DTYPE_F32) return __ldg(reinterpret_cast<const float *>(a.bias) + m);
  const unsigned short h = __ldg(reinterpret_cast<const unsigned short *>(a.bias) + m);
  return a.y_dtype == GEMV_DTYPE_F16 ? __half2float(__ushort_as_half(h)) : __uint_as_float((uint32_t)h << 16);
}
__device__ __forceinline__ void f8_store(const F8Args &a, int64_t i, float v) {
  if (a.y_dtype == GEMV_DTYPE_F32)
    reinterpret_cast<float *>(a.y)[i] = v;
  else
    reinterpret_cast<unsigned short *>(a.y)[i] = f8_round16(v, a.y_dtype);
}

// ------------------------------------------------------------------ work of a CTA
// The k-blocks of the `shared` first tiles, R = shared x groups of them, are cut into
// W = `sharers` equal ranges (range w: [w R / W, (w + 1) R / W)), one for each CTA, or for
// each of the first R: so a few tiles keep every SM busy.  A range is no longer than a
// tile's k-blocks, so it meets two tiles at most.  The other tiles, a multiple of the
// CTAs, go round whole.  Each role of a CTA walks the same segments.
// Or (slices > 1) the CTAs form clusters, and each of the shared tiles is one cluster's, its
// k-blocks cut among the cluster's CTAs, which add their sums in distributed shared memory:
// one launch and no scratch buffer.  The whole tiles go first then, for the sums need the
// rings idle.
constexpr int kF8Whole = -1, kF8Sliced = -2;
struct F8Seg {
  int tile, k0, k1;
  int slot;  // which of the CTA's two partial sums it fills; or kF8Whole, kF8Sliced
};
struct F8Walk {  // (the host limits tiles, and the k-blocks of a CTA, to 32 bits)
  uint32_t lo, hi;
  int next_tile, tiles, groups, part;
  bool sliced;  // [lo, hi) is a slice of the cluster's tile
  __device__ F8Walk(const F8Args &a) {
    groups = a.groups;
    part = 0;
    const int64_t w = blockIdx.x;
    next_tile = (int)(a.shared + w);
    tiles = (int)a.tiles;
    sliced = false;
    if (a.slices > 1) {
      const uint32_t tile = blockIdx.x / a.slices, r = blockIdx.x - tile * a.slices;
      sliced = tile < a.shared;
      lo = tile * groups + r * groups / a.slices;
      hi = sliced ? tile * groups + (r + 1) * groups / a.slices : lo;
      return;
    }
    const int64_t R = a.shared * a.groups;
    lo = w < a.sharers ? (uint32_t)(w * R / a.sharers) : 0u;
    hi = w < a.sharers ? (uint32_t)((w + 1) * R / a.sharers) : 0u;
  }
  __device__ bool next(F8Seg &s) {
    if (lo < hi && !(sliced && next_tile < tiles)) {
      s.tile = (int)(lo / groups);
      s.k0 = (int)(lo - (uint32_t)s.tile * groups);
      s.k1 = hi - lo < (uint32_t)(groups - s.k0) ? s.k0 + (int)(hi - lo) : groups;
      s.slot = sliced ? kF8Sliced : s.k0 == 0 && s.k1 == groups ? kF8Whole : part;
      ++part;
      lo += s.k1 - s.k0;
      return true;
    }
    if (next_tile >= tiles) return false;
    s.tile = next_tile;
    s.k0 = 0;
    s.k1 = groups;
    s.slot = kF8Whole;
    next_tile += gridDim.x;
    return true;
  }
};
// The CTA whose range holds k-block u of the shared tiles: the last w with w R / W <= u.
__host__ __device__ inline int64_t f8_owner(int64_t u, int64_t R, int64_t W) { return ((u + 1) * W - 1) / R; }

// Tile -> (tile of weight rows, tile of vectors).  Whole bands of 16 weight tiles, their
// weights read once into L2, meet every tile of vectors before the next band.
__device__ __forceinline__ void f8_tile(const F8Args &a, int t, int &im, int &in) {
  constexpr int kBand = 16;
  const int band = t / (kBand * a.tn), r = t - band * (kBand * a.tn);
  const int w = a.tm - band * kBand < kBand ? a.tm - band * kBand : kBand;
  in = r / w;
  im = band * kBand + (r - in * w);
}

// ------------------------------------------------------------------ instructions
// kind::f8f6f4, both operands e4m3 (format 0), fp32 accumulator, both K-major; 32
// columns of k.
__device__ __forceinline__ uint32_t f8_idesc(int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kF8Rows >> 4) << 24);
}
__device__ __forceinline__ void f8_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// C accumulator columns of this warp's 32 tensor-memory lanes; the values are there
// after f8_ld_wait, which names them so that no use moves above it.
template <int C>
__device__ __forceinline__ void f8_ld(uint32_t addr, uint32_t (&r)[C]) {
  static_assert(C == 16 || C == 32);
  if constexpr (C == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
  }
}
template <int C>
__device__ __forceinline__ void f8_ld_wait(uint32_t (&r)[C]) {
  if constexpr (C == 16) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
  } else {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29])
                 :
                 : "memory");
    asm volatile("" : "+r"(r[30]), "+r"(r[31]));
  }
}

// One lane of a converged warp.  The copies and the MMAs are issued by a whole warp that
// waits together, with only these instructions under its predicate: their operands stay
// in the warp's uniform registers (issued from a branch of one lane, the four MMAs and
// two commits of a k-block took 430 to 640 cycles, more than its product).
__device__ __forceinline__ bool f8_elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// Four bytes by an asynchronous copy, zeros unless `has`; f8_copy4_arrive: the mbarrier
// gets one arrival once this thread's copies have come.
__device__ __forceinline__ void f8_copy4(void *dst, const void *src, bool has) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc_smem_u32(dst)), "l"(src), "r"(has ? 4 : 0) : "memory");
}
__device__ __forceinline__ void f8_copy4_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc_smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void f8_copy4_drain() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void f8_prefetch_map(const CUtensorMap *m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}
// Two values of a 16-bit output type, `a` in the low half.
__device__ __forceinline__ uint32_t f8_pack16(float a, float b, int dt) {
  uint32_t r;
  if (dt == GEMV_DTYPE_F16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// Four consecutive values of y's row b, from column m (a multiple of 4) on, with the bias.
// (The type is asked once: a branch for each value chains their latencies.)
__device__ __forceinline__ void f8_store_along(const F8Args &a, int64_t b, int64_t m, float4 q) {
  float v[4] = {q.x, q.y, q.z, q.w};
  const int n = a.M - m < 4 ? (int)(a.M - m) : 4;
  if (a.bias != nullptr) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += j < n ? f8_bias(a, m + j) : 0.f;
  }
  const bool f32 = a.y_dtype == GEMV_DTYPE_F32, vec = a.M % 4 == 0;
  const int64_t i = b * a.M + m;
  if (f32) {
    float *p = reinterpret_cast<float *>(a.y) + i;
    if (vec && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0) {
      *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n) p[j] = v[j];
    }
  } else {
    const uint32_t lo = f8_pack16(v[0], v[1], a.y_dtype), hi = f8_pack16(v[2], v[3], a.y_dtype);
    unsigned short *p = reinterpret_cast<unsigned short *>(a.y) + i;
    if (vec && (reinterpret_cast<uintptr_t>(a.y) & 7) == 0) {
      *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
    } else {
      p[0] = (unsigned short)lo;
      if (n > 1) p[1] = (unsigned short)(lo >> 16);
      if (n > 2) p[2] = (unsigned short)hi;
      if (n > 3) p[3] = (unsigned short)(hi >> 16);
    }
  }
}
// C values of y's column m, from row b on; bias: the column's.
template <int C>
__device__ __forceinline__ void f8_store_down(const F8Args &a, int b, int64_t m, const float *v, float bias) {
  const int64_t i = (int64_t)b * a.M + m;
  if (a.y_dtype == GEMV_DTYPE_F32) {
    float *p = reinterpret_cast<float *>(a.y) + i;
#pragma unroll
    for (int j = 0; j < C; ++j, p += a.M)
      if (b + j < a.B) *p = v[j] + bias;
  } else {
    unsigned short *p = reinterpret_cast<unsigned short *>(a.y) + i;
    uint32_t w[C / 2];
#pragma unroll
    for (int j = 0; j < C / 2; ++j) w[j] = f8_pack16(v[2 * j] + bias, v[2 * j + 1] + bias, a.y_dtype);
#pragma unroll
    for (int j = 0; j < C; ++j, p += a.M)
      if (b + j < a.B) *p = (unsigned short)(w[j / 2] >> (16 * (j & 1)));
  }
}
// (s0, s1) += (f0, f1) * (v0, v1), one packed instruction.
__device__ __forceinline__ void f8_fma2(float &s0, float &s1, float f0, float f1, uint32_t v0, uint32_t v1) {
  asm("{\n\t.reg .b64 s, f, v;\n\tmov.b64 s, {%0, %1};\n\tmov.b64 f, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\t"
      "fma.rn.f32x2 s, v, f, s;\n\tmov.b64 {%0, %1}, s;\n\t}"
      : "+f"(s0), "+f"(s1)
      : "f"(f0), "f"(f1), "r"(v0), "r"(v1));
}

// A warp's 32 vectors (from b0 on) of COLS weight rows each (from m0 on), a vector to a
// lane: bias, rounding, and out through the warp's staging buffer, 64 bytes of each vector
// at a time (16-byte pieces, their order rotated by the lane: free of bank conflicts), so
// that four lanes store 64 consecutive bytes of y.
template <int COLS>
__device__ __forceinline__ void f8_rows_out(const F8Args &a, float (&acc)[COLS], unsigned char *mine, int lane, int64_t b0, int64_t m0) {
  const bool f32 = a.y_dtype == GEMV_DTYPE_F32;
  const int esz = f32 ? 4 : 2;
  const bool vec = (a.M * esz) % 16 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
  if (a.bias != nullptr) {  // through the staging buffer, four columns a lane
    float *sb = reinterpret_cast<float *>(mine);
#pragma unroll
    for (int j = 0; j < COLS; j += 32) sb[j + lane] = m0 + j + lane < a.M ? f8_bias(a, m0 + j + lane) : 0.f;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < COLS; j += 4) {
      const float4 q = *reinterpret_cast<const float4 *>(sb + j);
      acc[j] += q.x;
      acc[j + 1] += q.y;
      acc[j + 2] += q.z;
      acc[j + 3] += q.w;
    }
    __syncwarp();
  }
  // columns c0 .. of the tile's COLS, `per` to a piece, lie staged: store them
  auto pass = [&](int64_t c0, int per) {
    if (c0 >= a.M) return;
    __syncwarp();
    if (vec) {  // M is a whole number of pieces
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int rr = it * 8 + (lane >> 2), pc = lane & 3;
        const uint4 w = *reinterpret_cast<const uint4 *>(mine + rr * 64 + ((pc ^ ((rr >> 1) & 3)) * 16));
        const int64_t b = b0 + rr, m = c0 + pc * per;
        if (b < a.B && m < a.M) *reinterpret_cast<uint4 *>(reinterpret_cast<char *>(a.y) + (b * a.M + m) * esz) = w;
      }
    } else if (f32) {  // rows that start anywhere: neighbouring lanes store neighbouring values
      const int jj = lane & 15, r0 = lane >> 4;
      uint32_t *dst = reinterpret_cast<uint32_t *>(a.y) + (b0 + r0) * a.M + c0 + jj;
      const int rows = c0 + jj < a.M ? (a.B - b0 < 32 ? (int)(a.B - b0) : 32) : 0;
#pragma unroll 8
      for (int rr = r0; rr < 32; rr += 2, dst += 2 * a.M) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(mine + rr * 64 + (((jj >> 2) ^ ((rr >> 1) & 3)) * 16) + (jj & 3) * 4);
        if (rr < rows) *dst = w;
      }
    } else {
      unsigned short *dst = reinterpret_cast<unsigned short *>(a.y) + b0 * a.M + c0 + lane;
      const int rows = c0 + lane < a.M ? (a.B - b0 < 32 ? (int)(a.B - b0) : 32) : 0;
#pragma unroll 8
      for (int rr = 0; rr < 32; ++rr, dst += a.M) {
        const unsigned short w =
            *reinterpret_cast<const unsigned short *>(mine + rr * 64 + (((lane >> 3) ^ ((rr >> 1) & 3)) * 16) + (lane & 7) * 2);
        if (rr < rows) *dst = w;
      }
    }
    __syncwarp();  // read before the next pass overwrites the buffer
  };
  unsigned char *const my_row = mine + lane * 64;
  const int turn = (lane >> 1) & 3;
  if (f32) {
#pragma unroll
    for (int h = 0; h < COLS; h += 16) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<float4 *>(my_row + ((q ^ turn) * 16)) =
            make_float4(acc[h + q * 4], acc[h + q * 4 + 1], acc[h + q * 4 + 2], acc[h + q * 4 + 3]);
      pass(m0 + h, 4);
    }
  } else {
#pragma unroll
    for (int h = 0; h < COLS; h += 32) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float *v = acc + h + q * 8;
        *reinterpret_cast<uint4 *>(my_row + ((q ^ turn) * 16)) =
            make_uint4(f8_pack16(v[0], v[1], a.y_dtype), f8_pack16(v[2], v[3], a.y_dtype),
                       f8_pack16(v[4], v[5], a.y_dtype), f8_pack16(v[6], v[7], a.y_dtype));
      }
      pass(m0 + h, 8);
    }
  }
}

// ------------------------------------------------------------------ the product
// kPrompt = false: a tile is 128 weight rows x N vectors (one tile of vectors, B <= N);
//   thread = weight row, column = vector.
// kPrompt = true: a tile is 128 vectors x N weight rows (128, or 256 in two blocks, one per
//   scaling warpgroup); thread = vector, so that its factor sa sx is one number per k-block.
// What bounds it, on a GB300: up to some hundred vectors the weights' bytes (28672x4096 with
// 16 vectors 23.4 us, 5.1 TB/s; 128256x4096 with 64 90.6 us, 6.0 TB/s) and, for small matrices,
// the start of the ring and the sum of the slices (6144x4096 with one vector 7.8 us);
// beyond, the hand-over of the accumulators between the MMA warp and the scaling warps.
template <int N, bool kPrompt>
struct F8Form {
  static constexpr int kGroupsOfWarps = N >= 64 ? 2 : 1;                     // scaling warpgroups
  static constexpr int kBlocks = kPrompt ? N / kF8Group : 1;                 // blocks of weight rows of a tile
  static constexpr bool kSplitRegs = N == 256;                               // roles give registers to the scaling warps
  static constexpr int kThreads = kF8RoleThreads + 128 * kGroupsOfWarps;
  static constexpr int kCols = N / kGroupsOfWarps;                           // columns of a thread
  // k-blocks of a stage: its copies, products and scales are handed on together, which
  // takes each role some hundred cycles a stage
  static constexpr int kAtoms = N <= 16 ? 4 : N <= 128 ? 2 : 1;
  static constexpr int kAcc = N >= 128 ? 2 : 4;                              // stages' accumulators in tensor memory
  static constexpr int kTmemCols = kAcc * kAtoms * N < 32 ? 32 : kAcc * kAtoms * N;
  static constexpr int kRowsBytes = kF8Rows * kF8Group, kColsBytes = N * kF8Group;  // a k-block's two operands
  static constexpr int kStage = kAtoms * (kRowsBytes + kColsBytes);
  // after the ring: the scales of kScales stages, and (prompts) each scaling warp's
  // output staging
  static constexpr int kScales = 8;
  static constexpr int kScaleFloats = (kPrompt ? kF8Rows : N) + 4;  // of a k-block: the vectors', then the weight blocks'
  static constexpr int kWarpBytes = kPrompt ? 32 * 64 : 0;
  static constexpr int kTail = kScales * kAtoms * kScaleFloats * 4 + 4 * kGroupsOfWarps * kWarpBytes;
  static constexpr int kStages = (226 * 1024 - kTail) / kStage < kF8MaxStages ? (226 * 1024 - kTail) / kStage : kF8MaxStages;
  static constexpr int kSmem = 1024 + kStages * kStage + kTail;
  static constexpr int64_t kPartial = (int64_t)kF8Rows * N;                  // floats of a partial sum
};

// map_p: the operand of the tile's 128 rows, map_q: that of its N columns; 8-bit, box
// 128 bytes x 128 or N rows, 128-byte swizzle, zeros outside the matrix.
template <int N, bool kPrompt>
__global__ void __launch_bounds__(F8Form<N, kPrompt>::kThreads, 1)
    k_f8(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q, const F8Args a) {
  using F = F8Form<N, kPrompt>;
  constexpr int S = F::kStages, NACC = F::kAcc, COLS = F::kCols, KA = F::kAtoms;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[S], empty[S], accf[NACC], acce[NACC], facf[F::kScales], face[F::kScales];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag, abort_of[kTcMaxSlices];
  __shared__ int sh_loaded, sh_consumed, sh_committed;  // for the drain after an abort
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char *smem = smem_raw + ((1024u - (tc_smem_u32(smem_raw) & 1023u)) & 1023u);

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      tc_mbar_init(&full[s], 1);
      tc_mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < NACC; ++b) {
      tc_mbar_init(&accf[b], 1);
      tc_mbar_init(&acce[b], 4 * F::kGroupsOfWarps);
    }
    for (int b = 0; b < F::kScales; ++b) {
      tc_mbar_init(&facf[b], 32);
      tc_mbar_init(&face[b], 4 * F::kGroupsOfWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    abort_flag = 0;
    sh_loaded = sh_consumed = sh_committed = -1;
  }
  if (tid == 32) {
    f8_prefetch_map(&map_p);
    f8_prefetch_map(&map_q);
  }
  __syncwarp();
  __syncthreads();
  pdl_wait();  // every read (TMA included) after the kernel before has finished
  // Tensor memory only now: before, the kernel before could be waiting for it.  Who does not
  // need it, the copies above all, goes ahead.
  uint32_t tmem = 0;
  if (warp == 1 || warp >= 4) {
    if (warp == 1) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_smem_u32(&tmem_slot)),
                   "r"((uint32_t)F::kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    asm volatile("bar.sync 1, %0;" ::"n"(32 + 128 * F::kGroupsOfWarps) : "memory");
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    tmem = tmem_slot;
  }
  volatile int *abort = &abort_flag;
  const int G = a.groups;
  const bool sliced = a.slices > 1 && blockIdx.x < a.shared * a.slices;  // the cluster ends with a tile of its own
  float *scales = reinterpret_cast<float *>(smem + (size_t)S * F::kStage);
  // after an abort nothing may be in flight when the CTA frees its tensor memory and exits:
  // the last committed MMAs (their commit covers all earlier ones) and every copy issued
  // but not waited for
  auto drain = [&]() {
    if (a.status != nullptr) atomicOr(a.status, kTcStatusMma);
    const int committed = sh_committed, consumed = sh_consumed, loaded = sh_loaded;
    bool drained = committed < 0 || tc_mbar_wait(&accf[committed % NACC], (uint32_t)((committed / NACC) & 1), a.timeout_ns);
    for (int t = consumed + 1; t <= loaded && drained; ++t)
      drained = tc_mbar_wait(&full[t % S], (uint32_t)((t / S) & 1), a.timeout_ns);
    if (!drained && a.status != nullptr) atomicOr(a.status, kTcStatusDrain);
  };

  if (warp < 4) {
    if constexpr (F::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    F8Walk walk(a);
    F8Seg g;
    bool ok = true;
    if (warp == 0) {  // copies
      int i = 0, s = 0;
      uint32_t ph = 1;  // the ring starts empty
      while (ok && walk.next(g)) {
        int im, in;
        f8_tile(a, g.tile, im, in);
        const int32_t p0 = kPrompt ? in * kF8Rows : im * kF8Rows, q0 = kPrompt ? im * N : in * N;
        for (int kb = g.k0; kb < g.k1; kb += KA) {
          ok = i < S || f8_wait(&empty[s], ph, a.timeout_ns, abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          unsigned char *st = smem + (size_t)s * F::kStage;
          if (f8_elect()) {
            const int n = g.k1 - kb < KA ? g.k1 - kb : KA;
            tc_mbar_arrive_expect_tx(&full[s], (uint32_t)n * (F::kRowsBytes + F::kColsBytes));
#pragma unroll
            for (int j = 0; j < KA; ++j) {
              if (j >= n) break;
              tc_tma_2d(st + j * F::kRowsBytes, &map_p, (kb + j) * kF8Group, p0, &full[s]);
              tc_tma_2d(st + KA * F::kRowsBytes + j * F::kColsBytes, &map_q, (kb + j) * kF8Group, q0, &full[s]);
            }
          }
          ++i;
          if (++s == S) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (lane == 0) sh_loaded = i - 1;
    } else if (warp == 1) {  // MMAs
      const uint32_t idesc = f8_idesc(N);
      const uint64_t dp0 = tc_smem_desc(tc_smem_u32(smem)), dq0 = dp0 + (KA * F::kRowsBytes >> 4);
      int i = 0, last = -1, consumed = -1;
      if (a.test_stall && blockIdx.x == 0) {  // test: the last stage of the first CTA never completes
        F8Walk w(a);
        while (w.next(g)) last += (g.k1 - g.k0 + KA - 1) / KA;
      }
      int s = 0, c = 0;
      uint32_t ph = 0, cph = 1;
      while (ok && walk.next(g)) {
        for (int kb = g.k0; kb < g.k1; kb += KA) {
          // (the copies are ahead as a rule: their wait is over before the accumulator's)
          ok = f8_wait(&full[s], ph, a.timeout_ns, abort) && (i < NACC || f8_wait(&acce[c], cph, a.timeout_ns, abort));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          consumed = i;
          if (a.test_stall && i == last) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          // (a descriptor's address counts 16 bytes, 32 columns are two of them)
          const uint64_t dp = dp0 + (uint64_t)(s * (F::kStage >> 4)), dq = dq0 + (uint64_t)(s * (F::kStage >> 4));
          if (f8_elect()) {
#pragma unroll
            for (int j = 0; j < KA; ++j) {
              if (kb + j >= g.k1) break;
#pragma unroll
              for (int kk = 0; kk < kF8Group / 32; ++kk)
                f8_mma(tmem + (uint32_t)((c * KA + j) * N), dp + j * (F::kRowsBytes >> 4) + 2 * kk,
                       dq + j * (F::kColsBytes >> 4) + 2 * kk, idesc, kk > 0);
            }
            tc_commit(&accf[c]);  // one commit: the scaling warps pass on that the stage is free
          }
          ++i;
          if (++s == S) {
            s = 0;
            ph ^= 1;
          }
          if (++c == NACC) {
            c = 0;
            cph ^= 1;
          }
        }
      }
      if (lane == 0) {
        sh_consumed = consumed;
        sh_committed = i - 1;
      }
    } else if (warp == 2) {  // scales, as far ahead of the products as their slots go
      constexpr int NV = kPrompt ? kF8Rows / 32 : (N + 31) / 32;
      int i = 0, t = 0;
      uint32_t ph = 1;
      while (ok && walk.next(g)) {
        int im, in;
        f8_tile(a, g.tile, im, in);
        const int64_t b0 = kPrompt ? (int64_t)in * kF8Rows : 0;     // the first vector
        const int64_t mb = (int64_t)im * F::kBlocks + lane;          // lane 0 (and 1): block of weight rows
        const bool va = lane < F::kBlocks && mb * kF8Group < a.M;
        const float *sa = a.a_scale + (va ? mb : 0) * G, *sx[NV];
        bool vx[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int64_t b = b0 + lane + 32 * v;
          vx[v] = b < a.B;
          sx[v] = a.x_scale + (vx[v] ? b : 0) * G;
        }
        for (int kb = g.k0; kb < g.k1; kb += KA) {
          ok = i < F::kScales || f8_wait(&face[t], ph, a.timeout_ns, abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          float *w = scales + t * (KA * F::kScaleFloats);
#pragma unroll
          for (int j = 0; j < KA; ++j, w += F::kScaleFloats) {
            if (kb + j >= g.k1) break;
#pragma unroll
            for (int v = 0; v < NV; ++v)
              if (kPrompt || lane + 32 * v < N) f8_copy4(w + lane + 32 * v, sx[v] + kb + j, vx[v]);
            if (lane < 2) f8_copy4(w + F::kScaleFloats - 4 + lane, sa + kb + j, va);
          }
          f8_copy4_arrive(&facf[t]);
          ++i;
          if (++t == F::kScales) {
            t = 0;
            ph ^= 1;
          }
        }
      }
      f8_copy4_drain();  // nothing in flight when the CTA exits
    }
    if (sliced) {  // (the scaling warps' meetings, below)
      __syncwarp();
      __syncthreads();
      if (tid == 0 && abort_flag != 0) drain();
      tc_cluster_sync();
      tc_cluster_sync();
    }
  } else {
    if constexpr (F::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int wq = warp & 3, wg = (warp >> 2) - 1;     // tensor-memory lanes 32 wq .. + 31
    const int row = wq * 32 + lane;                    // of the tile
    const int col0 = wg * COLS;
    unsigned char *mine = smem + (size_t)S * F::kStage + F::kScales * F::kAtoms * F::kScaleFloats * 4 + (size_t)(warp - 4) * F::kWarpBytes;
    constexpr int CH = COLS < 32 || N == 256 ? 16 : 32, P = COLS / CH, U = P < 2 ? 1 : 2;
    int c = 0, t = 0, st = 0;
    uint32_t cph = 0, tph = 0;
    F8Walk walk(a);
    F8Seg g;
    bool ok = true;
    while ((ok || sliced) && walk.next(g)) {
      int im, in;
      f8_tile(a, g.tile, im, in);
      float acc[COLS];
#pragma unroll
      for (int j = 0; j < COLS; ++j) acc[j] = 0.f;
      for (int kb = g.k0; kb < g.k1 && ok; kb += KA) {
        ok = f8_wait(&facf[t], tph, a.timeout_ns, abort) && f8_wait(&accf[c], cph, a.timeout_ns, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (warp == 4 && lane == 0) tc_mbar_arrive(&empty[st]);  // the product is done: its stage is free
        st = st + 1 == S ? 0 : st + 1;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const int n = g.k1 - kb < KA ? g.k1 - kb : KA;
#pragma unroll
        for (int ka = 0; ka < KA; ++ka) {
          if (ka >= n) break;
          const uint32_t at = tmem + ((uint32_t)(wq * 32) << 16) + (uint32_t)((c * KA + ka) * N + col0);
          // two pieces of CH columns on their way at a time
          uint32_t r[U][CH];
#pragma unroll
          for (int h = 0; h < U; ++h) f8_ld<CH>(at + h * CH, r[h]);
          const float *fs = scales + (t * KA + ka) * F::kScaleFloats;
          const float fa = fs[F::kScaleFloats - 4 + (kPrompt ? col0 / kF8Group : 0)], f = kPrompt ? fs[row] * fa : 0.f;
#pragma unroll
          for (int h0 = 0; h0 < P; h0 += U) {
#pragma unroll
            for (int h = 0; h < U; ++h) f8_ld_wait<CH>(r[h]);
            if (h0 + U >= P && ka + 1 == n) {
              asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
              __syncwarp();
              if (lane == 0) tc_mbar_arrive(&acce[c]);
            }
#pragma unroll
            for (int h = 0; h < U; ++h) {
              float *sum = acc + (h0 + h) * CH;
#pragma unroll
              for (int j = 0; j < CH; j += 4) {
                float4 q = make_float4(f, f, f, f);
                if constexpr (!kPrompt) {
                  q = *reinterpret_cast<const float4 *>(fs + col0 + (h0 + h) * CH + j);
                  q = make_float4(q.x * fa, q.y * fa, q.z * fa, q.w * fa);
                }
                f8_fma2(sum[j], sum[j + 1], q.x, q.y, r[h][j], r[h][j + 1]);
                f8_fma2(sum[j + 2], sum[j + 3], q.z, q.w, r[h][j + 2], r[h][j + 3]);
              }
              if (h0 + U + h < P) f8_ld<CH>(at + (h0 + U + h) * CH, r[h]);
            }
          }
        }
        __syncwarp();  // every lane has read the scales
        if (lane == 0) tc_mbar_arrive(&face[t]);
        if (++c == NACC) {
          c = 0;
          cph ^= 1;
        }
        if (++t == F::kScales) {
          t = 0;
          tph ^= 1;
        }
      }
      if (g.slot == kF8Sliced) {  // (reached after an abort, too: the cluster's CTAs meet here)
        // Every CTA of the cluster holds the sums of its slice.  CTA q adds up rows
        // ceil(128 q / slices) .. of the tile: all send it theirs, into its idle ring, and
        // it adds the slices in the order of the k-blocks.  [slice][group of four
        // columns][row]: a warp's rows lie side by side, so that they leave in whole lines
        // (16-byte pieces of 32 lines at a time cost two CTAs 128 x 128 sums 0.7 us more);
        // an odd number of rows against bank conflicts.
        __syncwarp();
        __syncthreads();
        const int n = a.slices, rank = (int)blockIdx.x % n, most = (kF8Rows + n - 1) / n;
        const bool aborted = abort_flag != 0;
        const int pitch = most | 1;
        float *parts = reinterpret_cast<float *>(smem);
        auto first_row = [&](int q) { return (kF8Rows * q + n - 1) / n; };
        // columns that y has
        const int cols = kPrompt ? (a.M - (int64_t)im * N < N ? (int)(a.M - (int64_t)im * N) : N) : (a.B < N ? a.B : N);
        tc_cluster_sync();  // every ring is idle
        const int to = row * n / kF8Rows;
        if (tid - kF8RoleThreads < n) tc_st_dsmem_int(&abort_of[rank], (uint32_t)(tid - kF8RoleThreads), aborted ? 1 : 0);
        if (!aborted) {
          const float *at = parts + 4 * ((rank * (N / 4) + col0 / 4) * pitch + row - first_row(to));
#pragma unroll
          for (int j = 0; j < COLS; j += 4, at += 4 * pitch)
            if (col0 + j < cols) tc_st_dsmem4(at, (uint32_t)to, acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
        }
        tc_cluster_sync();  // every slice's sums of the owned rows (and every abort flag) are here
        bool any = false;
        for (int q = 0; q < n; ++q) any |= abort_of[q] != 0;
        const int r0 = first_row(rank), rows = first_row(rank + 1) - r0;
        // neighbouring threads along y's rows: the tile's columns, four each (prompts), or its
        // rows, up to 64, 32 or 16 of them
        constexpr int kQuads = N / 4;
        const int lg = n <= 3 ? 6 : n <= 7 ? 5 : 4;
        const int items = kPrompt ? rows * kQuads : (cols + 3) / 4 << lg;
#pragma unroll 1
        for (int i = tid - kF8RoleThreads; i < items && !any; i += 128 * F::kGroupsOfWarps) {
          const int r = kPrompt ? i / kQuads : i & ((1 << lg) - 1), quad = kPrompt ? i % kQuads : i >> lg;
          if (kPrompt ? 4 * quad >= cols : r >= rows) continue;
          const float *at = parts + 4 * (quad * pitch + r);
          float4 v = *reinterpret_cast<const float4 *>(at);
#pragma unroll 1
          for (int q = 1; q < n; ++q) {
            const float4 u = *reinterpret_cast<const float4 *>(at + q * N * pitch);
            v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
          }
          if constexpr (kPrompt) {
            const int64_t b = (int64_t)in * kF8Rows + r0 + r;
            if (b < a.B) f8_store_along(a, b, (int64_t)im * N + 4 * quad, v);
          } else {
            const int64_t m = (int64_t)im * kF8Rows + r0 + r;
            const float e[4] = {v.x, v.y, v.z, v.w};
            if (m < a.M) f8_store_down<4>(a, 4 * quad, m, e, a.bias != nullptr ? f8_bias(a, m) : 0.f);
          }
        }
        break;
      }
      if (!ok) continue;
      if (g.slot >= 0) {
        // a part of the tile's k-blocks: k_f8_join adds the parts.  Prompts [row][column]
        // (four columns at a time), else [column][row]: both as the join writes y
        float *p = a.ws + ((int64_t)blockIdx.x * 2 + g.slot) * F::kPartial;
        if constexpr (kPrompt) {
#pragma unroll
          for (int j = 0; j < COLS; j += 4)
            *reinterpret_cast<float4 *>(p + row * N + col0 + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < COLS; ++j)
            if (col0 + j < a.B) p[(col0 + j) * kF8Rows + row] = acc[j];
        }
        continue;
      }
      if constexpr (!kPrompt) {
        const int64_t m = (int64_t)im * kF8Rows + row;
        if (m < a.M) {
          f8_store_down<COLS>(a, col0, m, acc, a.bias != nullptr ? f8_bias(a, m) : 0.f);
        }
      } else {
        f8_rows_out<COLS>(a, acc, mine, lane, (int64_t)in * kF8Rows + wq * 32, (int64_t)im * N + col0);
      }
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncwarp();  // the role threads rejoin their warps: the CTA barrier counts whole warps
  __syncthreads();
  if (abort_flag != 0 && !sliced) {
    if (tid == 0) drain();
    __syncwarp();
    __syncthreads();
  }
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)F::kTmemCols) : "memory");
  }
}

// ------------------------------------------------------------------ pairs of SMs
// Prompts with many tiles: a tile is 256 vectors x 256 weight rows, done by a cluster of two
// CTAs whose tensor cores work as one (cta_group::2).  Each has the 128 vectors of its own
// accumulator rows and half of the weight rows in shared memory, so that a k-block writes
// and reads 32 KB in each SM instead of 48 (those 48 KB cost 768 cycles of shared-memory
// bandwidth, the MMA itself 512).  CTA 0's MMA warp issues for both; a commit reaches both
// CTAs' barriers, and both CTAs' scaling warps hand the accumulator back to CTA 0.
// Whole tiles only, round-robin over the pairs.  4096x14336 with 8192 vectors, thirty calls in
// a row: 390 us, 2470 TFLOP/s (425 with single SMs); in longer runs, at the power limit, 405;
// after a pause 375; a k-block takes 900 cycles, of which the MMA warp waits
// 500 for the accumulator (two of 256 columns fill the tensor memory).
struct F8Pair {
  static constexpr int kN = 256, kCols = 128, kThreads = 384, kAcc = 2;
  static constexpr int kHalf = 128 * kF8Group;                  // bytes of 128 rows of a k-block
  static constexpr int kStage = 2 * kHalf, kStages = 6;
  static constexpr int kBatch = 4, kBatches = 3;                // k-blocks whose scales come together, and such sets
  static constexpr int kScaleFloats = kF8Rows + 4;
  static constexpr int kScaleBytes = kBatches * kBatch * kScaleFloats * 4;
  static constexpr int kWarpBytes = 32 * 64;
  static constexpr int kSmem = 1024 + kStages * kStage + kScaleBytes + 8 * kWarpBytes;
};
__device__ __forceinline__ uint32_t f8_remote(const void *p, uint32_t rank) {  // the same place in the cluster's CTA `rank`
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(tc_smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ bool f8_try_wait_cluster(uint64_t *b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(tc_smem_u32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
// `bytes` of a barrier's phase that no copy will bring.
__device__ __forceinline__ void f8_complete_tx(uint64_t *b, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(tc_smem_u32(b)), "r"(bytes) : "memory");
}

// map_x: the vectors, map_a: the weights, both in boxes of 128 rows.  grid: pairs of CTAs.
static __global__ void __launch_bounds__(F8Pair::kThreads, 1)
    k_f8_pair(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_a, const F8Args a) {
  using F = F8Pair;
  constexpr int S = F::kStages, NACC = F::kAcc, COLS = F::kCols;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[S], empty[S], accf[NACC], acce[NACC], facf[F::kBatches], face[F::kBatches];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ int sh_loaded, sh_consumed, sh_committed;
  __shared__ int other[3];  // the other CTA's abort flag, k-blocks copied, k-blocks committed
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)(blockIdx.x & 1);
  unsigned char *smem = smem_raw + ((1024u - (tc_smem_u32(smem_raw) & 1023u)) & 1023u);
  float *scales = reinterpret_cast<float *>(smem + S * F::kStage);

  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_smem_u32(&tmem_slot)), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      tc_mbar_init(&full[s], 1);   // CTA 0's, for both CTAs' copies
      tc_mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < NACC; ++b) {
      tc_mbar_init(&accf[b], 1);
      tc_mbar_init(&acce[b], 16);  // CTA 0's: the scaling warps of both
    }
    for (int b = 0; b < F::kBatches; ++b) {
      tc_mbar_init(&facf[b], 32);
      tc_mbar_init(&face[b], 8);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    abort_flag = 0;
    sh_loaded = sh_consumed = sh_committed = -1;
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncwarp();
  __syncthreads();
  tc_cluster_sync();  // both CTAs' barriers and tensor memory are there
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_slot;
  volatile int *abort = &abort_flag;
  const int G = a.groups, pairs = (int)gridDim.x / 2;
  const int tiles = (int)a.tiles;
  // (bounded as f8_wait is, for arrivals from the other CTA)
  auto wait_cluster = [&](uint64_t *b, uint32_t parity) {
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
      if (f8_try_wait_cluster(b, parity)) return true;
      if ((i & 255) == 0) {
        if (*abort) return false;
        const uint64_t t = tc_global_ns();
        if (t0 == 0) t0 = t;
        if ((int64_t)(t - t0) > a.timeout_ns) {
          *abort = 1;
          return false;
        }
      }
    }
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    bool ok = true;
    if (warp == 0) {  // copies of this CTA's halves; CTA 0's barrier counts both CTAs'
      int i = 0, s = 0;
      uint32_t ph = 1;
      for (int tile = (int)blockIdx.x / 2; ok && tile < tiles; tile += pairs) {
        int im, in;
        f8_tile(a, tile, im, in);
        const int32_t p0 = (2 * in + rank) * 128, q0 = (2 * im + rank) * 128;
        // test: this CTA of the first pair never copies its last two k-blocks
        const bool stall = a.test_stall == 2 + rank && blockIdx.x < 2 && tile + pairs >= tiles;
        for (int kb = 0; kb < G; ++kb) {
          ok = i < S || f8_wait(&empty[s], ph, a.timeout_ns, abort);
          ok = __all_sync(0xffffffffu, ok) && !(stall && kb + 2 >= G);
          if (!ok) break;
          unsigned char *st = smem + s * F::kStage;
          if (f8_elect()) {
            if (rank == 0) tc_mbar_arrive_expect_tx(&full[s], 2 * F::kStage);
            const uint32_t bar = f8_remote(&full[s], 0);
#pragma unroll
            for (int h = 0; h < 2; ++h)
              asm volatile(
                  "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(
                      tc_smem_u32(st + h * F::kHalf)),
                  "l"(reinterpret_cast<uint64_t>(h == 0 ? &map_x : &map_a)), "r"(kb * kF8Group), "r"(h == 0 ? p0 : q0), "r"(bar)
                  : "memory");
          }
          ++i;
          if (++s == S) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (lane == 0) sh_loaded = i - 1;
    } else if (warp == 1 && rank == 0) {  // MMAs of both CTAs
      // M = 256 (both CTAs' rows), N = 256, e4m3
      const uint32_t idesc = (1u << 4) | ((uint32_t)(F::kN >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
      const uint64_t dp0 = tc_smem_desc(tc_smem_u32(smem)), dq0 = dp0 + (F::kHalf >> 4);
      int i = 0, consumed = -1, s = 0, c = 0;
      uint32_t ph = 0, cph = 1;
      for (int tile = (int)blockIdx.x / 2; ok && tile < tiles; tile += pairs) {
        const bool stall = a.test_stall == 1 && blockIdx.x == 0 && tile + pairs >= tiles;  // test: the last k-block never completes
        for (int kb = 0; kb < G; ++kb) {
          ok = f8_wait(&full[s], ph, a.timeout_ns, abort) && (i < NACC || wait_cluster(&acce[c], cph));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          consumed = i;
          if (stall && kb == G - 1) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint64_t dp = dp0 + (uint64_t)(s * (F::kStage >> 4)), dq = dq0 + (uint64_t)(s * (F::kStage >> 4));
          if (f8_elect()) {
#pragma unroll
            for (int kk = 0; kk < kF8Group / 32; ++kk)
              asm volatile(
                  "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                  "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem + (uint32_t)(c * F::kN)),
                  "l"(dp + 2 * kk), "l"(dq + 2 * kk), "r"(idesc), "r"(kk > 0 ? 1 : 0)
                  : "memory");
            asm volatile(
                "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                    tc_smem_u32(&accf[c])),
                "h"((uint16_t)3)
                : "memory");
          }
          ++i;
          if (++s == S) {
            s = 0;
            ph ^= 1;
          }
          if (++c == NACC) {
            c = 0;
            cph ^= 1;
          }
        }
      }
      if (lane == 0) {
        sh_consumed = consumed;
        sh_committed = i - 1;
      }
    } else if (warp == 2) {  // scales, a batch of k-blocks at a time
      int i = 0, t = 0;
      uint32_t ph = 1;
      for (int tile = (int)blockIdx.x / 2; ok && tile < tiles; tile += pairs) {
        int im, in;
        f8_tile(a, tile, im, in);
        const int64_t b0 = (int64_t)(2 * in + rank) * 128, mb = (int64_t)im * 2 + lane;
        const bool va = lane < 2 && mb * kF8Group < a.M;
        const float *sa = a.a_scale + (va ? mb : 0) * G, *sx[4];
        bool vx[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int64_t b = b0 + lane + 32 * v;
          vx[v] = b < a.B;
          sx[v] = a.x_scale + (vx[v] ? b : 0) * G;
        }
        for (int kb0 = 0; kb0 < G; kb0 += F::kBatch) {
          ok = i < F::kBatches || f8_wait(&face[t], ph, a.timeout_ns, abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          float *w = scales + t * (F::kBatch * F::kScaleFloats);
#pragma unroll
          for (int k = 0; k < F::kBatch; ++k, w += F::kScaleFloats) {
            if (kb0 + k >= G) break;
#pragma unroll
            for (int v = 0; v < 4; ++v) f8_copy4(w + lane + 32 * v, sx[v] + kb0 + k, vx[v]);
            if (lane < 2) f8_copy4(w + kF8Rows + lane, sa + kb0 + k, va);
          }
          f8_copy4_arrive(&facf[t]);
          ++i;
          if (++t == F::kBatches) {
            t = 0;
            ph ^= 1;
          }
        }
      }
      f8_copy4_drain();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int wq = warp & 3, wg = (warp >> 2) - 1;
    const int row = wq * 32 + lane, col0 = wg * COLS;
    unsigned char *mine = smem + S * F::kStage + F::kScaleBytes + (warp - 4) * F::kWarpBytes;
    const uint32_t back[NACC] = {f8_remote(&acce[0], 0), f8_remote(&acce[1], 0)};
    constexpr int CH = 16, P = COLS / CH, U = 2;
    int c = 0, t = 0, st = 0;
    uint32_t cph = 0, tph = 0;
    bool ok = true;
    for (int tile = (int)blockIdx.x / 2; ok && tile < tiles; tile += pairs) {
      int im, in;
      f8_tile(a, tile, im, in);
      float acc[COLS];
#pragma unroll
      for (int j = 0; j < COLS; ++j) acc[j] = 0.f;
      for (int kb = 0; kb < G; ++kb) {
        const int k = kb % F::kBatch;
        ok = (k != 0 || f8_wait(&facf[t], tph, a.timeout_ns, abort)) && f8_wait(&accf[c], cph, a.timeout_ns, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (warp == 4 && lane == 0) tc_mbar_arrive(&empty[st]);
        st = st + 1 == S ? 0 : st + 1;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t at = tmem + ((uint32_t)(wq * 32) << 16) + (uint32_t)(c * F::kN + col0);
        uint32_t r[U][CH];
#pragma unroll
        for (int h = 0; h < U; ++h) f8_ld<CH>(at + h * CH, r[h]);
        const float *fs = scales + (t * F::kBatch + k) * F::kScaleFloats;
        const float f = fs[row] * fs[kF8Rows + wg];
#pragma unroll
        for (int h0 = 0; h0 < P; h0 += U) {
#pragma unroll
          for (int h = 0; h < U; ++h) f8_ld_wait<CH>(r[h]);
          if (h0 + U >= P) {
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(c == 0 ? back[0] : back[1]) : "memory");
          }
#pragma unroll
          for (int h = 0; h < U; ++h) {
            float *sum = acc + (h0 + h) * CH;
#pragma unroll
            for (int j = 0; j < CH; j += 2) f8_fma2(sum[j], sum[j + 1], f, f, r[h][j], r[h][j + 1]);
            if (h0 + U + h < P) f8_ld<CH>(at + (h0 + U + h) * CH, r[h]);
          }
        }
        if (++c == NACC) {
          c = 0;
          cph ^= 1;
        }
        if (k == F::kBatch - 1 || kb == G - 1) {
          __syncwarp();  // every lane has read the batch's scales
          if (lane == 0) tc_mbar_arrive(&face[t]);
          if (++t == F::kBatches) {
            t = 0;
            tph ^= 1;
          }
        }
      }
      if (!ok) break;
      f8_rows_out<COLS>(a, acc, mine, lane, (int64_t)(2 * in + rank) * 128 + wq * 32, (int64_t)im * F::kN + col0);
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncwarp();
  __syncthreads();
  if (tid == 0) {
    tc_st_dsmem_int(&other[0], (uint32_t)(rank ^ 1), abort_flag);
    tc_st_dsmem_int(&other[1], (uint32_t)(rank ^ 1), sh_loaded);
    tc_st_dsmem_int(&other[2], (uint32_t)(rank ^ 1), sh_committed);
  }
  tc_cluster_sync();  // the other CTA's MMAs, copies and arrivals are done with this one; or:
  if (abort_flag != 0 || other[0] != 0) {
    // Nothing may be in flight when the pair frees its tensor memory and exits.  Both wait for
    // the last commit, which reaches both.  CTA 0's barriers count both CTAs' copies: for
    // k-blocks that it has not begun and the other has, it expects the other's half alone;
    // for those that only it has begun, it accounts for the other's half itself.  (None is
    // a ring's length past the last product, so each stage's phase is that of its k-block.)
    if (tid == 0) {
      if (a.status != nullptr) atomicOr(a.status, kTcStatusMma);
      const int committed = rank == 0 ? sh_committed : other[2];
      bool drained = committed < 0 || tc_mbar_wait(&accf[committed % NACC], (uint32_t)((committed / NACC) & 1), a.timeout_ns);
      if (rank == 0) {
        const int mine = sh_loaded, theirs = other[1], last = mine > theirs ? mine : theirs;
        for (int t = sh_consumed + 1; t <= last && drained; ++t) {
          if (t > mine)
            tc_mbar_arrive_expect_tx(&full[t % S], F::kStage);
          else if (t > theirs)
            f8_complete_tx(&full[t % S], F::kStage);
          drained = tc_mbar_wait(&full[t % S], (uint32_t)((t / S) & 1), a.timeout_ns);
        }
      }
      if (!drained && a.status != nullptr) atomicOr(a.status, kTcStatusDrain);
    }
    __syncwarp();
    __syncthreads();
    tc_cluster_sync();
  }
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// Tiles whose k-blocks several CTAs of k_f8 share: their partial sums, added in the
// order of the k-blocks, and the epilogue.  grid (shared tiles, pieces of 1024 values),
// a thread for four consecutive outputs: two or three dependent reads, 2 to 3 us after k_f8
// (prompts, whose parts are 128 KB: 14 us).
constexpr int kF8JoinThreads = 256, kF8JoinPiece = 4 * kF8JoinThreads;
template <int N, bool kPrompt>
__global__ void __launch_bounds__(kF8JoinThreads) k_f8_join(const F8Args a) {
  pdl_trigger();
  const int64_t R = a.shared * a.groups, u0 = (int64_t)blockIdx.x * a.groups;
  const int64_t w0 = f8_owner(u0, R, a.sharers), w1 = f8_owner(u0 + a.groups - 1, R, a.sharers);
  pdl_wait();            // by every CTA: the next kernel counts on it
  if (w0 == w1) return;  // one CTA had the whole tile and wrote it
  int im, in;
  f8_tile(a, blockIdx.x, im, in);
  const int e = (blockIdx.y * kF8JoinThreads + threadIdx.x) * 4;
  const int row = kPrompt ? e / N : e % kF8Rows, col = kPrompt ? e % N : e / kF8Rows;
  const int64_t b = kPrompt ? (int64_t)in * kF8Rows + row : col;
  const int64_t m = kPrompt ? (int64_t)im * N + col : (int64_t)im * kF8Rows + row;
  if (b >= a.B || m >= a.M) return;
  constexpr int64_t kStep = 2 * (int64_t)kF8Rows * N;
  // the first CTA's range may have begun in the tile before: then this is its second part
  const float *p = a.ws + w0 * kStep + (w0 * R / a.sharers < u0 ? kStep / 2 : 0) + e;
  const float *const q = a.ws + w0 * kStep + e;
  const int n = (int)(w1 - w0);
  float4 s = *reinterpret_cast<const float4 *>(p);
#pragma unroll 8
  for (int i = 1; i <= n; ++i) {
    const float4 v = *reinterpret_cast<const float4 *>(q + i * kStep);
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  f8_store_along(a, b, m, s);
}

// No columns: the empty sum.
static __global__ void k_f8_empty(const F8Args a) {
  pdl_trigger();
  pdl_wait();
  const int64_t n = a.M * a.B;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
    f8_store(a, i, a.bias != nullptr ? f8_bias(a, i % a.M) : 0.f);
}

// ------------------------------------------------------------------ the quantiser
// Two values to e4m3, round to nearest even; beyond +-448, infinities too, to +-448;
// NaN stays NaN.  `a` in the low byte.
__device__ __forceinline__ uint32_t f8_pack2(float a, float b) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// |v| if v is finite, else 0.
__device__ __forceinline__ float f8_finite_abs(float v) {
  const float m = fabsf(v);
  return m < __int_as_float(0x7f800000) ? m : 0.f;
}
// Eight lanes hold a group's 128 values, sixteen each, so the group is read once and its
// largest value found by three shuffles.  kWide: how many consecutive ones a lane reads and
// writes at a time: eight (rows of whole 16-byte pieces), two (rows of an even length) or
// one (us, 3204 x 5080, 5082 and 5081 in bf16: 9.2, 13.7 and 24.1).  The largest absolute value is taken
// first over all values, infinities among them, on two 16-bit values per instruction;
// only where it is infinite are the finite ones looked at one by one.  Bound by memory:
// 8192 x 14336 in bf16 50.5 us, 7.05 TB/s.
constexpr int kF8QThreads = 256, kF8QTeam = 8;
template <int DT>
struct F8Raw {  // eight values as loaded
  static constexpr int kWords = DT == GEMV_DTYPE_F32 ? 8 : 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void load(const void *p, int64_t i) {
    const uint4 *q = reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(p) + i * (DT == GEMV_DTYPE_F32 ? 4 : 2));
#pragma unroll
    for (int h = 0; h < kWords / 4; ++h) {
      const uint4 v = __ldg(q + h);
      w[4 * h] = v.x; w[4 * h + 1] = v.y; w[4 * h + 2] = v.z; w[4 * h + 3] = v.w;
    }
  }
  __device__ __forceinline__ void set(int e, const void *p, int64_t i) {  // value e from element i
    if constexpr (DT == GEMV_DTYPE_F32)
      w[e] = __ldg(reinterpret_cast<const uint32_t *>(p) + i);
    else
      w[e / 2] |= (uint32_t)__ldg(reinterpret_cast<const unsigned short *>(p) + i) << (16 * (e & 1));
  }
  __device__ __forceinline__ void set2(int e, const void *p, int64_t i) {  // values e, e + 1 (e even, i even)
    if constexpr (DT == GEMV_DTYPE_F32) {
      const uint2 v = __ldg(reinterpret_cast<const uint2 *>(reinterpret_cast<const uint32_t *>(p) + i));
      w[e] = v.x;
      w[e + 1] = v.y;
    } else {
      w[e / 2] = __ldg(reinterpret_cast<const uint32_t *>(reinterpret_cast<const unsigned short *>(p) + i));
    }
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (DT == GEMV_DTYPE_F32) return __uint_as_float(w[e]);
    if constexpr (DT == GEMV_DTYPE_F16) {
      const float2 f = f16x2_to_f2(w[e / 2]);
      return (e & 1) ? f.y : f.x;
    }
    return (e & 1) ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
  }
  // largest absolute value, NaN passed over
  __device__ __forceinline__ float top() const {
    if constexpr (DT == GEMV_DTYPE_F32) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(__uint_as_float(w[i])));
      return m;
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t v = w[i] & 0x7fff7fffu;
        if constexpr (DT == GEMV_DTYPE_F16)
          asm("max.f16x2 %0, %0, %1;" : "+r"(m) : "r"(v));
        else
          asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(v));
      }
      if constexpr (DT == GEMV_DTYPE_F16) {
        const float2 f = f16x2_to_f2(m);
        return fmaxf(f.x, f.y);
      }
      return fmaxf(bf16_lo(m), bf16_hi(m));
    }
  }
};
template <int DT, int kWide, int U>
__global__ void __launch_bounds__(kF8QThreads)
    k_f8_quantize(const void *x, uint8_t *q, float *scale, int64_t K, int G, int64_t groups) {
  pdl_trigger();
  pdl_wait();
  constexpr int kTeams = kF8QThreads / kF8QTeam;
  const int lane = threadIdx.x & (kF8QTeam - 1);
  const int64_t first = (int64_t)blockIdx.x * (kTeams * U) + threadIdx.x / kF8QTeam;
  F8Raw<DT> v[U][2];
  int64_t base[U];
  int n[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t t = first + u * kTeams;
    n[u] = 0;
    v[u][0].zero();
    v[u][1].zero();
    if (t >= groups) continue;
    base[u] = t * kF8Group;
    n[u] = kF8Group;
    if (K % kF8Group != 0) {  // rows end inside a group
      const int64_t b = groups <= 0x7fffffff ? (int64_t)((uint32_t)t / (uint32_t)G) : t / G;
      const int64_t k0 = (t - b * G) * kF8Group;
      base[u] = b * K + k0;
      n[u] = K - k0 < kF8Group ? (int)(K - k0) : kF8Group;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (kWide == 8) {
        if (h * 64 + lane * 8 < n[u]) v[u][h].load(x, base[u] + h * 64 + lane * 8);
      } else if constexpr (kWide == 2) {
#pragma unroll
        for (int e = 0; e < 8; e += 2)
          if (h * 64 + e * 8 + lane * 2 < n[u]) v[u][h].set2(e, x, base[u] + h * 64 + e * 8 + lane * 2);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (h * 64 + e * 8 + lane < n[u]) v[u][h].set(e, x, base[u] + h * 64 + e * 8 + lane);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float m = fmaxf(v[u][0].top(), v[u][1].top());
#pragma unroll
    for (int d = kF8QTeam / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (__any_sync(0xffffffffu, m == __int_as_float(0x7f800000))) {  // an infinity: the finite values' largest
      float f = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) f = fmaxf(f, fmaxf(f8_finite_abs(v[u][0].get(e)), f8_finite_abs(v[u][1].get(e))));
#pragma unroll
      for (int d = kF8QTeam / 2; d > 0; d >>= 1) f = fmaxf(f, __shfl_xor_sync(0xffffffffu, f, d));
      m = f;
    }
    if (n[u] == 0) continue;
    const float s = fmaxf(__fdiv_rn(m, 448.f), 0x1p-126f), r = __frcp_rn(s);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const F8Raw<DT> &w = v[u][h];
      if constexpr (kWide == 8) {
        uint32_t o[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          o[i] = f8_pack2(w.get(4 * i) * r, w.get(4 * i + 1) * r) | (f8_pack2(w.get(4 * i + 2) * r, w.get(4 * i + 3) * r) << 16);
        if (h * 64 + lane * 8 < n[u]) *reinterpret_cast<uint2 *>(q + base[u] + h * 64 + lane * 8) = make_uint2(o[0], o[1]);
      } else if constexpr (kWide == 2) {
#pragma unroll
        for (int e = 0; e < 8; e += 2)
          if (h * 64 + e * 8 + lane * 2 < n[u])
            *reinterpret_cast<unsigned short *>(q + base[u] + h * 64 + e * 8 + lane * 2) =
                (unsigned short)f8_pack2(w.get(e) * r, w.get(e + 1) * r);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (h * 64 + e * 8 + lane < n[u]) q[base[u] + h * 64 + e * 8 + lane] = (uint8_t)f8_pack2(w.get(e) * r, 0.f);
      }
    }
    if (lane == 0) scale[first + u * kTeams] = s;
  }
}

}  // namespace gemv
