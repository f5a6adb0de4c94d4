// Kernels of the attention of sequences that share a prefix (gemv_kv8_prefix_attention):
// the shared blocks against the queries of all sequences of a group, on the tensor cores,
// and the join with the parts of each sequence's own blocks (k_kv8_attention<.., kOwn>).
//
// A group's queries of one of the cache's heads are the rows of a matrix, row
// (s T + t) group + i for query head i of that head's group.  For a block of 64 tokens
//     S = Q K^T          128 rows x 64 tokens, tcgen05 kind::f16
//     P = 2^(S f - ..)   fp32, rounded to fp16
//     O += P V           128 rows x D channels, in tensor memory over all blocks
// The cached values become fp16 (exact) in shared memory once for all rows of the CTA; S, P and
// O, and Q where it fits, stay in tensor memory, so that shared memory only feeds K and V.
#pragma once

#include <type_traits>

#include "gemv_kv8.cuh"

namespace gemv {

template <int D>
struct PxForm {
  // Two sets of S, P and O where tensor memory holds them: an item has up to 256 rows, a tile of
  // 128 for each set; an item of up to 128 rows gives both sets its rows, and the blocks to
  // them by turns.  192 and 256 channels: one set, items of up to 128 rows.
  static constexpr int kSets = D <= 128 ? 2 : 1;
  static constexpr int kRows = 128 * kSets;
  static constexpr int kSoft = 4 * kSets, kConv = 4;                      // warps
  static constexpr int kWarps = kSoft + kConv + 3, kThreads = kWarps * 32;  // copies, the two products
  static constexpr int kRaw = kKvBlock * D, kStage = 2 * kRaw;   // bytes of a block's keys or values: as cached, as fp16
  static constexpr int kStages = D == 64 ? 4 : D == 128 ? 3 : 2;  // blocks as fp16
  static constexpr int kSlots = D == 64 ? 8 : D == 128 ? 5 : D == 192 ? 4 : 2;  // blocks as cached
  // tensor memory columns: O of each set, S and P of each, Q
  static constexpr int kS = kSets * D, kQ = kS + kSets * 96;
  // with 128 channels the second set's Q finds no room there: it stays in shared memory (48 cycles
  // an MMA, not 32)
  static constexpr bool kQShared = D == 128;
  static_assert(kQ + (kQShared ? 1 : kSets) * D / 2 <= 512);
  static constexpr int kQBytes = kQShared ? 128 * D * 2 : 0;
  static constexpr int kSmem = 1024 + kQBytes + 2 * (kStages * kStage + kSlots * kRaw);
  // one CTA an SM (each takes all of the tensor memory)
  static_assert(kSmem > 114 * 1024 && kSmem <= 226 * 1024);
  // floats of a partial result's set: O as [D / 4][128 rows][4], the weights' references, their sums
  static constexpr int64_t kPart = 128 * (D + 2);
};
// Blocks whose scales are kept.  While the softmax is at block j, the converters are at
// j + kStages + 1 at most, and the copies kSlots + 1 further on.
constexpr int kPxMeta = 32;
constexpr int kPxCost1 = 1, kPxCost2 = 2;  // places of a block: of an item of up to 128 rows, of more
constexpr int kPxLeast = 4;       // blocks that a CTA takes at least
// The weights leave with a factor of 2^8, and O is scaled anew (a warp takes some 1000 cycles
// for that) once those of a row and block come to 2^15: fp16 holds them, and in full down to
// 2^-22 of the reference.
constexpr float kPxLift = 8.f, kPxFull = 32768.f;

// A group's part of the work list: its tiles of kRows rows, of each the heads, of each the
// shared blocks.  (The host limits all groups' places to 31 bits: the first thing that a CTA
// does is to find its share, and a 64-bit division there costs a microsecond, most of it for
// the code to come.)
struct PxGroup {
  int first, blocks, rows, tiles;
  int leader;              // the first sequence that shares the blocks: they are taken from its table
  unsigned last, places;  // places of a block in the last tile; of the group
};
template <int D>
__host__ __device__ constexpr unsigned px_full() { return PxForm<D>::kRows > 128 ? kPxCost2 : kPxCost1; }  // in a whole tile
// kWarp: by a converged warp for one group, else by each lane for a group of its own.
template <int D, bool kWarp>
__device__ __forceinline__ PxGroup px_group(const KvArgs &a, int g, int lane) {
  PxGroup p;
  const KvGroup k = kv_group(a, g);
  p.first = k.first;
  p.blocks = k.blocks;
  p.leader = k.end;
  const int need = k.blocks * kKvBlock + a.T;  // (a length beyond the table counts as the table's size)
  if (k.blocks > 0 && (int64_t)need <= (int64_t)a.width * kKvBlock) {
    if constexpr (kWarp) {
      for (int s = k.first; s < k.end; s += 32) {
        const unsigned sees = __ballot_sync(0xffffffffu, s + lane < k.end && __ldg(a.lens + s + lane) >= need);
        if (sees != 0) {
          p.leader = s + __ffs(sees) - 1;
          break;
        }
      }
    } else {
      for (int s = k.first; s < k.end && p.leader == k.end; ++s)
        if (__ldg(a.lens + s) >= need) p.leader = s;
    }
  }
  if (p.leader == k.end) p.blocks = 0;  // no one shares them
  p.rows = (k.end - k.first) * a.T * a.group;
  constexpr int R = PxForm<D>::kRows;
  p.tiles = (p.rows + R - 1) / R;
  p.last = p.rows - (p.tiles - 1) * R > 128 ? kPxCost2 : kPxCost1;
  p.places = p.tiles == 0 ? 0u : (unsigned)a.heads * p.blocks * ((unsigned)(p.tiles - 1) * px_full<D>() + p.last);
  return p;
}
// Number of a group's first tile, rising with the groups, none twice (a group has at most
// one more than the rows before its end, by the tile, take it further on).
template <int D>
__device__ __forceinline__ int px_tile0(const KvArgs &a, int g, int first) {
  return first * a.T * a.group / PxForm<D>::kRows + g;
}

struct PxSeg {
  int tile, h;      // tile of its group's rows, head
  int b0, b1;       // its blocks; none: the share's end
  int rows;         // of the tile
  int first;        // the group's first sequence
  int table;        // the sequence whose table has the blocks
  int item;         // (tile's number) x heads + head
  int parts;        // with the item's first blocks: CTAs that have some of it; else 0
};
// The CTA's share of the work list: places [at, hi), of all groups' `total`.  Blocks whose
// first place is in there are its own.
template <int D>
struct PxWalk {
  unsigned each, more;    // places of a CTA, the first `more` have one more
  unsigned at, hi, base;  // next place, end, place of the group's first
  int g;
  PxGroup p;
  __device__ unsigned owner(unsigned u) const {
    const unsigned longer = more * (each + 1);
    return u < longer ? u / (each + 1) : more + (u - longer) / each;
  }
  // Places of group g + lane.
  __device__ unsigned near(const KvArgs &a, int g, int lane) const {
    return g + lane < a.groups ? px_group<D, false>(a, g + lane, lane).places : 0u;
  }
  __device__ void begin(const KvArgs &a, int lane) {  // one warp, converged
    p = px_group<D, true>(a, 0, lane);
    const unsigned n = near(a, 1, lane);
    unsigned total = p.places + __reduce_add_sync(0xffffffffu, n);
    for (int g0 = 33; g0 < a.groups; g0 += 32) total += __reduce_add_sync(0xffffffffu, near(a, g0, lane));
    unsigned W = total / (kPxLeast * kPxCost2);
    W = W < 1 ? 1 : W < gridDim.x ? W : gridDim.x;
    each = total / W;
    more = total - each * W;
    auto first = [&](unsigned w) { return w >= W ? total : w * each + (w < more ? w : more); };
    at = first(blockIdx.x);
    hi = first(blockIdx.x + 1);
    g = 0;
    base = 0;
    if (at < hi && at >= p.places) seek(a, lane, n);
  }
  // The group of place `at`, behind group g, 32 at a time (one after the other, some 0.6 us each, a
  // CTA behind 1000 groups began that much later); n: the places of the next 32.
  __device__ void seek(const KvArgs &a, int lane, unsigned n) {
    base += p.places;
    for (++g;;) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const unsigned o = __shfl_up_sync(0xffffffffu, n, d);
        if (lane >= d) n += o;
      }
      const unsigned past = __ballot_sync(0xffffffffu, n > at - base);
      if (past != 0) {
        const int f = __ffs(past) - 1;
        const unsigned before = __shfl_sync(0xffffffffu, n, f > 0 ? f - 1 : 0);
        if (f > 0) base += before;
        g += f;
        p = px_group<D, true>(a, g, lane);
        return;
      }
      base += __shfl_sync(0xffffffffu, n, 31);
      g += 32;
      if (g >= a.groups) break;
      n = near(a, g, lane);
    }
    at = hi;  // (none: `firsts` that do not rise, so that the groups' places pass 32 bits)
  }
  __device__ bool next(const KvArgs &a, int lane, PxSeg &s) {
    while (at < hi) {
      if (at - base >= p.places) {
        seek(a, lane, near(a, g + 1, lane));
        continue;
      }
      unsigned r = at - base;
      const unsigned per_block = (unsigned)a.heads * p.blocks, tile = per_block * px_full<D>();
      const int last = p.tiles - 1;
      s.tile = last == 0 ? 0 : (int)(r / tile);
      if (s.tile > last) s.tile = last;
      r -= s.tile * tile;
      const unsigned cost = s.tile == last ? p.last : px_full<D>(), item = p.blocks * cost;
      s.h = (int)(r / item);
      r -= s.h * item;
      const unsigned item0 = at - r, left = hi - item0;
      s.first = p.first;
      s.table = p.leader;
      s.rows = s.tile == last ? p.rows - last * PxForm<D>::kRows : PxForm<D>::kRows;
      s.item = (px_tile0<D>(a, g, p.first) + s.tile) * a.heads + s.h;
      s.b0 = (int)((r + cost - 1) / cost);
      s.b1 = left >= item ? p.blocks : (int)((left + cost - 1) / cost);
      s.parts = s.b0 == 0 ? (int)(owner(item0 + (p.blocks - 1) * cost) - blockIdx.x) + 1 : 0;
      at = left >= item ? item0 + item : hi;
      if (s.b0 < s.b1) return true;
    }
    s = {0, 0, 0, 0, 0, 0, 0, 0, 0};
    return false;
  }
};
constexpr int kPxSegs = 4;  // segments that the copies' warp is ahead

// ------------------------------------------------------------------ instructions
// D (tensor memory, fp32) (+)= A (tensor memory, fp16, two columns of k to a word) B, by
// the elected lane.  The instruction is predicated, not branched around: addresses worked out
// inside a branch of one lane leave the uniform registers (75 cycles to issue each, not 32).
__device__ __forceinline__ void px_mma(uint32_t elected, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}
// The same with A in shared memory.
__device__ __forceinline__ void px_mma_shared(uint32_t elected, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void px_commit(uint32_t elected, uint64_t *b) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(tc_smem_u32(b)),
      "r"(elected)
      : "memory");
}
// 32 words of this thread's tensor-memory lane; stored after px_st_wait.
__device__ __forceinline__ void px_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void px_st16(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void px_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void px_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void px_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ float px_log2(float v) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// (x, y) = (x, y) f + c;  (x, y) += (u, v)
__device__ __forceinline__ void px_fma2(float &x, float &y, float f, float c) {
  asm("{\n\t.reg .b64 a, f, c;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 f, {%2, %2};\n\tmov.b64 c, {%3, %3};\n\t"
      "fma.rn.f32x2 a, a, f, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(f), "f"(c));
}
__device__ __forceinline__ void px_add2(float &x, float &y, float u, float v) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tadd.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(u), "f"(v));
}

// Eight 16-bit values from anywhere (a call: such rows are rare).
static __device__ __noinline__ uint4 px_load8(const unsigned short *p) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = __ldg(p + 2 * j) | ((uint32_t)__ldg(p + 2 * j + 1) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ------------------------------------------------------------------ the shared blocks
// One CTA per SM over its share of the work list.  Warps:
//   copies       finds the share's segments and tells the others; a block's keys and values by the
//                bulk copy engine into a ring of raw slots, its scales beside them
//   converters   raw e4m3 to fp16, in the 128-byte swizzle that the MMA reads: keys as 64 rows of
//                tokens, values as D rows of channels, both along the product's k
//   scores, sums the two products, a warp each: the queue between it and the tensor cores is
//                short, and they idle while a single warp waits for its next barrier.  Step i
//                uses set i % 2 and block i / 2 (more than 128 rows: both sets meet every block), or
//                block i.  S of a set's next step is begun as soon as its softmax has read the last
//                one: P has columns of its own
//   softmax      four warps a set, a row to a thread: Q to tensor memory at an item's start, S to P
//                for each step, O out at its end
// O is scaled anew only where a row's weights (times their block's value scale, which goes
// into P) come to 2^15 of its units: as a rule in the first blocks only.
// 16 x 64 queries of 4 heads behind 16384 tokens, 8 key heads of 128 (275 GFLOP): 250 us, 1100
// TFLOP/s; 64 queries behind 32768 (67 MB, 34 GFLOP) 56 us.  A block of 64 tokens takes some 2000
// cycles for 256 rows, where the products take 1150, exp2 512 and shared memory 1250: bound by
// the softmax warps' chains of dependent instructions (39 % of the issue slots, 25 % of the tensor
// cycles in use); the registers hold no more of them.  Some 13 us pass until the first weights
// (share, queries, blocks, instructions, one after the other), 4 at the end.
template <int D, int DT>
__global__ void __launch_bounds__(PxForm<D>::kThreads, 1) k_kv8_prefix(const KvArgs a) {
  using F = PxForm<D>;
  constexpr int R = F::kSlots, NS = F::kStages;
  static_assert(NS + R + 3 < kPxMeta);
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t rawf[R], rawe[R], wf[NS], we[NS], gf[kPxSegs], ge[kPxSegs], ql, fin;
  __shared__ __align__(8) uint64_t qf[F::kSets], sf[F::kSets], sr[F::kSets], pf[F::kSets], of[F::kSets];
  __shared__ PxSeg segs[kPxSegs];
  __shared__ float meta[kPxMeta][2];  // of a block: the keys' and the values' scale
  __shared__ int meta_bad[kPxMeta];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char *smem = smem_raw + ((1024u - (tc_smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char *qst = smem, *kst = smem + F::kQBytes, *vst = kst + NS * F::kStage, *raw = vst + NS * F::kStage;
  constexpr int kLoad = F::kSoft + F::kConv, kScores = kLoad + 1, kSums = kLoad + 2;
  if (warp == kSums) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_smem_u32(&tmem_slot)), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < R; ++i) {
      tc_mbar_init(&rawf[i], 2);  // keys and values, and the scales
      tc_mbar_init(&rawe[i], F::kConv);
    }
    for (int i = 0; i < NS; ++i) {
      tc_mbar_init(&wf[i], F::kConv);
      tc_mbar_init(&we[i], 2 * F::kSets);  // both products of each set
    }
    tc_mbar_init(&ql, F::kSoft);  // the first queries have been read
    for (int i = 0; i < F::kSets; ++i) {
      tc_mbar_init(&qf[i], 4);  // Q is there
      tc_mbar_init(&sf[i], 1);  // S is
      tc_mbar_init(&sr[i], 4);  // S has been read
      tc_mbar_init(&pf[i], 4);  // P is there
      tc_mbar_init(&of[i], 1);  // P V is done
    }
    for (int i = 0; i < kPxSegs; ++i) {
      tc_mbar_init(&gf[i], 1);
      tc_mbar_init(&ge[i], F::kSoft + F::kConv + 2);
    }
    tc_mbar_init(&fin, 2);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    abort_flag = 0;
  }
  px_fence_before();
  __syncwarp();
  __syncthreads();
  // After the wait: the next kernels read the batch's lengths before theirs.  With the tensor memory
  // at hand: one that takes some and waits for this one cannot keep it from it.
  pdl_trigger();
  px_fence_after();
  const uint32_t tmem = tmem_slot;
  volatile int *abort = &abort_flag;
  auto wait = [&](uint64_t *b, int n, int of) {  // phase n of a ring of `of`
    return __all_sync(0xffffffffu, f8_wait(b, (uint32_t)(n / of) & 1u, a.timeout_ns, abort)) != 0;
  };

  bool ok = true;
  int c0 = 0;  // blocks of the segments before; of the copies and the converters, so far
  int seg = 0;
  PxSeg s;
  auto take = [&]() {  // the next segment; false at the end
    const int at = seg % kPxSegs;
    ok = ok && wait(&gf[at], seg, kPxSegs);
    if (!ok) return false;
    s = segs[at];
    __syncwarp();
    if (lane == 0) tc_mbar_arrive(&ge[at]);
    ++seg;
    return s.b0 < s.b1;
  };
  if (warp == kLoad) {  // ---- copies
    PxWalk<D> walk;
    walk.begin(a, lane);
    for (bool more = true; more;) {
      more = walk.next(a, lane, s);
      const int at = seg % kPxSegs;
      ok = seg < kPxSegs || wait(&ge[at], seg - kPxSegs, kPxSegs);
      if (!ok) break;
      if (lane == 0) {
        segs[at] = s;
        tc_mbar_arrive(&gf[at]);
      }
      __syncwarp();
      ++seg;
      int32_t entries = 0;
      for (int b = s.b0; ok && b < s.b1; ++b, ++c0) {
        const int i = (b - s.b0) & 31, to = c0 % R, n = c0 % kPxMeta;
        if (i == 0) entries = b + lane < s.b1 ? __ldg(a.table + (int64_t)s.table * a.width + b + lane) : -1;
        const int32_t entry = __shfl_sync(0xffffffffu, entries, i);
        const bool good = entry >= 0 && entry < a.blocks;
        const int64_t unit = (good ? (int64_t)entry : 0) * a.heads + s.h;  // (of an entry that is no block: any, unseen)
        // the first queries' reads go before most of the first blocks': behind them all they take
        // three times as long
        if (c0 == 2) ok = wait(&ql, 0, 1);
        ok = ok && (c0 < R || wait(&rawe[to], c0 - R, R));
        if (!ok) break;
        if (f8_elect()) {
          meta_bad[n] = !good;
          if (!good && a.status != nullptr) atomicOr(a.status, kKvStatusTable);
          f8_copy4(&meta[n][0], a.k_scale + unit, true);
          f8_copy4(&meta[n][1], a.v_scale + unit, true);
          f8_copy4_arrive(&rawf[to]);
          tc_mbar_arrive_expect_tx(&rawf[to], 2 * F::kRaw);
          unsigned char *at = raw + (size_t)to * (2 * F::kRaw);
          kv_bulk(at, a.k + unit * F::kRaw, F::kRaw, &rawf[to]);
          if (!a.test_stall) kv_bulk(at + F::kRaw, a.v + unit * F::kRaw, F::kRaw, &rawf[to]);  // test: no values ever come
        }
        __syncwarp();
      }
      if (!ok) break;
    }
    f8_copy4_drain();
  } else if (warp == kScores || warp == kSums) {  // ---- products
    // (Addresses and counts that the compiler knows to be alike in all lanes stay in uniform
    // registers, which the MMA takes: __reduce_max_sync and the votes give such.)
    constexpr uint32_t kAll = 0xffffffffu;
    const uint32_t tm = __reduce_max_sync(kAll, tmem), elected = f8_elect();
    const std::integral_constant<int, 0> set0;
    const std::integral_constant<int, F::kSets - 1> set1;
    uint32_t ix = 0, iph = 0, ph[2] = {0, 0}, qph[2] = {0, 0};  // stage in use, phases
    auto ready = [&](uint64_t *b, uint32_t parity) { ok = ok && __all_sync(kAll, f8_wait(b, parity, a.timeout_ns, abort)) != 0; };
    auto pass = [&]() {  // to the next stage
      if (++ix == NS) {
        ix = 0;
        iph ^= 1;
      }
    };
    if (warp == kScores) {
      const uint32_t id = tc_idesc(false, kKvBlock);
      const uint64_t dk = tc_smem_desc(tc_smem_u32(kst)), dq = tc_smem_desc(tc_smem_u32(qst));
      while (__any_sync(kAll, take())) {
        const bool both = __any_sync(kAll, F::kSets > 1 && s.rows > 128);
        const int nb = (int)__reduce_max_sync(kAll, (unsigned)(s.b1 - s.b0)), n = both ? 2 * nb : nb;
        auto step = [&](auto set, bool first) {  // S of the set's next step, once it has read the last
          constexpr int x = decltype(set)::value;
          if (!(both && x == 1)) ready(&wf[ix], iph);
          if (!first) {
            ready(&sr[x], ph[x]);
            ph[x] ^= 1;
          }
          if (!ok) return;
          px_fence_after();
          const uint32_t d = tm + F::kS + x * 96;
          const uint64_t at = dk + (uint64_t)(ix * (F::kStage >> 4));
          if (x == 1 && F::kQShared && both) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              px_mma_shared(elected, d, dq + (k >> 2) * (128 * 128 >> 4) + (k & 3) * 2, at + (k >> 2) * (kKvBlock * 128 >> 4) + (k & 3) * 2,
                            id, k > 0);
          } else {
            const uint32_t q = tm + F::kQ + (x == 1 && both ? D / 2 : 0);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              px_mma(elected, d, q + k * 8, at + (k >> 2) * (kKvBlock * 128 >> 4) + (k & 3) * 2, id, k > 0);
          }
          px_commit(elected, &sf[x]);
          px_commit(elected, &we[ix]);
          if (F::kSets > 1 && !both) px_commit(elected, &we[ix]);  // (no other set needs the stage)
          if (!both || x == 1) pass();
        };
        ready(&qf[0], qph[0]);
        qph[0] ^= 1;
        if (both) {
          ready(&qf[F::kSets - 1], qph[1]);
          qph[1] ^= 1;
        }
        for (int i = 0; i < n && ok; i += F::kSets) {
          step(set0, i == 0);
          if (F::kSets > 1 && ok && i + 1 < n) step(set1, i == 0);
        }
        // each set's last S is read, too: the phases of the next segment begin behind it
        if (n > 0) {
          ready(&sr[0], ph[0]);
          ph[0] ^= 1;
        }
        if (F::kSets > 1 && n > 1) {
          ready(&sr[F::kSets - 1], ph[F::kSets - 1]);
          ph[F::kSets - 1] ^= 1;
        }
      }
    } else {
      const uint32_t id = tc_idesc(false, D);
      const uint64_t dv = tc_smem_desc(tc_smem_u32(vst));
      while (__any_sync(kAll, take())) {
        const bool both = __any_sync(kAll, F::kSets > 1 && s.rows > 128);
        const int nb = (int)__reduce_max_sync(kAll, (unsigned)(s.b1 - s.b0)), n = both ? 2 * nb : nb;
        auto step = [&](auto set, bool add) {  // P V of the set's step
          constexpr int x = decltype(set)::value;
          if (!(both && x == 1)) ready(&wf[ix], iph);
          ready(&pf[x], ph[x]);
          if (!ok) return;
          ph[x] ^= 1;
          px_fence_after();
          const uint32_t d = tm + x * D, w = tm + F::kS + x * 96 + 64;
          const uint64_t at = dv + (uint64_t)(ix * (F::kStage >> 4));
#pragma unroll
          for (int k = 0; k < kKvBlock / 16; ++k) px_mma(elected, d, w + k * 8, at + k * 2, id, k > 0 || add);
          px_commit(elected, &of[x]);
          px_commit(elected, &we[ix]);
          if (F::kSets > 1 && !both) px_commit(elected, &we[ix]);
          if (!both || x == 1) pass();
        };
        for (int i = 0; i < n && ok; i += F::kSets) {
          step(set0, i > 0);
          if (F::kSets > 1 && ok && i + 1 < n) step(set1, i > 0);
        }
      }
    }
  } else if (warp >= F::kSoft && warp < kLoad) {  // ---- e4m3 to fp16
    const int ct = tid - F::kSoft * 32;
    auto widen = [&](const uint4 &x, unsigned char *row, int chunk, int turn, bool swap) {
      const uint4 lo = make_uint4(kv_half2_lo(x.x), kv_half2_hi(x.x), kv_half2_lo(x.y), kv_half2_hi(x.y));
      const uint4 hi = make_uint4(kv_half2_lo(x.z), kv_half2_hi(x.z), kv_half2_lo(x.w), kv_half2_hi(x.w));
      // (which half goes first: neighbouring threads' stores spread over the banks)
      *reinterpret_cast<uint4 *>(row + (((chunk + (swap ? 1 : 0)) ^ turn) * 16)) = swap ? hi : lo;
      *reinterpret_cast<uint4 *>(row + (((chunk + (swap ? 0 : 1)) ^ turn) * 16)) = swap ? lo : hi;
    };
    constexpr int kPer = kKvBlock * D / 16 / (F::kConv * 32);  // 16-byte pieces of a thread, of keys and of values
    constexpr int kBoth = D <= 128 ? 2 * kPer : kPer;          // of which the registers hold so many at a time
    while (take()) {
      for (int b = s.b0; b < s.b1; ++b, ++c0) {
        const int st = c0 % NS, at = c0 % R;
        ok = wait(&rawf[at], c0, R) && (c0 < NS || wait(&we[st], c0 - NS, NS));
        if (!ok) break;
        const bool bad = meta_bad[c0 % kPxMeta] != 0;
        const uint4 *from = reinterpret_cast<const uint4 *>(raw + (size_t)at * (2 * F::kRaw)) + ct;
#pragma unroll
        for (int i0 = 0; i0 < 2 * kPer; i0 += kBoth) {
          uint4 x[kBoth];
#pragma unroll
          for (int i = 0; i < kBoth; ++i) x[i] = from[(i0 + i) * F::kConv * 32];  // (the values follow the keys)
#pragma unroll
          for (int i = 0; i < kBoth; ++i) {
            const int p = (i0 + i) % kPer * F::kConv * 32 + ct;
            if (i0 + i < kPer) {
              const int tok = p / (D / 16), cp = p - tok * (D / 16);
              widen(x[i], kst + st * F::kStage + (cp >> 2) * (kKvBlock * 128) + tok * 128, (cp & 3) * 2, tok & 7, (cp >> 2) & 1);
            } else {
              const int d = p >> 2;
              if (bad) x[i] = make_uint4(0, 0, 0, 0);
              widen(x[i], vst + st * F::kStage + d * 128, (p & 3) * 2, d & 7, false);
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          tc_mbar_arrive(&wf[st]);
          tc_mbar_arrive(&rawe[at]);
        }
      }
    }
  } else if (warp < F::kSoft) {  // ---- softmax
    const int x = warp >> 2, quarter = warp & 3;
    const int in_tile = quarter * 32 + lane;  // row of its tile: tensor-memory lane
    const uint32_t mine = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t ts = mine + F::kS + x * 96, to = mine + x * D;
    uint32_t ph = 0;   // phase of sf; of of, once a step on
    uint32_t ph1 = 0;  // (first set) phase of the second's sf
    while (take()) {
      const bool both = F::kSets > 1 && s.rows > 128;
      const int nb = s.b1 - s.b0, n = nb * (both ? 2 : 1);
      const int row0 = (both ? x * 128 : 0) + quarter * 32;
      const bool alive = row0 + lane < s.rows, any = row0 < s.rows;  // the row's, the warp's
      float *part = a.px_ws + ((int64_t)blockIdx.x + s.item) * (F::kSets * F::kPart) + x * F::kPart;
      if (s.parts > 0 && tid == 0) a.px_parts[s.item] = make_int4((int)blockIdx.x, s.parts, 0, 0);
      if (F::kSets > 1 && x >= n) {  // a single block, the other set's
        if (c0 == 0 && lane == 0) tc_mbar_arrive(&ql);
        part[128 * D + in_tile] = -INFINITY;
        part[128 * (D + 1) + in_tile] = 0.f;
        c0 += nb;
        continue;
      }
      // Q: each row scaled by a power of two so that its largest value lies in [2^14, 2^15), as fp16;
      // the softmax's factor is what is left, its sign goes with Q
      float f = 0.f;
      if (any) {
        const int row = s.tile * F::kRows + row0 + lane, of_seq = a.T * a.group;
        const int sq = s.first + row / of_seq, rt = row % of_seq, t = rt / a.group;
        const unsigned short *qp = reinterpret_cast<const unsigned short *>(a.q) + ((int64_t)sq * a.T + t) * a.q_stride +
                                   ((int64_t)s.h * a.group + rt - t * a.group) * D;
        const bool vec = (reinterpret_cast<uintptr_t>(a.q) & 15) == 0 && a.q_stride % 8 == 0;
        uint32_t top = 0;
        auto larger = [&](const uint4 &v) {
          top = kv_max2(kv_max2(top, v.x & 0x7fff7fffu, DT), v.y & 0x7fff7fffu, DT);
          top = kv_max2(kv_max2(top, v.z & 0x7fff7fffu, DT), v.w & 0x7fff7fffu, DT);
        };
        float up = 0.f;
        auto factors = [&]() {
          const float mx = fmaxf(kv_wide_lo(top, DT), kv_wide_hi(top, DT));
          int e = (__float_as_int(mx) >> 23) & 0xff;  // (an infinity takes the largest exponent)
          e = e < 16 ? 16 : e;
          up = __int_as_float((127 + 14 + 127 - e) << 23);
          f = fabsf(a.scale_log2) / up;
          if (a.scale_log2 < 0.f) up = -up;
        };
        auto put = [&](int c, const uint4 (&v)[4]) {  // channels c .. c + 31
          uint32_t u[16];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) u[4 * j + i] = kv_pack_half(kv_wide_lo(w[i], DT) * up, kv_wide_hi(w[i], DT) * up);
          }
          if (F::kQShared && x == 1) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint4 *>(qst + c / 64 * (128 * 128) + in_tile * 128 + ((((c / 8 + j) & 7) ^ (in_tile & 7)) * 16)) =
                  make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
          } else {
            px_st16(mine + F::kQ + x * (D / 2) + c / 2, u);
          }
        };
        constexpr int kHeld = D <= 128 ? D : 0;  // channels of a row that the registers hold
        uint4 v[kHeld > 0 ? kHeld / 8 : 4];
        if (kHeld > 0 && vec) {
#pragma unroll
          for (int j = 0; j < kHeld / 8; ++j)
            v[j] = alive ? __ldg(reinterpret_cast<const uint4 *>(qp) + j) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int j = 0; j < kHeld / 8; ++j) larger(v[j]);
          if (c0 == 0) {
            __syncwarp();
            if (lane == 0) tc_mbar_arrive(&ql);
          }
          factors();
          if (both || x == 0) {
#pragma unroll
            for (int j = 0; j < kHeld / 8; j += 4) {
              const uint4 w[4] = {v[j], v[j + 1], v[j + 2], v[j + 3]};
              put(8 * j, w);
            }
          }
        } else {  // wide heads, rows that start anywhere: read twice
          auto fetch = [&](int c) {
            if (!alive) return make_uint4(0, 0, 0, 0);
            return vec ? __ldg(reinterpret_cast<const uint4 *>(qp + c)) : px_load8(qp + c);
          };
#pragma unroll 8
          for (int c = 0; c < D; c += 8) larger(fetch(c));
          if (c0 == 0) {
            __syncwarp();
            if (lane == 0) tc_mbar_arrive(&ql);
          }
          factors();
          if (both || x == 0) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              const uint4 w[4] = {fetch(c), fetch(c + 8), fetch(c + 16), fetch(c + 24)};
              put(c, w);
            }
          }
        }
        if (both || x == 0) {
          px_st_wait();
          if (F::kQShared && x == 1) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
      } else if (c0 == 0 && lane == 0) {
        tc_mbar_arrive(&ql);
      }
      px_fence_before();
      __syncwarp();
      if (lane == 0 && (both || x == 0)) tc_mbar_arrive(&qf[x]);

      // O's reference, a logit plus the log2 of its block's value scale; the weights' own, the
      // largest logit of those looked for; the weights' sum, in units of 2^own
      float ref = 0.f, own = 0.f, l = 0.f;
      bool begun = false;
      const int by = F::kSets > 1 && !both ? 2 : 1;  // from one of its blocks to the next
#pragma unroll 1
      for (int blk = c0 + (by == 2 ? x : 0); blk < c0 + nb; blk += by) {
        const bool first = blk < c0 + by;
        const int slot = blk % kPxMeta;
        ok = wait(&sf[x], ph, 1);
        if (!ok) break;
        px_fence_after();
        uint32_t r[2][32];
        if (any) {
          f8_ld<32>(ts, r[0]);
          f8_ld<32>(ts + 32, r[1]);
        }
        // (S is there, so its keys were converted, so the block's scales had come)
        const bool bad = meta_bad[slot] != 0;
        // (a scale of 0, and of a block that is none, far below any other)
        const float ff = f * meta[slot][0], lv = bad ? -INFINITY : fmaxf(px_log2(meta[slot][1]), -200.f);
        if (any) {
          f8_ld_wait<32>(r[0]);
          f8_ld_wait<32>(r[1]);
        }
        // P = 2^(logit + up): the weight times the value scale, in units of 2^(ref - kPxLift).  Whether
        // a weight has outgrown the reference its row's sum tells: no largest logit is looked for
        // where all is as expected.
        bool grow = false;
        float shrink = 1.f;
        if (any) {
          float up = lv - ref + kPxLift, sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            float u = __uint_as_float(r[j >> 4][2 * (j & 15)]), v = __uint_as_float(r[j >> 4][2 * (j & 15) + 1]);
            px_fma2(u, v, ff, up);
            u = kv_exp2(u);
            v = kv_exp2(v);
            px_add2(sum[2 * (j & 1)], sum[2 * (j & 1) + 1], u, v);
            r[0][j] = kv_pack_half(u, v);  // (in the place of values that are used up)
          }
          float total = (sum[0] + sum[2]) + (sum[1] + sum[3]);
          // P's unit, as a weight.  Far above the weights' own (value scales far below the reference's)
          // P loses weights that count
          const float unit = -up - own;
          // (or no reference yet, or too large for fp16)
          if (__any_sync(0xffffffffu, !begun || total > kPxFull || unit > 80.f)) {
            if (!bad) {
              f8_ld<32>(ts, r[0]);
              f8_ld<32>(ts + 32, r[1]);
              f8_ld_wait<32>(r[0]);
              f8_ld_wait<32>(r[1]);
              float mx = -INFINITY, my = -INFINITY;
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                mx = fmaxf(mx, fmaxf(__uint_as_float(r[0][j]), __uint_as_float(r[0][j + 1])));
                my = fmaxf(my, fmaxf(__uint_as_float(r[1][j]), __uint_as_float(r[1][j + 1])));
              }
              const float bm = fmaxf(mx, my) * ff;
              grow = !begun || bm + lv > ref;
              if (grow) {
                shrink = begun ? kv_exp2(ref - (bm + lv)) : 0.f;
                ref = bm + lv;
              }
              const float top = begun ? fmaxf(own, bm) : bm;
              // (chosen, not multiplied by 0: a first block far below 0 makes the factor infinite)
              l = begun ? l * kv_exp2(own - top) : 0.f;
              own = top;
              begun = true;
              up = lv - ref + kPxLift;
              total = 0.f;
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                float u = __uint_as_float(r[j >> 4][2 * (j & 15)]), v = __uint_as_float(r[j >> 4][2 * (j & 15) + 1]);
                total += kv_exp2(fmaf(u, ff, -own)) + kv_exp2(fmaf(v, ff, -own));
                r[0][j] = kv_pack_half(kv_exp2(fmaf(u, ff, up)), kv_exp2(fmaf(v, ff, up)));
              }
              l += total;
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) r[0][j] = 0;
            }
          } else {
            l = fmaf(total, kv_exp2(unit), l);
          }
        }
        px_fence_before();
        __syncwarp();
        if (lane == 0) tc_mbar_arrive(&sr[x]);
        // the product before this one: done with P, with its values, with O
        if (!first) {
          ok = wait(&of[x], ph ^ 1, 1);
          if (!ok) break;
          px_fence_after();
          if (__any_sync(0xffffffffu, grow)) {
            const float to_new = grow ? shrink : 1.f;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              f8_ld<16>(to + c, o);
              f8_ld_wait<16>(o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * to_new);
              px_st16(to + c, o);
            }
          }
        }
        if (any) {
          px_st32(ts + 64, r[0]);
          px_st_wait();
        }
        px_fence_before();
        __syncwarp();
        if (lane == 0) tc_mbar_arrive(&pf[x]);
        ph ^= 1;
      }
      if (!ok) break;
      ok = wait(&of[x], ph ^ 1, 1);
      if (!ok) break;
      px_fence_after();
      if (F::kSets > 1 && x == 0) {
        // one Q for both sets: the other's last scores have to be done before the next Q comes
        const int other = both ? nb : nb / 2;
        ph1 ^= other & 1;
        if (!both && other > 0) {
          ok = wait(&sf[F::kSets - 1], ph1 ^ 1, 1);
          if (!ok) break;
        }
      }
      if (any) {
        // O in the weights' units: 2^(ref - own), a value scale as a rule and down to 2^-126, less what
        // rounding takes, and 2^-kPxLift.  (In one exponent the two would be flushed to 0.)
        const float units = kv_exp2(ref - own + 0.5f), down = kv_exp2(-kPxLift - 0.5f);
        float4 *out = reinterpret_cast<float4 *>(part) + in_tile;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          f8_ld<32>(to + c, o);
          f8_ld_wait<32>(o);
          if (alive) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              out[(c + j) / 4 * 128] = make_float4(__uint_as_float(o[j]) * down * units, __uint_as_float(o[j + 1]) * down * units,
                                                   __uint_as_float(o[j + 2]) * down * units, __uint_as_float(o[j + 3]) * down * units);
          }
        }
        if (alive) {
          part[128 * D + in_tile] = begun ? own : -INFINITY;
          part[128 * (D + 1) + in_tile] = l * kKvLifted;
        }
      }
      c0 += nb;
    }
  }
  px_fence_before();
  __syncwarp();
  __syncthreads();
  if (abort_flag != 0) {
    // after an abort nothing may be in flight when the CTA frees its tensor memory and exits
    if (warp == kScores || warp == kSums) {
      if (f8_elect()) tc_commit(&fin);
      __syncwarp();
      const bool drained = tc_mbar_wait(&fin, 0, a.timeout_ns);
      if (lane == 0 && a.status != nullptr) atomicOr(a.status, drained ? kTcStatusMma : kTcStatusMma | kTcStatusDrain);
    }
    if (warp == kLoad) {
      bool drained = true;
      for (int i = c0 > R ? c0 - R : 0; i < c0; ++i)
        if (!tc_mbar_wait(&rawf[i % R], (uint32_t)(i / R) & 1u, a.timeout_ns)) drained = false;
      if (!drained && lane == 0 && a.status != nullptr) atomicOr(a.status, kTcStatusDrain);
    }
    __syncwarp();
    __syncthreads();
  }
  if (warp == kSums) {
    px_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// ------------------------------------------------------------------ join
// A sequence's rows of a head: the parts of its own blocks and of its group's shared ones,
// in that order; zeros where there are none.  A thread adds up sixteen channels of a row (four
// times four), kGroups threads share the parts of the same channels.  grid (S, items, pieces
// of a tile's rows).  Bound by its chain of dependent reads (lengths, where the parts are,
// parts): small CTAs, so that all are there at once, and several reads of a thread on their way.
constexpr int kPxJoinThreads = 128;
template <int D, int NT, int kGroups>
__global__ void __launch_bounds__(kPxJoinThreads) k_kv8_prefix_join(const KvArgs a, int ctas) {
  constexpr int kAlong = kPxJoinThreads / kGroups, kStep = D / 16;  // threads along the channels and rows; quads between a thread's
  using F = PxForm<D>;
  __shared__ float4 sums[kGroups > 1 ? kGroups - 1 : 1][4][kGroups > 1 ? kAlong : 1];
  __shared__ float2 stats[kGroups > 1 ? kGroups - 1 : 1][kGroups > 1 ? kAlong : 1];
  pdl_trigger();
  const int s = blockIdx.x, item = blockIdx.y, items = a.heads * a.row_tiles;
  // (lens, prefix and firsts are older than the kernel before, which let this one start after
  // its own wait)
  const KvSeen seen = kv_seen<true>(a, s);
  const int h = item / a.row_tiles, row0 = (item - h * a.row_tiles) * NT * 8;
  const int rows = a.T * a.group - row0 < NT * 8 ? a.T * a.group - row0 : NT * 8;
  const int64_t own_item = (int64_t)s * items + item;
  const int along = threadIdx.x % kAlong, grp = threadIdx.x / kAlong;
  const int idx = blockIdx.z * kAlong + along, quad = idx / rows, r = idx - quad * rows;
  const bool on = quad < kStep;
  // the row's place among those of its group
  int px_item = 0, px_set = 0, rr = 0, sets = 0;
  if (seen.from > 0 && on) {
    const int g = kv_group_of(a, s);
    const KvGroup k = kv_group(a, g);
    const int of_seq = a.T * a.group, row = (s - k.first) * of_seq + row0 + r, tile = row / F::kRows;
    const bool both = F::kSets > 1 && (k.end - k.first) * of_seq - tile * F::kRows > 128;
    const int in_tile = row - tile * F::kRows;
    px_item = (px_tile0<D>(a, g, k.first) + tile) * a.heads + h;
    sets = F::kSets > 1 && !both ? 2 : 1;
    px_set = both ? in_tile / 128 : 0;
    rr = in_tile % 128;
  }
  pdl_wait();  // by every CTA: the next kernel counts on it
  // (a kernel whose wait ran out leaves its entries as the scratch memory had them: what is
  // read stays within the partial results)
  int4 of = make_int4(0, 0, 0, 0), w = of;
  if (seen.count > 0) of = __ldcg(&a.parts[own_item]);
  if (sets > 0) w = __ldcg(&a.px_parts[px_item]);
  if (of.x < 0 || of.y < 0 || (int64_t)of.x + of.y > a.workers) of.y = 0;
  if (w.x < 0 || w.y < 0 || (int64_t)w.x + w.y > ctas) w.y = 0;
  const float *const own = a.ws + ((int64_t)of.x + own_item) * kv_part<D, NT>();
  const float *const px = a.px_ws + ((int64_t)w.x + px_item) * (F::kSets * F::kPart) + px_set * F::kPart;
  // two sets of a CTA's part lie one behind the other, with one set it is the next CTA's
  const int64_t step = sets == 2 ? F::kPart : F::kSets * F::kPart;
  float m = -INFINITY, den = 0.f;
  float4 v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float fm, float fden, const float4 (&f)[4]) {
    if (fm == -INFINITY && fden == 0.f) return;  // (a set that had no block has no sums, either)
    const float big = fmaxf(m, fm), z = big == -INFINITY ? 0.f : big, x = kv_exp2(m - z), y = kv_exp2(fm - z);
    m = big;
    den = den * x + fden * y;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j].x = v[j].x * x + f[j].x * y;
      v[j].y = v[j].y * x + f[j].y * y;
      v[j].z = v[j].z * x + f[j].z * y;
      v[j].w = v[j].w * x + f[j].w * y;
    }
  };
  constexpr int kOnWay = kGroups > 1 ? 4 : 2;  // parts whose reads are on their way (many parts: 84 us with two, 83)
  if (on) {
    const int total = of.y + w.y * sets;
    for (int i0 = grp; i0 < total; i0 += kOnWay * kGroups) {
      float fm[kOnWay], fden[kOnWay];
      float4 f[kOnWay][4];
#pragma unroll
      for (int k = 0; k < kOnWay; ++k) {
        const int i = i0 + k * kGroups;
        if (i < total) {
          const bool mine = i < of.y;
          const float *q = mine ? own + (int64_t)i * kv_part<D, NT>() : px + (i - of.y) * step;
          fm[k] = __ldcg(q + (mine ? NT * 8 * D + r : 128 * D + rr));
          fden[k] = __ldcg(q + (mine ? NT * 8 * (D + 1) + r : 128 * (D + 1) + rr));
          q += mine ? r * D + quad * 4 : (quad * 128 + rr) * 4;
#pragma unroll
          for (int j = 0; j < 4; ++j) f[k][j] = __ldcg(reinterpret_cast<const float4 *>(q + j * kStep * (mine ? 4 : 128 * 4)));
        }
      }
#pragma unroll
      for (int k = 0; k < kOnWay; ++k)
        if (i0 + k * kGroups < total) add(fm[k], fden[k], f[k]);
    }
  }
  if constexpr (kGroups > 1) {
    if (grp > 0) {
      stats[grp - 1][along] = make_float2(m, den);
#pragma unroll
      for (int j = 0; j < 4; ++j) sums[grp - 1][j][along] = v[j];
    }
    __syncthreads();
    if (grp > 0) return;
#pragma unroll
    for (int k = 0; k < kGroups - 1; ++k) {
      const float4 f[4] = {sums[k][0][along], sums[k][1][along], sums[k][2][along], sums[k][3][along]};
      add(stats[k][along].x, stats[k][along].y, f);
    }
  }
  if (!on) return;
  const int64_t at_row = kv_out_row(a, s, h, row0 + r);
  const float inv = den == 0.f ? 0.f : kKvLifted * (1.f / den);
  unsigned short *out = reinterpret_cast<unsigned short *>(a.out) + at_row * D + quad * 4;
  const bool vec = (reinterpret_cast<uintptr_t>(a.out) & 7) == 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint2 o = make_uint2(f8_pack16(v[j].x * inv, v[j].y * inv, a.dtype), f8_pack16(v[j].z * inv, v[j].w * inv, a.dtype));
    unsigned short *p = out + j * kStep * 4;
    if (vec) {
      *reinterpret_cast<uint2 *>(p) = o;
    } else {
      p[0] = (unsigned short)o.x;
      p[1] = (unsigned short)(o.x >> 16);
      p[2] = (unsigned short)o.y;
      p[3] = (unsigned short)(o.y >> 16);
    }
  }
  if (quad == 0 && a.lse != nullptr) a.lse[at_row] = kv_lse(m, den);
}

}  // namespace gemv
